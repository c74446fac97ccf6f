// Attention of many rows over the 8-bit cache: the same formula as in
// kv_attn_rows.hip, on tiles.
//
// A workgroup of four wavefronts owns 128 rows (tokens times the query heads
// that share a cache head), 32 a wavefront, and walks the pages that any of
// them sees.  A page's codes are decoded once for the workgroup, into LDS as
// FP16 operands of v_mfma_f32_32x32x16_f16 in the order in which lanes read
// them (no bank conflicts), one page ahead, the page after that on its way
// into registers meanwhile.  Scores come out transposed (a lane has one row's
// scores of 32 tokens of the page, its partner 32 lanes on the others), so
// the softmax needs one exchange, and the weights are the next product's
// operand where they are.  Heavy tiles (the last of a causal prompt) start
// first; the workgroups of a cache head are neighbours modulo the number of
// heads, so that an XCD's L2 keeps few heads' pages.
#include "kv_attn.h"

namespace tern {
namespace {

constexpr int kTileWaves = 4, kCus = 256;

template <int D>
__global__ __launch_bounds__(64 * kTileWaves, D <= 128 ? 2 : 1) void attn_tile_kernel(const AttnArgs a) {
  constexpr int THREADS = 64 * kTileWaves, ROWS = 32 * kTileWaves;
  constexpr int KS = D / 16;                        // products of 16 dimensions in a score
  constexpr int DB = D / 32;                        // blocks of 32 dimensions of the sums
  constexpr int PIECES = kPage * D / 16 / THREADS;  // of 16 codes a thread, keys and values each
  __shared__ kw4_t lk[2][kPage * D / 8], lv[2][kPage * D / 8];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c32 = lane & 31, hq = lane >> 5;
  int bid = blockIdx.x;
  const int head = bid % a.c.heads;
  bid /= a.c.heads;
  const int s = bid % a.b.count;
  bid /= a.b.count;
  const int part = bid % a.parts;
  int tile = a.tiles - 1 - bid / a.parts;
  // Where the card holds the whole grid at once, every CU's second workgroup is
  // the lighter the heavier its first.
  const int per = a.c.heads * a.b.count * a.parts, firsts = (kCus + per - 1) / per;
  if (a.tiles * per <= 2 * kCus && bid / a.parts >= firsts) tile = bid / a.parts - firsts;
  const Span sp = span_of(a.b, s);
  const int total = sp.n * a.group;
  if (tile * ROWS >= total) return;
  const Range all = range_of_rows(a, sp, tile * ROWS, min(tile * ROWS + ROWS, total) - 1);
  const Parts parts = parts_of(a, all);
  if (part >= parts.count) return;
  const Range mine = part_of(all, parts, part);

  const int r = tile * ROWS + wave * 32 + c32, j = r / a.group, h = r % a.group;
  const bool there = r < total;
  const Sees sees = sees_of(a, sp, sp.from + j, there);
  // tokens that every row of the wavefront sees, and that any does
  int low = there ? sees.low : 0, high = there ? sees.high : 0x7fffffff;
  int least = there ? sees.low : 0x7fffffff, most = there ? sees.high : 0;
  for (int i = 1; i < 32; i <<= 1) {
    low = max(low, __shfl_xor(low, i));
    high = min(high, __shfl_xor(high, i));
    least = min(least, __shfl_xor(least, i));
    most = max(most, __shfl_xor(most, i));
  }
  low = __builtin_amdgcn_readfirstlane(low);
  high = __builtin_amdgcn_readfirstlane(high);
  least = __builtin_amdgcn_readfirstlane(least);
  most = __builtin_amdgcn_readfirstlane(most);

  kh8_t q[KS];
  const uint16_t* const from = a.q + (int64_t)(sp.first + (there ? j : 0)) * a.q_stride + (head * a.group + h) * D;
#pragma unroll
  for (int i = 0; i < KS; ++i) q[i] = *reinterpret_cast<const kh8_t*>(from + 16 * i + 8 * hq);
  kf16_t o[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int v = 0; v < 16; ++v) o[d][v] = 0.f;
  Row row = new_row();

  // A thread's pieces: of the keys 16 dimensions (16 st ..) of a token, of the
  // values 16 tokens (16 part ..) of a dimension; a wavefront's 64 are
  // neighbours in LDS.
  kw4_t kr[PIECES], vr[PIECES];
  auto page_at = [&](int p) { return p < mine.end ? __builtin_amdgcn_readfirstlane(page_of(a.b, a.c, s, p)) : -1; };
  auto load = [&](int id) {
    const size_t at = ((size_t)max(id, 0) * a.c.heads + head) * (kPage * D);
    const __amdgpu_buffer_rsrc_t fk = kv_buffer(a.c.k + at, id < 0 ? 0 : kPage * D), fv = kv_buffer(a.c.v + at, id < 0 ? 0 : kPage * D);
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int st = i * kTileWaves + wave;
      kr[i] = kv_load16(fk, ((st / 4 * 4 + lane / 4 % 4) * 64 + st % 4 * 16 + lane / 16 * 4 + lane % 4) * 16);
      const int part = st % 4, d = st / 4 * 64 + lane;
      vr[i] = kv_load16(fv, ((d / 16 * 4 + part) * 16 + d % 16) * 16);
    }
  };
  auto decode = [&](kw4_t* ks, kw4_t* vs) {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int st = i * kTileWaves + wave;
      kw4_t* const k = ks + (st * 2 + lane / 32) * 64 + lane % 32;
      k[0] = __builtin_bit_cast(kw4_t, codes8(kr[i][0], kr[i][1]));
      k[32] = __builtin_bit_cast(kw4_t, codes8(kr[i][2], kr[i][3]));
      const int part = st % 4, d = st / 4 * 64 + lane;
      kw4_t* const v = vs + (d / 32 * 4 + part) * 64 + d % 32;
      v[0] = __builtin_bit_cast(kw4_t, codes8(vr[i][0], vr[i][2]));
      v[32] = __builtin_bit_cast(kw4_t, codes8(vr[i][1], vr[i][3]));
    }
  };

  auto compute = [&](int p, int id, const kw4_t* ks, const kw4_t* vs) {
    if (p * kPage >= most || p * kPage + kPage <= least) return;  // none of the wavefront's rows sees it
    const size_t at = (size_t)max(id, 0) * a.c.heads + head;
    const float kscale = kv_const(a.c.ks, at) * a.scale, vscale = kv_const(a.c.vs, at);
    kf16_t z[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
#pragma unroll
      for (int v = 0; v < 16; ++v) z[b][v] = 0.f;
#pragma unroll
      for (int i = 0; i < KS; ++i)
        z[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(kh8_t, ks[(i * 2 + b) * 64 + lane]), q[i], z[b], 0, 0, 0);
    }
    const bool whole = id >= 0 && p * kPage >= low && p * kPage + kPage <= high;
    float by = kscale, best = -INFINITY;  // the scores are by z
    if (!whole) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int token = p * kPage + 32 * b + 8 * (v / 4) + 4 * hq + v % 4;
          z[b][v] = id < 0 || token < sees.low || token >= sees.high ? -INFINITY : z[b][v] * by;
        }
      by = 1.0f;
    }
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int v = 0; v < 16; ++v) best = fmaxf(best, z[b][v]);
    best = fmaxf(best, __shfl_xor(best, 32)) * by;
    float lift, back;
    const float factor = step_row(row, best, vscale == 0.f ? 1.f : vscale, lift, back);
    const float shift = lift - top_of(row);
    if (__any(factor != 1.0f)) {
#pragma unroll
      for (int d = 0; d < DB; ++d) o[d] *= factor;
    }
    kh8_t w[4];
    float sum = 0.f;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(z[b][v], by, shift));
        sum += e;
        w[b * 2 + v / 8][v % 8] = (_Float16)e;
      }
    row.sum += sum * back;
    if (vscale == 0.f) return;  // values of 0, whatever the codes
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int t = 0; t < 4; ++t)
        o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(kh8_t, vs[(d * 4 + t) * 64 + lane]), w[t], o[d], 0, 0, 0);
  };

  __builtin_amdgcn_s_waitcnt(0x0F70);  // the queries, once: in the loop their wait would be for the pages too
  int p = mine.begin, id = page_at(p);
  if (p < mine.end) {
    load(id);
    decode(lk[0], lv[0]);
    load(page_at(p + 1));
    __syncthreads();
  }
  for (int cur = 0; p < mine.end; ++p, cur ^= 1) {
    const int next = page_at(p + 1);
    compute(p, id, lk[cur], lv[cur]);
    if (p + 1 < mine.end) {
      decode(lk[cur ^ 1], lv[cur ^ 1]);
      if (p + 2 < mine.end) load(page_at(p + 2));
    }
    id = next;
    __syncthreads();
  }

  float sum = row.sum;
  sum += __shfl_xor(sum, 32);
  if (!there) return;
  const size_t out = (size_t)(sp.first + j) * a.q_heads + head * a.group + h;
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const kf4_t x = {o[d][4 * v], o[d][4 * v + 1], o[d][4 * v + 2], o[d][4 * v + 3]};
      store_row<D>(a, parts, part, out, d * 32 + 8 * v + 4 * hq, x * (row.unit / kLift), row.top, sum);
    }
}

template <int D>
hipError_t tile(const AttnArgs& a, long long grid, hipStream_t s) {
  hipLaunchKernelGGL((attn_tile_kernel<D>), dim3((unsigned)grid), dim3(64 * kTileWaves), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_tile(const AttnArgs& a, int dim, hipStream_t s) {
  const long long grid = (long long)a.b.count * a.c.heads * a.parts * a.tiles;
  if (!kv_grid_fits(grid, 64 * kTileWaves)) return hipErrorInvalidConfiguration;
  if (dim == 64) return tile<64>(a, grid, s);
  return dim == 128 ? tile<128>(a, grid, s) : tile<256>(a, grid, s);
}

}  // namespace tern
