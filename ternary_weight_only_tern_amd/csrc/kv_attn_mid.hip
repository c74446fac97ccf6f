// Attention over the 8-bit cache on tiles of 64 rows: the formula of
// kv_attn_rows.hip, with pages decoded into LDS once for the workgroup as in
// kv_attn_tile.hip.
//
// Each of four wavefronts has 16 rows, the columns of v_mfma_f32_16x16x32_f16,
// and walks the pages that any of the tile's rows sees.  A page's codes are in the
// order of these instructions' operands already (kv.h): 16 bytes become two
// operands, 1 KB a wavefront's store.  A step multiplies the next page's keys with
// the queries, decodes the keys after those and the next values, asks for the
// codes behind them, and turns this page's scores into weights and sums.
//
// Bound by the chain of a wavefront's step, about 3000 cycles at 128 dimensions
// (scores 740, most of it the LDS, decoding and requests 970, softmax 850, sums
// 330), which a second workgroup on the CU hides in part: every wavefront reads
// all operands for 16 rows, so that long prompts are better off with 32
// (kv_attn_tile.hip), and few rows, short prompts and small dimensions here.  A
// prompt of 512 tokens, 32 heads over 8, 15-16 us (128-row tiles 19.5); 64
// sequences of 1000 with 10 rows 36-42 (44.0); two prompts of 2048, 12 heads of 64,
// 34-36 (42.6), 360 TFLOP/s; one of 2048, 16 heads of 256 over 8, 80 (97).  With this
// page's scores multiplied in the step itself the last took 91, the others as long.
#include "kv_attn.h"

namespace tern {
namespace {

constexpr int kMidWaves = 4;

template <int D>
__global__ __launch_bounds__(64 * kMidWaves, D <= 128 ? 2 : 1) void attn_mid_kernel(const AttnArgs a) {
  constexpr int THREADS = 64 * kMidWaves, ROWS = kAttnMid;
  constexpr int C = D / 64, DT = D / 16;  // a wavefront's pieces of 16 codes a lane, of keys and of values; blocks of the sums
  __shared__ kw4_t lk[2][kPage * D / 8], lv[2][kPage * D / 8];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, kq = lane >> 4;
  const Work work = work_of(a, D == 128);
  const int s = work.s, head = work.head, tile = work.tile;
  const Span sp = span_of(a.b, s);
  const int total = sp.n * a.group;
  if (tile * ROWS >= total) return;
  const Range all = range_of_rows(a, sp, tile * ROWS, min(tile * ROWS + ROWS, total) - 1);
  const Parts parts = parts_of(a, all);
  if (work.part >= parts.count) return;
  const Range mine = part_of(all, parts, work.part);

  const int r = tile * ROWS + wave * 16 + col, j = r / a.group, h = r % a.group;
  const bool there = r < total;
  const Sees sees = sees_of(a, sp, sp.from + j, there);
  // tokens that every row of the wavefront sees, and that any does
  int low = there ? sees.low : 0, high = there ? sees.high : 0x7fffffff;
  int least = there ? sees.low : 0x7fffffff, most = there ? sees.high : 0;
  for (int i = 1; i < 16; i <<= 1) {
    low = max(low, __shfl_xor(low, i));
    high = min(high, __shfl_xor(high, i));
    least = min(least, __shfl_xor(least, i));
    most = max(most, __shfl_xor(most, i));
  }
  low = __builtin_amdgcn_readfirstlane(low);
  high = __builtin_amdgcn_readfirstlane(high);
  least = __builtin_amdgcn_readfirstlane(least);
  most = __builtin_amdgcn_readfirstlane(most);

  kh8_t q[C][2];
  const uint16_t* const from = a.q + (int64_t)(sp.first + (there ? j : 0)) * a.q_stride + (head * a.group + h) * D;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int u = 0; u < 2; ++u) q[c][u] = *reinterpret_cast<const kh8_t*>(from + 64 * c + 16 * kq + 8 * u);
  kf4_t o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) o[d] = kf4_t{0.f, 0.f, 0.f, 0.f};
  Row row = new_row();

  // A page that is not there, or lies behind the last, reads as page 0, and is
  // masked or not looked at.  Its number and scales come by vector loads, a step
  // and more ahead, as in kv_attn_tile.hip.
  kw4_t kr[C], vr[C];
  const __amdgpu_buffer_rsrc_t table = kv_buffer(a.b.pages + (size_t)s * a.b.max_pages, min(a.b.max_pages, kMaxTokens / kPage) * 4);
  auto load_id = [&](int p) { return (int)__builtin_amdgcn_raw_buffer_load_b32(table, p * 4, 0, 0); };
  auto id_of = [&](int raw, int p) {
    const int id = __builtin_amdgcn_readfirstlane(raw);
    return p < mine.end && id >= 0 && id < a.c.pages ? id : -1;
  };
  auto place_in = [&](int id) { return (size_t)max(id, 0) * a.c.heads + head; };
  int zero;
  asm("v_mov_b32 %0, 0" : "=v"(zero));  // the same in every lane, which the compiler does not see
  auto load_scale = [&](const float* scales, size_t at) { return (scales + at)[zero]; };
  auto load_page = [&](const uint8_t* pages, size_t at, kw4_t* to) {
    const uint8_t* const f = pages + at * (kPage * D);
#pragma unroll
    for (int i = 0; i < C; ++i) to[i] = *reinterpret_cast<const kw4_t*>(f + ((i * kMidWaves + wave) * 64 + lane) * 16);
  };
  auto decode = [&](const kw4_t* codes, kw4_t* to) {
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int u = 0; u < 2; ++u)
        to[((i * kMidWaves + wave) * 2 + u) * 64 + lane] = __builtin_bit_cast(kw4_t, codes8(codes[i][2 * u], codes[i][2 * u + 1]));
  };
  auto operand = [&](const kw4_t* in, int piece, int u) { return __builtin_bit_cast(kh8_t, in[(piece * 2 + u) * 64 + lane]); };
  // whether any of the wavefront's rows sees page p
  auto seen = [&](int p) { return p * kPage < most && p * kPage + kPage > least; };

  int p = mine.begin, cur = 0;
  int raw = load_id(p), raw1 = load_id(p + 1), raw2 = load_id(p + 2), raw3 = load_id(p + 3);
  int id = id_of(raw, p), id1 = id_of(raw1, p + 1), id2 = id_of(raw2, p + 2);
  const size_t at0 = place_in(id), at1 = place_in(id1);
  load_page(a.c.k, at0, kr);  // the first pages together
  load_page(a.c.v, at0, vr);
  kw4_t k1[C], v1[C];
  load_page(a.c.k, at1, k1);
  load_page(a.c.v, at1, v1);
  float ks0 = load_scale(a.c.ks, at0), vs0 = load_scale(a.c.vs, at0);  // this page's, the next one's
  float ks1 = load_scale(a.c.ks, at1), vs1 = load_scale(a.c.vs, at1);
  kf4_t z[4];
  auto multiply = [&](const kw4_t* ks, kf4_t* z) {  // a page's scores
#pragma unroll
    for (int t = 0; t < 4; ++t) z[t] = kf4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int t = 0; t < 4; ++t) z[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(operand(ks, c * 4 + t, u), q[c][u], z[t], 0, 0, 0);
  };
  if (mine.begin < mine.end) {
    decode(kr, lk[0]);
    decode(vr, lv[0]);
    decode(k1, lk[1]);
    load_page(a.c.k, place_in(id2), kr);
#pragma unroll
    for (int i = 0; i < C; ++i) vr[i] = v1[i];
    __syncthreads();
    multiply(lk[0], z);
    __syncthreads();
  }
  for (; p < mine.end; ++p, cur ^= 1) {
    const kw4_t* const vs = lv[cur];
    const bool any = seen(p);
    // Behind the last page the next scores are of what lies there, and not used.
    kf4_t next[4];
    multiply(lk[cur ^ 1], next);
    decode(kr, lk[cur]);
    decode(vr, lv[cur ^ 1]);
    const size_t at2 = place_in(id2);
    const float ks2 = load_scale(a.c.ks, at2), vs2 = load_scale(a.c.vs, at2);
    const int id3 = id_of(raw3, p + 3);
    raw3 = load_id(p + 4);
    load_page(a.c.k, place_in(id3), kr);
    load_page(a.c.v, at2, vr);
    if (any) {
      const float vscale = __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__float_as_int(vs0)));
      float by = ks0 * a.scale, best = -INFINITY;  // the scores are by z
      const int first = p * kPage, side = first + 16 * kq;
      const bool none = id < 0, below = none || first < low, above = first + kPage > high;
      if (below || above) {
        if (!(by > 0.f)) {  // of no use beside infinities
#pragma unroll
          for (int t = 0; t < 4; ++t) z[t] *= by;
          by = 1.0f;
        }
        const int begin = none ? kPage : sees.low - side, end = sees.high - side;
#pragma unroll
        for (int x = 0; x < 16; ++x)
          if (x < begin || x >= end) z[x / 4][x % 4] = -INFINITY;
      }
#pragma unroll
      for (int x = 0; x < 16; ++x) best = fmaxf(best, z[x / 4][x % 4]);
      best = max_of_32(max_of_16(best)) * by;
      float lift, back;
      const float factor = step_row(row, best, vscale == 0.f ? 1.f : vscale, lift, back);
      const float shift = lift - top_of(row);
      if (__any(factor != 1.0f)) {
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] *= factor;
      }
      kh8_t w[2];
      float sum = 0.f;
#pragma unroll
      for (int x = 0; x < 16; x += 2) {  // the sum is of the rounded weights, as in kv_attn_tile.hip
        kh2_t two;
        two.x = (_Float16)__builtin_amdgcn_exp2f(__builtin_fmaf(z[x / 4][x % 4], by, shift));
        two.y = (_Float16)__builtin_amdgcn_exp2f(__builtin_fmaf(z[x / 4][x % 4 + 1], by, shift));
        w[x / 8][x % 8] = two.x;
        w[x / 8][x % 8 + 1] = two.y;
        sum = __builtin_amdgcn_fdot2(two, kh2_t{(_Float16)1.0f, (_Float16)1.0f}, sum, false);
      }
      row.sum += sum * back;
      if (vscale == 0.f) w[0] = w[1] = kh8_t{0, 0, 0, 0, 0, 0, 0, 0};  // values of 0, whatever the codes
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(operand(vs, d, u), w[u], o[d], 0, 0, 0);
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) z[t] = next[t];
    id = id1;
    id1 = id2;
    id2 = id3;
    ks0 = ks1;
    vs0 = vs1;
    ks1 = ks2;
    vs1 = vs2;
    __syncthreads();
  }

  float sum = row.sum;
  sum += __shfl_xor(sum, 16);
  sum += __shfl_xor(sum, 32);
  if (!there) return;
  if (parts.count == 1) {
    const size_t out = ((size_t)(sp.first + j) * a.q_heads + head * a.group + h) * D;
#pragma unroll
    for (int d = 0; d < DT; ++d) finish_row(a, out + 16 * d + 4 * kq, o[d] * (row.unit / kLift), sum);
    return;
  }
  // A part's sums as the lanes have them, 1 KB a store.
  const size_t slot = part_slot(a, s, head, tile) + work.part;
  kf4_t* const to = reinterpret_cast<kf4_t*>(a.part) + slot * DT * THREADS + threadIdx.x;
#pragma unroll
  for (int d = 0; d < DT; ++d) to[d * THREADS] = o[d] * (row.unit / kLift);
  if (kq == 0) part_totals<D, ROWS>(a)[slot * ROWS + wave * 16 + col] = kw2_t{__float_as_uint(row.top), __float_as_uint(sum)};
}

template <int D>
hipError_t mid(const AttnArgs& a, long long grid, hipStream_t s) {
  return kv_launch(attn_mid_kernel<D>, dim3((unsigned)grid), 64 * kMidWaves, s, a);
}

}  // namespace

hipError_t launch_attn_mid(const AttnArgs& a, int dim, hipStream_t s) {
  const long long grid = (long long)a.b.count * a.c.heads * a.parts * a.tiles;
  if (!kv_grid_fits(grid, 64 * kMidWaves)) return hipErrorInvalidConfiguration;
  if (dim == 64) return mid<64>(a, grid, s);
  return dim == 128 ? mid<128>(a, grid, s) : mid<256>(a, grid, s);
}

}  // namespace tern
