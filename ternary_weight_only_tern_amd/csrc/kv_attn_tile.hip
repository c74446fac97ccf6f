// Attention of many rows over the 8-bit cache: the same formula as in
// kv_attn_rows.hip, on tiles.
//
// A workgroup of four wavefronts owns 128 rows (tokens times the query heads
// that share a cache head), 32 a wavefront, and walks the pages that any of
// them sees.  A page's codes are decoded once for the workgroup, into LDS as
// FP16 operands of v_mfma_f32_32x32x16_f16 in the order in which lanes read
// them (no bank conflicts), one page ahead, the page after that on its way
// into registers meanwhile.  Up to 128 dimensions a step multiplies the next page's
// keys while it looks for this page's largest scores.  Scores come out
// transposed (a lane has one row's scores of 32 tokens of the page, its partner
// 32 lanes on the others), so the softmax needs one exchange, and the weights are
// the next product's operand where they are.  Heavy tiles (the last of a causal
// prompt) start first; the workgroups of a cache head are neighbours modulo the
// number of heads, so that an XCD's L2 keeps few heads' pages.  Where tiles are
// few, their contexts are cut into parts (parts_for in kv_api.cpp), whose sums
// attn_join_tile_kernel adds.
//
// Bound by instructions: a wavefront's page of 128 dimensions is 32 matrix
// instructions (1024 cycles) and about 1400 cycles of exponentials, maxima,
// roundings and decoding, which overlap little: 2048 rows of 32 heads over 8
// after 1000 tokens 90 us, 755 TFLOP/s; 8192 rows 595 us, 924 TFLOP/s (the
// library's FP16 product of 8192^3: 1200-1340).  Other orders of the tiles, other
// priorities and three wavefronts a SIMD (at 64 dimensions) gained nothing or spilled.  Where tiles
// are short, 3 to 5 us pass before a workgroup's first page: four dependent trips
// to memory and code that no cache holds yet.  At 256 dimensions a CU has one
// workgroup, and its operands from LDS take as long as its matrix instructions (4
// prompts of 2048 rows, 8 heads, 120 us, 571 TFLOP/s).
#include "kv_attn.h"

namespace tern {
namespace {

constexpr int kTileWaves = 4;

template <int D>
__global__ __launch_bounds__(64 * kTileWaves, D <= 128 ? 2 : 1) void attn_tile_kernel(const AttnArgs a) {
  constexpr int THREADS = 64 * kTileWaves, ROWS = 32 * kTileWaves;
  constexpr int KS = D / 16;                        // products of 16 dimensions in a score
  constexpr int DB = D / 32;                        // blocks of 32 dimensions of the sums
  constexpr int PIECES = kPage * D / 16 / THREADS;  // of 16 codes a thread, keys and values each
  // Whether a step computes the next page's scores (two pages' scores are in
  // registers then, which there are not enough of at 256 dimensions).
  constexpr bool LEAD = D <= 128;
  __shared__ kw4_t lk[2][kPage * D / 8], lv[2][kPage * D / 8];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c32 = lane & 31, hq = lane >> 5;
  const Work work = work_of(a, D <= 128);
  const int s = work.s, head = work.head, part = work.part, tile = work.tile;
  const Span sp = span_of(a.b, s);
  const int total = sp.n * a.group;
  if (tile * ROWS >= total) return;
  const Range all = range_of_rows(a, sp, tile * ROWS, min(tile * ROWS + ROWS, total) - 1);
  const Parts parts = parts_of(a, all);
  if (part >= parts.count) return;
  const Range mine = part_of(all, parts, part);

  // Two workgroups on a CU have their first rows on different SIMDs: where a
  // tile has 64 rows or fewer, each SIMD has one wavefront with rows.
  const int block = (wave + blockIdx.x / kCus % 2 * 2) % kTileWaves;
  const int r = tile * ROWS + block * 32 + c32, j = r / a.group, h = r % a.group;
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
  // Page numbers and scales come by vector loads, a step and more ahead: they
  // are there with the pages that the decoding waits for, and no scalar load
  // in flight makes an LDS read wait.
  const int32_t* const table = a.b.pages + (size_t)s * a.b.max_pages;
  auto load_id = [&](int p) {
    return (int)__builtin_amdgcn_raw_buffer_load_b32(kv_buffer(table + (p < mine.end ? p : 0), p < mine.end ? 4 : 0), 0, 0, 0);
  };
  auto id_of = [&](int raw, int p) {
    const int id = __builtin_amdgcn_readfirstlane(raw);
    return p < mine.end && id >= 0 && id < a.c.pages ? id : -1;
  };
  auto load_scale = [&](const float* scales, int id) {
    return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(kv_buffer(scales + (size_t)max(id, 0) * a.c.heads + head, 4), 0, 0, 0));
  };
  auto buffer = [&](const uint8_t* pages, int id) {
    return kv_buffer(pages + ((size_t)max(id, 0) * a.c.heads + head) * (kPage * D), id < 0 ? 0 : kPage * D);
  };
  auto load_keys = [&](int id) {
    const __amdgpu_buffer_rsrc_t f = buffer(a.c.k, id);
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int st = i * kTileWaves + wave;
      kr[i] = kv_load16(f, ((st / 4 * 4 + lane / 4 % 4) * 64 + st % 4 * 16 + lane / 16 * 4 + lane % 4) * 16);
    }
  };
  auto load_values = [&](int id) {
    const __amdgpu_buffer_rsrc_t f = buffer(a.c.v, id);
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int st = i * kTileWaves + wave, part = st % 4, d = st / 4 * 64 + lane;
      vr[i] = kv_load16(f, ((d / 16 * 4 + part) * 16 + d % 16) * 16);
    }
  };
  // An eighth or so of a page's decoding: half a piece of the keys (units below
  // 2 PIECES) or of the values.
  auto decode = [&](int unit, kw4_t* keys, kw4_t* values) {
    const int i = unit / 2 % PIECES, half = unit % 2, st = i * kTileWaves + wave;
    if (unit < 2 * PIECES) {
      keys[(st * 2 + lane / 32) * 64 + lane % 32 + 32 * half] = __builtin_bit_cast(kw4_t, codes8(kr[i][2 * half], kr[i][2 * half + 1]));
    } else {
      const int part = st % 4, d = st / 4 * 64 + lane;
      values[(d / 32 * 4 + part) * 64 + d % 32 + 32 * half] = __builtin_bit_cast(kw4_t, codes8(vr[i][half], vr[i][2 + half]));
    }
  };
  // Operand i of a step from LDS: the next page's keys, then this page's
  // values, in an order in which neighbours add to different sums.
  constexpr int MK = 2 * KS, AHEAD = D == 64 ? 8 : 4;  // instructions of a product, operands on their way
  auto operand = [&](int i, const kw4_t* ks, const kw4_t* vs) {
    if (i < MK) return __builtin_bit_cast(kh8_t, ks[i * 64 + lane]);
    const int t = (i - MK) / DB, db = (i - MK) % DB;
    return __builtin_bit_cast(kh8_t, vs[(db * 4 + t) * 64 + lane]);
  };
  kf16_t z[2];
  auto multiply = [&](const kw4_t* ks) {  // the scores of a page alone
#pragma unroll
    for (int v = 0; v < 16; ++v) z[0][v] = z[1][v] = 0.f;
#pragma unroll
    for (int i = 0; i < MK; ++i)
      z[i % 2] = __builtin_amdgcn_mfma_f32_32x32x16_f16(operand(i, ks, nullptr), q[i / 2], z[i % 2], 0, 0, 0);
  };
  // whether any of the wavefront's rows sees page p
  auto seen = [&](int p) { return p * kPage < most && p * kPage + kPage > least; };

  // A step multiplies the next page's (LEAD) or this page's keys with the
  // queries while the vector units find this page's largest score and decode
  // the keys after those and the next values; then it sums this page's values
  // while the vector units turn scores into weights, 16 tokens ahead.
  int p = mine.begin, cur = 0;
  int raw = load_id(p), raw1 = load_id(p + 1), raw2 = load_id(p + 2), raw3 = load_id(p + 3);
  int id = id_of(raw, p), id1 = id_of(raw1, p + 1), id2 = id_of(raw2, p + 2);
  load_keys(id1);  // the first pages together, the second's keys kept aside
  kw4_t second[PIECES];
#pragma unroll
  for (int i = 0; i < PIECES; ++i) second[i] = kr[i];
  load_keys(id);
  load_values(id);
  float ks0 = load_scale(a.c.ks, id), vs0 = load_scale(a.c.vs, id);  // this page's, the next one's
  float ks1 = load_scale(a.c.ks, id1), vs1 = load_scale(a.c.vs, id1);
  __builtin_amdgcn_s_waitcnt(0x0F70);  // with the queries, once: in the loop their wait would be for the pages too
  if (mine.begin < mine.end) {
#pragma unroll
    for (int u = 0; u < 4 * PIECES; ++u) decode(u, lk[0], lv[0]);
#pragma unroll
    for (int i = 0; i < PIECES; ++i) kr[i] = second[i];
    if constexpr (LEAD) {
#pragma unroll
      for (int u = 0; u < 2 * PIECES; ++u) decode(u, lk[1], nullptr);
      load_keys(id2);
    }
    load_values(id1);
    __syncthreads();
    if constexpr (LEAD) {
      multiply(lk[0]);
      __syncthreads();
    }
  }
  int id3 = -1;
  float ks2 = 0.f, vs2 = 0.f;
  auto fetch = [&]() {  // what the next step decodes
    id3 = id_of(raw3, p + 3);
    load_keys(LEAD ? id3 : id2);
    load_values(id2);
    ks2 = load_scale(a.c.ks, id2);
    vs2 = load_scale(a.c.vs, id2);
    raw3 = load_id(p + 4);
  };
  for (; p < mine.end; ++p, cur ^= 1) {
    const kw4_t *const ks = lk[LEAD ? cur ^ 1 : cur], *const vs = lv[cur];
    kw4_t* const keys = lk[LEAD ? cur : cur ^ 1];
    if (seen(p)) {
      const float vscale = __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__float_as_int(vs0)));
      float by = ks0 * a.scale, best = -INFINITY;  // the scores are by z
      // Minus infinity where a row does not see the token: one comparison a
      // score, on the side where the page crosses a border.
      auto mask = [&]() {
        const int first = p * kPage, side = first + 4 * hq;
        const bool none = id < 0, below = none || first < low, above = first + kPage > high;
        if (!below && !above) return;
        if (!(by > 0.f)) {  // of no use beside infinities
#pragma unroll
          for (int x = 0; x < 32; ++x) z[x / 16][x % 16] *= by;
          by = 1.0f;
        }
        if (below) {
          const int from = none ? kPage : sees.low - side;
#pragma unroll
          for (int x = 0; x < 32; ++x)
            if (x / 4 * 8 + x % 4 < from) z[x / 16][x % 16] = -INFINITY;
        }
        if (above) {
          const int to = sees.high - side;
#pragma unroll
          for (int x = 0; x < 32; ++x)
            if (x / 4 * 8 + x % 4 >= to) z[x / 16][x % 16] = -INFINITY;
        }
      };
      if (LEAD) mask();
      kh8_t f[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) f[i] = operand(i, ks, vs);
      // Behind the last page the next scores are of what lies there, and not used.
      const kf16_t zero = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      kf16_t next[2];
      auto largest = [&](int x, int n) {
#pragma unroll
        for (int y = x; y < x + n; ++y) best = fmaxf(best, z[y / 16][y % 16]);
      };
#pragma unroll
      for (int i = 0; i < MK; ++i) {
        __builtin_amdgcn_sched_barrier(0);
        next[i % 2] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f[i % AHEAD], q[i / 2], i < 2 ? zero : next[i % 2], 0, 0, 0);
        f[i % AHEAD] = operand(i + AHEAD, ks, vs);
        if (i < MK / 2) {
          if (LEAD) largest(i * (64 / MK), 64 / MK);
        } else {
          decode(i - MK / 2, keys, lv[cur ^ 1]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      fetch();
      if (!LEAD) {
        z[0] = next[0];
        z[1] = next[1];
        mask();
        largest(0, 32);
      }
      best = max_of_32(best) * by;
      float lift, back;
      const float factor = step_row(row, best, vscale == 0.f ? 1.f : vscale, lift, back);
      float shift = lift - top_of(row);
      if (__any(factor != 1.0f)) {
#pragma unroll
        for (int d = 0; d < DB; ++d) o[d] *= factor;
      }
      // This page's weights, 16 tokens ahead of the sums of its values.
      kh8_t w[4];
      float sum = 0.f;
      auto weigh = [&](int x) { z[x / 16][x % 16] = __builtin_amdgcn_exp2f(__builtin_fmaf(z[x / 16][x % 16], by, shift)); };
      // The sum is of the rounded weights, two by one instruction: what a weight
      // loses against the values it loses in the sum too.
      auto round2 = [&](int x) {
        const kh2_t two = {(_Float16)z[x / 16][x % 16], (_Float16)z[x / 16][x % 16 + 1]};
        w[x / 8][x % 8] = two.x;
        w[x / 8][x % 8 + 1] = two.y;
        sum = __builtin_amdgcn_fdot2(two, kh2_t{(_Float16)1.0f, (_Float16)1.0f}, sum, false);
      };
      if (vscale == 0.f) {  // values of 0, whatever the codes: the weights' sum alone
        float alone = 0.f;
#pragma unroll
        for (int x = 0; x < 32; ++x) alone += __builtin_amdgcn_exp2f(__builtin_fmaf(z[x / 16][x % 16], by, shift));
        row.sum += alone * back;
        shift = -INFINITY;
      }
#pragma unroll
      for (int x = 0; x < 8; ++x) weigh(x);
#pragma unroll
      for (int x = 0; x < 8; x += 2) round2(x);
#pragma unroll
      for (int i = 0; i < MK; ++i) {
        const int t = i / DB, db = i % DB;
        constexpr int E = 8 / DB;
        __builtin_amdgcn_sched_barrier(0);
        if (t > 0 && db == 0)
#pragma unroll
          for (int x = t * 8 + 8 - (E > 2 ? E : 2); x < t * 8 + 8; x += 2) round2(x);
        o[db] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f[(MK + i) % AHEAD], w[t], o[db], 0, 0, 0);
        if (i + AHEAD < MK) f[(MK + i) % AHEAD] = operand(MK + i + AHEAD, ks, vs);
        if (t < 3) {
#pragma unroll
          for (int x = (t + 1) * 8 + db * E; x < (t + 1) * 8 + db * E + E; ++x) weigh(x);
          // of the instruction before
#pragma unroll
          for (int x = (t + 1) * 8 + (db - 1) * E; db > 0 && x < (t + 1) * 8 + db * E; ++x)
            if (x % 2) round2(x - 1);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      row.sum += sum * back;
      if (LEAD) {
        z[0] = next[0];
        z[1] = next[1];
      }
    } else {
      if (LEAD && seen(p + 1)) multiply(ks);
#pragma unroll
      for (int u = 0; u < 4 * PIECES; ++u) decode(u, keys, lv[cur ^ 1]);
      fetch();
    }
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
  sum += __shfl_xor(sum, 32);
  if (!there) return;
  if (parts.count == 1) {
    const size_t out = ((size_t)(sp.first + j) * a.q_heads + head * a.group + h) * D;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      const kf4_t x = {o[i / 4][i % 4 * 4], o[i / 4][i % 4 * 4 + 1], o[i / 4][i % 4 * 4 + 2], o[i / 4][i % 4 * 4 + 3]};
      finish_row(a, out + 8 * i + 4 * hq, x * (row.unit / kLift), sum);
    }
    return;
  }
  // A part's sums as the lanes have them, 1 KB a store.
  const size_t slot = part_slot(a, s, head, tile) + part;
  kf4_t* const to = reinterpret_cast<kf4_t*>(a.part) + slot * (D / 8) * THREADS + block * 64 + lane;
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    const kf4_t x = {o[i / 4][i % 4 * 4], o[i / 4][i % 4 * 4 + 1], o[i / 4][i % 4 * 4 + 2], o[i / 4][i % 4 * 4 + 3]};
    to[i * THREADS] = x * (row.unit / kLift);
  }
  if (hq == 0) part_totals<D, ROWS>(a)[slot * ROWS + block * 32 + c32] = kw2_t{__float_as_uint(row.top), __float_as_uint(sum)};
}

// y from the sums of a tile's parts, in an order of their own: a workgroup has one
// of the fours of dimensions that a thread holds, the threads of each of its
// SIDES what the tile's own threads left (32 rows a wavefront and 4 of 8 dimensions
// a lane, or 16 rows and 4 of 16), of every SIDES-th part.  Four sides where parts
// are more than 32 (us with the tiles: 130 parts of six 32.6 -> 25.0, 63 of eight 26.6 ->
// 24.1, 16 of 32 20.8 -> 21.4).
template <int D, int ROWS, int SIDES>
__global__ __launch_bounds__(64 * kTileWaves * SIDES) void attn_join_tile_kernel(const AttnArgs a) {
  constexpr int THREADS = 64 * kTileWaves, R = ROWS / kTileWaves, L = 64 / R * 4;  // rows a wavefront, dimensions of a store
  __shared__ kf4_t side_sums[SIDES > 1 ? SIDES - 1 : 1][SIDES > 1 ? THREADS : 1];
  __shared__ float2 side_totals[SIDES > 1 ? SIDES - 1 : 1][SIDES > 1 ? THREADS : 1];
  const int head = blockIdx.x % a.c.heads, s = blockIdx.x / a.c.heads % a.b.count, tile = blockIdx.x / a.c.heads / a.b.count;
  const Span sp = span_of(a.b, s);
  const int total = sp.n * a.group;
  if (tile * ROWS >= total) return;
  const int count = parts_of(a, range_of_rows(a, sp, tile * ROWS, min(tile * ROWS + ROWS, total) - 1)).count;
  if (count == 1) return;
  const int side = threadIdx.x / THREADS, thread = threadIdx.x % THREADS;
  const int lane = thread & 63, in = thread / 64 * R + lane % R, r = tile * ROWS + in;
  const size_t slot = part_slot(a, s, head, tile);
  const kf4_t* const sums = reinterpret_cast<const kf4_t*>(a.part) + (slot * (D / L) + blockIdx.y) * THREADS + thread;
  const kw2_t* const totals = part_totals<D, ROWS>(a) + slot * ROWS + in;
  kf4_t v = {0.f, 0.f, 0.f, 0.f};
  float sum = 0.f, top = -INFINITY;
  auto add = [&](float own, float own_sum, kf4_t x) {
    const float most = fmaxf(top, own);
    const float keep = top == most ? 1.f : __builtin_amdgcn_exp2f(top - most);
    const float f = own == most ? 1.f : __builtin_amdgcn_exp2f(own - most);
    sum = sum * keep + own_sum * f;
    v = v * keep + x * f;
    top = most;
  };
  if (r < total) {  // what lies behind the rows was not written
#pragma unroll 4
    for (int i = side; i < count; i += SIDES) {
      const kw2_t t = totals[(size_t)i * ROWS];
      add(__uint_as_float(t.x), __uint_as_float(t.y), sums[(size_t)i * (D / L) * THREADS]);
    }
  }
  if (SIDES > 1) {
    if (side > 0) {
      side_sums[side - 1][thread] = v;
      side_totals[side - 1][thread] = make_float2(top, sum);
    }
    __syncthreads();
    if (side > 0) return;
    for (int i = 0; i < SIDES - 1; ++i) add(side_totals[i][thread].x, side_totals[i][thread].y, side_sums[i][thread]);
  }
  if (r >= total) return;
  const size_t out = ((size_t)(sp.first + r / a.group) * a.q_heads + head * a.group + r % a.group) * D;
  finish_row(a, out + L * blockIdx.y + lane / R * 4, v, sum);
}

template <int D>
hipError_t tile(const AttnArgs& a, long long grid, hipStream_t s) {
  return kv_launch(attn_tile_kernel<D>, dim3((unsigned)grid), 64 * kTileWaves, s, a);
}

template <int D, int ROWS>
hipError_t join(const AttnArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)(a.b.count * a.c.heads * a.tiles), D * ROWS / (64 * kTileWaves * 4));
  if (a.parts > 32) return kv_launch(attn_join_tile_kernel<D, ROWS, 4>, grid, 64 * kTileWaves * 4, s, a);
  return kv_launch(attn_join_tile_kernel<D, ROWS, 1>, grid, 64 * kTileWaves, s, a);
}
template <int D>
hipError_t join(const AttnArgs& a, int rows, hipStream_t s) {
  return rows == kAttnTile ? join<D, kAttnTile>(a, s) : join<D, kAttnMid>(a, s);
}

}  // namespace

hipError_t launch_attn_tile(const AttnArgs& a, int dim, hipStream_t s) {
  const long long grid = (long long)a.b.count * a.c.heads * a.parts * a.tiles;
  if (!kv_grid_fits(grid, 64 * kTileWaves)) return hipErrorInvalidConfiguration;
  if (dim == 64) return tile<64>(a, grid, s);
  return dim == 128 ? tile<128>(a, grid, s) : tile<256>(a, grid, s);
}

hipError_t launch_attn_join_tile(const AttnArgs& a, int dim, int rows, hipStream_t s) {
  if (dim == 64) return join<64>(a, rows, s);
  return dim == 128 ? join<128>(a, rows, s) : join<256>(a, rows, s);
}

}  // namespace tern
