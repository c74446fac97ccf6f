// Attention of few rows over the 8-bit cache (tern_kv_attention in tern.h):
//   y = sum_t exp(z_t) v_t / sum_t exp(z_t),  z_t = scale q . k_t.
//
// A unit is a sequence's cache head: its rows, R = rows * group of them (the
// query heads that share the cache head), are the 16 columns of a matrix
// operand (NT of them), its pages a run.  All units' pages form one line, cut
// into equal pieces by the lengths that the device finds, a piece for every
// wavefront: a ragged batch fills the card evenly, and nothing waits for
// another wavefront.  A wavefront walks its pages one by one: 16-byte loads of
// codes in operand order (kv.h), K^T products in FP32 from exact FP16 codes, the
// page's softmax in registers, the weights rounded to FP16 (the only rounding;
// 2^-11 of a weight, as the output's own) against the value codes.  The keys'
// scale multiplies the scores, the values' scale the weights, in FP32.  The
// next page's keys are requested when this page's have been multiplied, the
// values likewise, page numbers two pages ahead, and the next unit's queries
// when this unit's last scores are done.  A unit that lies in one piece goes
// to y; others leave their sums in the workspace, at most two a wavefront,
// which attn_join_kernel adds in the pieces' order.  Where pages are few, a
// workgroup of several wavefronts has a unit instead, and adds their sums itself.
//
// Bound by the cache's bytes, of which it is asked 16 a lane at a time: 64
// sequences of up to 8192 tokens, 8 heads of 128, 99 us, 5.9 TB/s (a plain read
// of as much 6.4-7.0); four sequences of up to 120000 tokens, five rows each,
// 106-118 us, 5.6-6.2 TB/s.  More wavefronts, deeper prefetch and other page orders gained
// nothing; loads that pass the L2 by (kv_stream) took 123 us to 113.  One token of 8 heads
// after 4000: 6.5 us and 4.0-5.0 for joining, a chain of trips to memory.
#include "kv_attn.h"

namespace tern {
namespace {

// A page of the line: sequence, head and page, the page's number in the cache;
// left: pages behind it that are this wavefront's.
struct Step {
  int s, head, p, id, left;
};

// A sequence's pages, for the cursor along the line.
struct Run {
  Span sp;
  Range r;
};
__device__ inline Run run_of(const AttnArgs& a, int s) {
  Run x;
  x.sp = span_of(a.b, s);
  x.r = range_of(a, x.sp, max(x.sp.from, 0), x.sp.from + x.sp.n - 1);
  if (x.sp.n <= 0) x.r = {0, 0};
  return x;
}
__device__ inline int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Where this wavefront's pieces of a unit that does not lie in one piece go: two
// slots a wavefront, the first for a unit that others have begun.
struct Slot {
  float* sums;  // [R][D]
  kw2_t* tops;  // [R]
};
template <int D>
__device__ inline Slot slot_of(const AttnArgs& a, long long wave, int which) {
  const size_t rows = (size_t)a.b.max_rows * a.group, at = (size_t)(wave * 2 + which) * rows;
  return {a.part + at * D, reinterpret_cast<kw2_t*>(a.part + (size_t)a.pieces * 2 * rows * D) + at};
}

// W > 1: a workgroup of W wavefronts has a whole unit, whose pages they share
// and whose sums they add through LDS.
template <int D, int NT, int W>
__global__ __launch_bounds__(64 * W, NT * D <= 128 ? 2 : 1) void attn_rows_kernel(const AttnArgs a) {
  constexpr int C = D / 64, DT = D / 16;
  const int lane = threadIdx.x & 63, col = lane & 15, kq = lane >> 4;
  const int wave = blockIdx.x, share = W > 1 ? uniform(threadIdx.x >> 6) : 0;
  __shared__ kf4_t unit_sums[W > 1 ? W * 16 * D / 4 : 1];
  __shared__ kw2_t unit_tops[W > 1 ? W * 16 : 1];

  // The line's length, then where this wavefront's piece begins.
  Step now = {0, 0, 0, -1, -1};
  Run run = {};
  uint32_t per = 1;
  if (a.whole) {  // a unit each, whatever its length
    now.s = wave / a.c.heads;
    now.head = wave % a.c.heads;
    run = run_of(a, now.s);
    const int n = run.r.end - run.r.begin, each = (n + W - 1) / W;
    now.p = run.r.begin + share * each;
    now.left = min(each, n - share * each) - 1;
  } else {
    auto pages = [&](int x) {
      if (x >= a.b.count) return 0;
      const Run r = run_of(a, x);
      return r.r.end - r.r.begin;
    };
    const int n0 = pages(lane);
    uint32_t total = 0;
    for (int s0 = 0; s0 < a.b.count; s0 += 64) {
      int n = s0 ? pages(s0 + lane) : n0;
      for (int i = 1; i < 64; i <<= 1) n += __shfl_xor(n, i);
      total += uniform(n);
    }
    total *= a.c.heads;
    per = max((uint32_t)a.per, (total + a.pieces - 1) / a.pieces);
    const uint32_t from = wave * per;
    if (from < total) {
      uint32_t before = 0;  // pages of the sequences before s0
      for (int s0 = 0;; s0 += 64) {
        const int n = s0 ? pages(s0 + lane) : n0;
        int upto = n;
        for (int i = 1; i < 64; i <<= 1) {
          const int other = __shfl_up(upto, i);
          if (lane >= i) upto += other;
        }
        const unsigned long long mine = __ballot(from < (before + upto) * a.c.heads);
        if (mine || s0 + 64 >= a.b.count) {
          const int at = mine ? __ffsll(mine) - 1 : 0;
          now.s = s0 + at;
          before += uniform(__shfl(upto - n, at));
          break;
        }
        before += uniform(__shfl(upto, 63));
      }
      run = run_of(a, now.s);
      const int n = max(run.r.end - run.r.begin, 1), off = (int)(from - before * a.c.heads);
      now.head = off / n;
      now.p = run.r.begin + off % n;
      now.left = (int)(min(per, total - from) - 1);
    }
  }
  // units without pages: their rows are zero
  for (int u = wave; share == 0 && u < a.b.count * a.c.heads; u += a.pieces) {
    const Run x = run_of(a, u / a.c.heads);
    if (x.r.end > x.r.begin) continue;
    for (int i = lane; i < x.sp.n * a.group * (D / 4); i += 64) {
      const int r = i / (D / 4);
      const size_t out = (size_t)(x.sp.first + r / a.group) * a.q_heads + u % a.c.heads * a.group + r % a.group;
      finish_row(a, out * D + i % (D / 4) * 4, kf4_t{0.f, 0.f, 0.f, 0.f}, 0.f);
    }
    if (lane == 0 && !a.whole) a.info[u] = make_int2(0, 1);
  }
  if (W == 1 && now.left < 0) return;

  // The step behind one; the run it lies in.
  auto number = [&](const Step& x) { return uniform(page_of(a.b, a.c, x.s, x.p)); };
  auto behind = [&](Step x, Run& in) {
    if (x.left <= 0) return Step{-1, 0, 0, -1, -1};
    --x.left;
    if (++x.p >= in.r.end) {
      if (++x.head >= a.c.heads) {  // the line goes on: a sequence with pages follows
        x.head = 0;
        do {
          if (++x.s >= a.b.count) return Step{-1, 0, 0, -1, -1};
          in = run_of(a, x.s);
        } while (in.r.end <= in.r.begin);
      }
      x.p = in.r.begin;
    }
    x.id = number(x);
    return x;
  };

  // Two blocks' queries of 256 dimensions lie in LDS: there are no registers for them.
  constexpr bool kInLds = NT * C > 4;
  __shared__ kw4_t lq[kInLds ? NT * C * 2 * 64 : 1];
  kh8_t q[kInLds ? 1 : NT][C][2];
  auto query = [&](int n, int c, int u) {
    return kInLds ? __builtin_bit_cast(kh8_t, lq[((n * C + c) * 2 + u) * 64 + lane]) : q[kInLds ? 0 : n][c][u];
  };
  Sees sees[NT];
  int low, high;  // tokens that every row sees
  Row row[NT];
  kf4_t o[NT][DT];
  // of a unit's row: its place in q (bytes) and y (heads), from the first's
  int place_q[NT], place_y[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = n * 16 + col;
    place_q[n] = (r / a.group * (int)a.q_stride + r % a.group * D + 16 * kq) * 2;
    place_y[n] = r / a.group * a.q_heads + r % a.group;
  }
  auto load_q = [&](const Step& x, const Span& sp) {
    const __amdgpu_buffer_rsrc_t from = kv_buffer(a.q + sp.first * a.q_stride + x.head * a.group * D, 0x7fffffff);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int at = n * 16 + col < sp.n * a.group ? place_q[n] : kFarAway;
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const kw4_t v = kv_load16(from, at + 128 * c + 16 * u);
          if (kInLds)
            lq[((n * C + c) * 2 + u) * 64 + lane] = v;
          else
            q[kInLds ? 0 : n][c][u] = __builtin_bit_cast(kh8_t, v);
        }
    }
  };
  auto begin_rows = [&](const Span& sp) {
    low = 0;
    high = 0x7fffffff;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = n * 16 + col;
      const bool there = r < sp.n * a.group;
      sees[n] = sees_of(a, sp, sp.from + r / a.group, there);
      if (there) {
        low = max(low, sees[n].low);
        high = min(high, sees[n].high);
      }
      row[n] = new_row();
#pragma unroll
      for (int d = 0; d < DT; ++d) o[n][d] = kf4_t{0.f, 0.f, 0.f, 0.f};
    }
    for (int i = 1; i < 16; i <<= 1) {
      low = max(low, __shfl_xor(low, i));
      high = min(high, __shfl_xor(high, i));
    }
    low = uniform(low);
    high = uniform(high);
  };

  // a page that is not there reads as zeros, and is masked
  kw4_t kr[C][4], vr[DT];
  auto page_at = [&](const uint8_t* pages, const Step& x) {
    return kv_buffer(pages + ((size_t)max(x.id, 0) * a.c.heads + x.head) * (kPage * D), x.id < 0 ? 0 : kPage * D);
  };
  auto load_keys = [&](const Step& x) {
    const __amdgpu_buffer_rsrc_t from = page_at(a.c.k, x);
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int t = 0; t < 4; ++t) kr[c][t] = kv_load16<kv_stream>(from, ((4 * c + t) * 64 + lane) * 16);
  };
  auto load_values = [&](const Step& x) {
    const __amdgpu_buffer_rsrc_t from = page_at(a.c.v, x);
#pragma unroll
    for (int d = 0; d < DT; ++d) vr[d] = kv_load16<kv_stream>(from, (d * 64 + lane) * 16);
  };
  auto scale_at = [&](const float* scales, const Step& x) { return kv_const(scales, (size_t)max(x.id, 0) * a.c.heads + x.head); };

  if (now.left < 0) now.p = -1;  // of W wavefronts: more than there are pages
  now.id = now.left < 0 ? -1 : number(now);
  Run ahead = run;  // of the step that is looked at first
  Step next = behind(now, ahead);
  Run run_next = ahead;
  load_keys(now);
  load_q(now, run.sp);
  load_values(now);
  float ks_next = scale_at(a.c.ks, now), vs_next = scale_at(a.c.vs, now);
  begin_rows(run.sp);
  bool opened = now.p == run.r.begin;  // the unit begins in this piece,
  int room = now.left + 1;             // which had so many pages left then

  for (; W == 1 || now.left >= 0;) {
    const Step later = behind(next, ahead);
    const float ks = ks_next * a.scale, vs = vs_next;
    ks_next = scale_at(a.c.ks, next);
    vs_next = scale_at(a.c.vs, next);
    const bool last = next.left < 0 || next.head != now.head || next.s != now.s;  // of the unit, here
    const bool whole = now.id >= 0 && now.p * kPage >= low && now.p * kPage + kPage <= high;
    kh8_t w[NT][2];
    kf4_t z[NT][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (NT > 1) __builtin_amdgcn_sched_barrier(0);  // decoding far ahead takes registers that are not there
#pragma unroll
      for (int n = 0; n < NT; ++n) z[n][t] = kf4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const kh8_t k = codes8(kr[c][t][2 * u], kr[c][t][2 * u + 1]);
#pragma unroll
          for (int n = 0; n < NT; ++n) z[n][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, query(n, c, u), z[n][t], 0, 0, 0);
        }
    }
    __builtin_amdgcn_sched_barrier(0);
    load_keys(next);
    if (last && next.left >= 0) load_q(next, run_next.sp);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float best = -INFINITY;
#pragma unroll
      for (int t = 0; t < 4; ++t) z[n][t] *= ks;
      if (!whole) {
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const int token = now.p * kPage + 16 * kq + x;
          if (now.id < 0 || token < sees[n].low || token >= sees[n].high) z[n][x / 4][x % 4] = -INFINITY;
        }
      }
#pragma unroll
      for (int x = 0; x < 16; ++x) best = fmaxf(best, z[n][x / 4][x % 4]);
      best = max_of_32(max_of_16(best));
      float lift, back;
      const float factor = step_row(row[n], best, vs == 0.f ? 1.f : vs, lift, back);
      const float top = top_of(row[n]);
      if (__any(factor != 1.0f)) {
#pragma unroll
        for (int d = 0; d < DT; ++d) o[n][d] *= factor;
      }
      float sum = 0.f;
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        const float e = __builtin_amdgcn_exp2f((z[n][x / 4][x % 4] - top) + lift);  // the reference's weight is exact
        sum += e;
        w[n][x / 8][x % 8] = (_Float16)e;
      }
      row[n].sum += sum * back;
      if (vs == 0.f) w[n][0] = w[n][1] = kh8_t{0, 0, 0, 0, 0, 0, 0, 0};  // values of 0, whatever the codes
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      if (NT > 1 && d % 2 == 0) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const kh8_t v = codes8(vr[d][2 * u], vr[d][2 * u + 1]);
#pragma unroll
        for (int n = 0; n < NT; ++n) o[n][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, w[n][u], o[n][d], 0, 0, 0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    load_values(next);
    if (last) {
      const bool all = opened && now.p + 1 == run.r.end;
      const Slot slot = slot_of<D>(a, wave, opened ? 1 : 0);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int r = n * 16 + col;
        float sum = row[n].sum;
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        if (r >= run.sp.n * a.group) continue;
        const float unit = row[n].unit / kLift;
        const size_t out = (size_t)run.sp.first * a.q_heads + now.head * a.group + place_y[n];
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const kf4_t v = o[n][d] * unit;
          if (W > 1)
            unit_sums[(share * 16 + r) * (D / 4) + 4 * d + kq] = v;
          else if (all)
            finish_row(a, out * D + 16 * d + 4 * kq, v, sum);
          else
            *reinterpret_cast<kf4_t*>(slot.sums + (size_t)r * D + 16 * d + 4 * kq) = v;
        }
        if (W > 1 && kq == 0) unit_tops[share * 16 + r] = kw2_t{__float_as_uint(row[n].top), __float_as_uint(sum)};
        if (W == 1 && !all && kq == 0) slot.tops[r] = kw2_t{__float_as_uint(row[n].top), __float_as_uint(sum)};
      }
      if (opened && lane == 0 && !a.whole) {
        const int more = run.r.end - run.r.begin - room;
        a.info[now.s * a.c.heads + now.head] = make_int2(wave, more > 0 ? 1 + (int)(((uint32_t)more + per - 1) / per) : 1);
      }
      if (next.left < 0) break;
      begin_rows(run_next.sp);
      opened = next.p == run_next.r.begin;
      room = next.left + 1;
    }
    now = next;
    run = run_next;
    next = later;
    run_next = ahead;
  }
  if constexpr (W > 1) {
    const Run unit = run_of(a, wave / a.c.heads);
    const int n = unit.r.end - unit.r.begin, each = (n + W - 1) / W, rows = unit.sp.n * a.group;
    if (n <= 0) return;
    const int shares = (n + each - 1) / each;
    __syncthreads();
    for (int i = threadIdx.x; i < rows * (D / 4); i += 64 * W) {
      const int r = i / (D / 4), d = i % (D / 4);
      float top = -INFINITY, sum = 0.f;
      kf4_t v = {0.f, 0.f, 0.f, 0.f};
      for (int x = 0; x < shares; ++x) top = fmaxf(top, __uint_as_float(unit_tops[x * 16 + r].x));
      for (int x = 0; x < shares; ++x) {
        const kw2_t t = unit_tops[x * 16 + r];
        const float own = __uint_as_float(t.x), f = own == top ? 1.f : __builtin_amdgcn_exp2f(own - top);
        sum += __uint_as_float(t.y) * f;
        v += unit_sums[(x * 16 + r) * (D / 4) + d] * f;
      }
      const size_t out = (size_t)(unit.sp.first + r / a.group) * a.q_heads + wave % a.c.heads * a.group + r % a.group;
      finish_row(a, out * D + 4 * d, v, sum);
    }
  }
}

// y from the sums of a unit's pieces, in their order: a workgroup has a row's
// head, its groups of lanes take turns at the pieces.
template <int D>
__global__ __launch_bounds__(256) void attn_join_kernel(const AttnArgs a) {
  constexpr int L = D / 4, G = 256 / L;  // lanes of a row, groups
  __shared__ kf4_t sums[256];
  __shared__ float2 totals[G];
  const int s = blockIdx.x / a.b.max_rows, j = blockIdx.x % a.b.max_rows, head = blockIdx.y;
  const int unit = s * a.c.heads + head / a.group;  // read with the span, not behind it
  const int2 info = make_int2(kv_const(&a.info[0].x, 2 * unit), kv_const(&a.info[0].x, 2 * unit + 1));
  const Span sp = span_of(a.b, s);
  if (j >= sp.n) return;
  const int count = info.y;
  if (count == 1) return;  // written where it was computed
  // the pieces' rows: the second slot of the first, the others' first ones
  const size_t rows = (size_t)a.b.max_rows * a.group, step = 2 * rows, all = (size_t)a.pieces * step;
  const size_t first = (size_t)info.x * step + j * a.group + head % a.group, out = (size_t)(sp.first + j) * a.q_heads + head;
  auto at = [&](int i) { return first + i * step + (i == 0 ? rows : 0); };
  const int g = threadIdx.x / L, d = threadIdx.x % L * 4;
  const kw2_t* const tops = reinterpret_cast<const kw2_t*>(a.part + all * D);
  // one pass: every group keeps its own reference
  kf4_t v = {0.f, 0.f, 0.f, 0.f};
  float sum = 0.f, top = -INFINITY;
#pragma unroll 4
  for (int i = g; i < count; i += G) {
    const kw2_t t = tops[at(i)];
    const kf4_t x = *reinterpret_cast<const kf4_t*>(a.part + at(i) * D + d);
    const float own = __uint_as_float(t.x), most = fmaxf(top, own);
    const float keep = top == most ? 1.f : __builtin_amdgcn_exp2f(top - most);
    const float f = own == most ? 1.f : __builtin_amdgcn_exp2f(own - most);
    sum = sum * keep + __uint_as_float(t.y) * f;
    v = v * keep + x * f;
    top = most;
  }
  sums[threadIdx.x] = v;
  if (threadIdx.x % L == 0) totals[g] = make_float2(top, sum);
  __syncthreads();
  if (threadIdx.x >= L) return;
  for (int i = 1; i < G; ++i) top = fmaxf(top, totals[i].x);
  v = kf4_t{0.f, 0.f, 0.f, 0.f};
  sum = 0.f;
  for (int i = 0; i < G; ++i) {
    const float f = totals[i].x == top ? 1.f : __builtin_amdgcn_exp2f(totals[i].x - top);
    v += sums[i * L + threadIdx.x] * f;
    sum += totals[i].y * f;
  }
  finish_row(a, out * D + d, v, sum);
}

template <int D>
hipError_t rows(const AttnArgs& a, int blocks, int shares, hipStream_t s) {
  const dim3 grid((unsigned)a.pieces);
  if (!kv_grid_fits(a.pieces, 64 * shares)) return hipErrorInvalidConfiguration;
  if (blocks == 2) return kv_launch(attn_rows_kernel<D, 2, 1>, grid, 64, s, a);
  if (shares == 2) return kv_launch(attn_rows_kernel<D, 1, 2>, grid, 128, s, a);
  if (shares == 4) return kv_launch(attn_rows_kernel<D, 1, 4>, grid, 256, s, a);
  if constexpr (D < 256)
    if (shares == 8) return kv_launch(attn_rows_kernel<D, 1, 8>, grid, 512, s, a);
  return kv_launch(attn_rows_kernel<D, 1, 1>, grid, 64, s, a);
}

template <int D>
hipError_t join(const AttnArgs& a, hipStream_t s) {
  const long long x = (long long)a.b.count * a.b.max_rows;
  if (a.q_heads > 65535 || !kv_grid_fits(x * a.q_heads, 256)) return hipErrorInvalidConfiguration;
  return kv_launch(attn_join_kernel<D>, dim3((unsigned)x, (unsigned)a.q_heads), 256, s, a);
}

}  // namespace

hipError_t launch_attn_rows(const AttnArgs& a, int dim, int blocks, int shares, hipStream_t s) {
  if (dim == 64) return rows<64>(a, blocks, shares, s);
  return dim == 128 ? rows<128>(a, blocks, shares, s) : rows<256>(a, blocks, shares, s);
}

hipError_t launch_attn_join_rows(const AttnArgs& a, int dim, hipStream_t s) {
  if (dim == 64) return join<64>(a, s);
  return dim == 128 ? join<128>(a, s) : join<256>(a, s);
}

}  // namespace tern
