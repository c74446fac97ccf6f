// Device code shared by the attention kernels: what a workgroup looks at, and
// the running softmax of a row (q. v. kv_attn_rows.hip).
#pragma once

#include "kv.h"

namespace tern {

#ifdef __HIPCC__
// Pages [begin, end) that the rows at positions first..last see.
struct Range {
  int begin, end;
};
__device__ inline Range range_of(const AttnArgs& a, const Span& sp, int first, int last) {
  const int end = min(a.causal ? last + 1 : sp.len, sp.len);
  const int begin = a.window > 0 ? max(first - a.window + 1, 0) : 0;
  Range r = {begin / kPage, min((end + kPage - 1) / kPage, a.b.max_pages)};
  if ((a.causal && last < 0) || r.end < r.begin) r.end = r.begin;
  return r;
}

// Pages of a part: what the host chose, or more where the context is longer
// than it was told; and the parts that there are.
struct Parts {
  int per, count;
};
__device__ inline Parts parts_of(const AttnArgs& a, const Range& r) {
  const int n = r.end - r.begin;
  Parts p;
  p.per = max(a.per, (n + a.parts - 1) / a.parts);
  p.count = max(1, (n + p.per - 1) / p.per);
  return p;
}
__device__ inline Range part_of(const Range& r, const Parts& p, int part) {
  const int begin = r.begin + part * p.per;
  return {begin, min(begin + p.per, r.end)};
}

// A workgroup's tile, in the order in which they start: heavy tiles (the last
// of a causal prompt) first, the cache heads neighbours.  `pairs`: where the card
// holds the whole grid at once, two workgroups a CU, its second is the lighter
// the heavier its first.
constexpr int kCus = 256;
struct Work {
  int s, head, part, tile;
};
__device__ inline Work work_of(const AttnArgs& a, bool pairs) {
  Work w;
  int bid = blockIdx.x;
  w.head = bid % a.c.heads;
  bid /= a.c.heads;
  w.s = bid % a.b.count;
  bid /= a.b.count;
  w.part = bid % a.parts;
  w.tile = a.tiles - 1 - bid / a.parts;
  const int per = a.c.heads * a.b.count * a.parts, firsts = (kCus + per - 1) / per;
  if (pairs && a.tiles * per <= 2 * kCus && bid / a.parts >= firsts) w.tile = bid / a.parts - firsts;
  return w;
}

// A tile's first part among all parts' sums, and the references and sums of
// weights behind those, for tiles of R rows.
__device__ inline size_t part_slot(const AttnArgs& a, int s, int head, int tile) {
  return (((size_t)tile * a.b.count + s) * a.c.heads + head) * a.parts;
}
template <int D, int R>
__device__ inline kw2_t* part_totals(const AttnArgs& a) {
  return reinterpret_cast<kw2_t*>(a.part + (size_t)a.tiles * a.b.count * a.c.heads * a.parts * R * D);
}

// What the rows first .. last (token * group + query head) of a sequence see.
__device__ inline Range range_of_rows(const AttnArgs& a, const Span& sp, int first, int last) {
  return range_of(a, sp, max(sp.from + first / a.group, 0), sp.from + last / a.group);
}

// Tokens [low, high) that the row at position pos sees.
struct Sees {
  int low, high;
};
__device__ inline Sees sees_of(const AttnArgs& a, const Span& sp, int pos, bool there) {
  Sees s = {a.window > 0 ? max(pos - a.window + 1, 0) : 0, a.causal ? min(pos + 1, sp.len) : sp.len};
  if (!there || (a.causal && pos < 0)) s.high = 0;
  return s;
}

// A row's running softmax, held by every lane of the row: the reference of
// the exponents (log2), the sum of the weights, and the scale of the values in
// whose units the sums stand.
//
// The reference follows the largest score only where that has grown by more
// than kLag (weights stay below 2^5; exponents and FP16's 11 bits do not
// care), and the units follow the pages' scales only where a page's is larger
// or kSpan times smaller: most pages rescale nothing.  A weight meets the codes
// in FP16, in the sums' units: times kLift and the page's scale, over the unit
// (below FP16's 2^16).  Where the page's scale is the unit, weights down to
// 2^-24 of the reference keep their 11 bits and smaller ones are off by 2^-35 of
// it at most; where it is kSpan times smaller, 2^-18 and 2^-29, of values that
// are as much smaller.
constexpr float kLag = 5.0f, kSpan = 64.0f, kLift = 1024.0f;
struct Row {
  float top, sum, unit, inv;  // inv: 1 / unit
};
__device__ inline Row new_row() { return {-INFINITY, 0.f, 0.f, 1.f}; }

// The row before the weights of a page: best is its largest score there
// (minus infinity: it sees nothing of it), scale the page's, not 0.  Returns
// what the row's sums have to be multiplied with.  A weight in the units of the
// sums is exp2(score - top_of(r) + lift), and `back` times that in its own.  A
// scale that is NaN goes into the sums of the rows that see a token of its page
// alone.
__device__ inline float top_of(const Row& r) { return r.top == -INFINITY ? 0.f : r.top; }
__device__ inline float step_row(Row& r, float best, float scale, float& lift, float& back) {
  const bool sees = best > -INFINITY;
  float factor = 1.0f;
  if (best > r.top + kLag || (sees && r.top == -INFINITY)) {
    factor = r.top == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(r.top - best);
    r.sum *= factor;
    r.top = best;
  }
  if (sees && (scale > r.unit || scale * kSpan < r.unit)) {
    r.inv = 1.0f / scale;
    factor *= r.unit * r.inv;
    r.unit = scale;
  }
  const float ratio = !sees ? 1.0f : scale == r.unit ? kLift : kLift * scale * r.inv;
  back = __builtin_amdgcn_rcpf(ratio);
  lift = __builtin_amdgcn_logf(ratio);
  return factor;
}

// The larger of a lane's value and its partner's, 32 or 16 lanes on, by swaps
// between registers: a shuffle's way through the LDS queues behind the operands'
// reads (128 pages of a 64-row tile 175 -> 169 us).
__device__ inline float max_of_32(float v) {
  const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ inline float max_of_16(float v) {
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}

// Four values of a row of y (0 where the row has seen nothing).
__device__ inline void finish_row(const AttnArgs& a, size_t at, kf4_t v, float sum) {
  const float inv = sum == 0.f ? 0.f : 1.0f / sum;
  v *= inv;
  *reinterpret_cast<kh4_t*>(a.y + at) = kh4_t{(_Float16)v.x, (_Float16)v.y, (_Float16)v.z, (_Float16)v.w};
}
#endif

}  // namespace tern
