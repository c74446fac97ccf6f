// Routing of tokens to experts: scores (softmax or sigmoid), a selection key
// (score + bias), selection of groups, top-k, weights.  The definition
// stands at tern_route in tern.h.
//
// What is chosen hangs on the order of the keys alone, so their order is
// that of the FP64 keys: FP32 scores near 1 (sigmoid) or tiny ones (softmax)
// tie where the exact ones do not.  Without a bias both scores grow with the
// logit and the logit itself is the key: where FP64 scores tie too (sigmoids
// of logits past 36, softmax scores 745 below the largest), it does not.
// Groups judged by two such experts go by the FP64 sums of their scores.
//
// Most rows need few FP64 keys.  route_kernel packs an FP32 key, rounded down
// by at most 256 steps, and its expert into one word, lets 16 or 32 lanes a
// token take the largest word topk + 1 times (a lane keeps its words sorted,
// the lanes' heads meet in four or five DPP steps), and looks at the gaps
// between the words taken: where every gap is wider than the keys' errors,
// the order is the exact one (logits from FP16 are exact in the word).
// Otherwise the FP64 keys of the words up to the next wide gap put these in
// order; groups in doubt are told apart by their FP64 sums.  A token that
// finds no such gap, or a softmax with a bias and a doubt, is routed again by
// exact_row, 64 lanes and FP64 keys for every expert.
// 16384 tokens, 256 experts, sigmoid, bias, 4 of 8 groups, top 8: 15.0 us,
// bound by the vector instructions (37 tokens of it 6.3 us, one token of 64
// experts 2.9 us: latency).
#include "q4.h"

namespace tern {
namespace {

constexpr int kWaves = 4;  // of a workgroup

__device__ inline double wave_sum(double v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  return v;
}
__device__ inline float wave_max(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}

// NaN counts as minus infinity, plus infinity as the largest value, -0 as 0.
__device__ inline float clean_logit(float v) {
  if (!(v == v)) v = -INFINITY;
  return fminf(v, 3.4028234663852886e38f) + 0.0f;
}

template <int F16>
__device__ inline float load_logit(const void* logits, size_t i) {
  float v = F16 ? (float)reinterpret_cast<const _Float16*>(logits)[i] : reinterpret_cast<const float*>(logits)[i];
  return clean_logit(v);
}

// The score of a logit that is not minus infinity (top, total: softmax's).
__device__ inline double score_of(float l, int sigmoid, float top, double total) {
  return sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - (double)top) / total;
}

template <int CTRL>
__device__ inline uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xF, 0xF, false);
}

// The largest word of LPR consecutive lanes (16, 32 or 64), in all of them.
template <int LPR>
__device__ inline uint32_t lanes_max(uint32_t v) {
  v = max(v, dpp<0x128>(v));  // row_ror 8, 4, 2, 1: the 16 lanes of a DPP row
  v = max(v, dpp<0x124>(v));
  v = max(v, dpp<0x122>(v));
  v = max(v, dpp<0x121>(v));
  if (LPR >= 32) {
    const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max(p[0], p[1]);
  }
  if (LPR == 64) {
    const auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = max(p[0], p[1]);
  }
  return v;
}

// FP64's bits in order; 0 for a masked expert.
__device__ inline uint64_t sortable(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);  // no -0: it ties with 0
  return v == -INFINITY ? 0 : (int64_t)b < 0 ? ~b : b | 0x8000000000000000ull;
}

// One token by one wavefront, keys in FP64; keys: its LDS, EPL * 64.
template <int EPL, int F16>
__device__ inline void exact_row(const RouteArgs& a, int row, double* keys) {
  const int lane = threadIdx.x & 63;
  const size_t base = (size_t)row * a.experts;

  float l[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = i * 64 + lane;
    l[i] = -INFINITY;
    if (e < a.experts) l[i] = load_logit<F16>(a.logits, base + e);
  }
  const bool plain_key = a.bias == nullptr;                          // the logit is the key
  const bool score_sums = plain_key && a.groups > 1 && a.best == 2;  // but groups go by scores
  float top = 0.f;
  double total = 1.0;
  if (!a.sigmoid) {
    top = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) top = fmaxf(top, l[i]);
    top = wave_max(top);
    if (top == -INFINITY) top = 0.f;
    if (!plain_key || score_sums || !a.renorm) {
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (l[i] != -INFINITY) sum += exp((double)l[i] - (double)top);
      total = fmax(wave_sum(sum), 1.0);
    }
  }
  double key[EPL];
  // One evaluation of the score serves key and group: a second one made the
  // packed kernel spill (16384 x 256 with a bias 16.3 against 15.0 us).
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = i * 64 + lane;
    key[i] = l[i];
    double judged = l[i];  // what its group goes by
    if ((!plain_key || score_sums) && l[i] != -INFINITY) {
      judged = score_of(l[i], a.sigmoid, top, total);
      if (a.bias) {
        judged += (double)a.bias[e];
        if (!(judged == judged)) judged = -INFINITY;
        key[i] = judged;
      }
    }
    if (a.groups > 1) keys[i * 64 + lane] = judged;
  }

  if (a.groups > 1) {
    const int size = a.experts / a.groups;
    __builtin_amdgcn_wave_barrier();
    __threadfence_block();
    double one = -INFINITY, two = -INFINITY;
    if (lane < a.groups)
      for (int i = 0; i < size; ++i) {
        const double v = keys[lane * size + i];
        if (v > one) {
          two = one;
          one = v;
        } else if (v > two) {
          two = v;
        }
      }
    double sum = one;
    if (a.best == 2 && two != -INFINITY) sum += two;
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
      const double v = __shfl(sum, g);
      if (v > sum || (v == sum && g < lane)) ++rank;
    }
    const unsigned long long kept = __ballot(lane < a.groups && rank < a.keep);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = i * 64 + lane;
      if (e < a.experts && !((kept >> (e / size)) & 1)) key[i] = -INFINITY;
    }
  }

  uint64_t q[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) q[i] = sortable(key[i]);
  int mine = -1;
  for (int j = 0; j < a.topk; ++j) {
    uint64_t best = 0;
    uint32_t at = 0;  // 1024 - expert: the lowest expert among equals
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (q[i] > best) {
        best = q[i];
        at = 1024 - (i * 64 + lane);
      }
    const uint32_t hi = lanes_max<64>((uint32_t)(best >> 32));
    if (hi == 0) break;  // only masked ones are left (an unmasked word has bits there)
    const uint32_t lo = lanes_max<64>((uint32_t)(best >> 32) == hi ? (uint32_t)best : 0u);
    const uint32_t who = lanes_max<64>((uint32_t)(best >> 32) == hi && (uint32_t)best == lo ? at : 0u);
    const int e = 1024 - (int)who;
    if (lane == j) mine = e;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (e == i * 64 + lane) q[i] = 0;
  }

  double g = 0.0;
  if (mine >= 0) g = score_of(load_logit<F16>(a.logits, base + mine), a.sigmoid, top, total);
  if (a.renorm) {
    const double sum = wave_sum(g);
    g = sum > 0.0 ? g / sum : 0.0;
  }
  if (lane < a.topk) {
    a.ids[(size_t)row * a.topk + lane] = mine;
    a.weights[(size_t)row * a.topk + lane] = (float)(g * (double)a.scale);
  }
}

template <int EPL, int F16>
__global__ __launch_bounds__(kWaves * 64) void route_exact_kernel(const RouteArgs a) {
  __shared__ double keys[kWaves][EPL * 64];
  const int wave = threadIdx.x >> 6, row = blockIdx.x * kWaves + wave;
  if (row < a.m) exact_row<EPL, F16>(a, row, keys[wave]);  // no barrier inside
}

// ---- packed keys
// Sortable words, expert in the low eight bits (the lower expert larger), 0
// for a masked one.  Keys that are logits: FP32's bits in order.  Scores plus
// bias: fixed point, 2^-29, for |key| < 2 (others are in doubt).
__device__ inline uint32_t pack_float(float v, int e) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  return (((int32_t)b < 0 ? ~b : b | 0x80000000u) & ~255u) | (uint32_t)(255 - e);
}
__device__ inline float unpack_float(uint32_t w) {
  w &= ~255u;
  return __builtin_bit_cast(float, w & 0x80000000u ? w & 0x7FFFFFFFu : ~w);
}
__device__ inline uint32_t pack_fixed(float v, int e) {
  return (((uint32_t)(int32_t)(v * 0x1p29f) ^ 0x80000000u) & ~255u) | (uint32_t)(255 - e);
}
__device__ inline float unpack_fixed(uint32_t w) { return (float)(int32_t)((w & ~255u) ^ 0x80000000u) * 0x1p-29f; }

// Two packed keys nearer than this are in doubt: an FP32 sigmoid is off by
// 2^-22 at most (|l| 2^-23 + 2^-23 from the exponential, times a slope of 1/4
// and at most 0.23 / |l|; the sum and the reciprocal), a softmax score by
// 2^-20.5 (its sum's error among them), a bias's addition by 2^-23, and a
// word drops up to 2^-21.
constexpr int kMore = 4;  // words beyond the topk-th that settle a doubt about it
constexpr float kSigmoidDoubt = 0x1p-19f, kSoftmaxDoubt = 0x1p-18f;


// LPR lanes a token, EPL consecutive experts each.  Takes topk + kMore <= LPR and, if
// there are groups, whole runs of a power of two of lanes.
template <int LPR, int EPL, int F16>
__global__ __launch_bounds__(kWaves * 64, 8) void route_kernel(const RouteArgs a) {
  constexpr int RPW = 64 / LPR;                       // tokens of a wavefront
  constexpr int XPL = (LPR * EPL + 63) / 64;          // experts per lane of exact_row
  constexpr unsigned long long kMine = LPR == 32 ? 0xFFFFFFFFull : 0xFFFFull;
  __shared__ double keys[kWaves][XPL * 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int in = lane % LPR;                          // lane among the token's
  const int first = (blockIdx.x * kWaves + wave) * RPW, row = first + lane / LPR;
  if (first >= a.m) return;  // no barrier below: a wavefront works alone
  const size_t base = (size_t)min(row, a.m - 1) * a.experts;
  const bool plain_key = a.bias == nullptr;                          // the logit is the key
  const bool score_sums = plain_key && a.groups > 1 && a.best == 2;  // but groups go by scores

  // this lane's logits and biases: 16 bytes a load where rows allow it
  float l[EPL], bias[EPL] = {};
  const bool whole = a.experts % EPL == 0 && !((uintptr_t)a.logits & 15) && !((uintptr_t)a.bias & 15);
  if (whole) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[i] = -INFINITY;
    if (in * EPL < a.experts) {
      if (F16) {
        typedef _Float16 hv_t __attribute__((ext_vector_type(EPL)));
        const hv_t v = *reinterpret_cast<const hv_t*>(reinterpret_cast<const _Float16*>(a.logits) + base + in * EPL);
#pragma unroll
        for (int i = 0; i < EPL; ++i) l[i] = (float)v[i];
      } else {
#pragma unroll
        for (int i = 0; i < EPL; i += 4) {
          const f4_t v = *reinterpret_cast<const f4_t*>(reinterpret_cast<const float*>(a.logits) + base + in * EPL + i);
#pragma unroll
          for (int j = 0; j < 4; ++j) l[i + j] = v[j];
        }
      }
      if (a.bias) {
#pragma unroll
        for (int i = 0; i < EPL; i += 4) {
          const f4_t v = *reinterpret_cast<const f4_t*>(a.bias + in * EPL + i);
#pragma unroll
          for (int j = 0; j < 4; ++j) bias[i + j] = v[j];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[i] = clean_logit(l[i]);
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = in * EPL + i;
      l[i] = -INFINITY;
      if (e < a.experts) {
        l[i] = load_logit<F16>(a.logits, base + e);
        if (a.bias) bias[i] = a.bias[e];
      }
    }
  }
  // softmax: the largest logit, and the sum where it is needed: FP64 for the
  // weights, FP32 for packed keys
  float top = 0.f;
  double total = 1.0;
  if (!a.sigmoid) {
    float most = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) most = fmaxf(most, l[i]);
    const uint32_t b = __builtin_bit_cast(uint32_t, most);
    const uint32_t w = lanes_max<LPR>((int32_t)b < 0 ? ~b : b | 0x80000000u);
    top = __builtin_bit_cast(float, w & 0x80000000u ? w & 0x7FFFFFFFu : ~w);
    if (top == -INFINITY) top = 0.f;
    if (!a.renorm || !plain_key || score_sums) {
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        if (a.renorm)
          sum += (double)__expf(l[i] - top);
        else if (l[i] != -INFINITY)
          sum += exp((double)l[i] - (double)top);
      }
#pragma unroll
      for (int d = 1; d < LPR; d <<= 1) sum += __shfl_xor(sum, d);
      total = fmax(sum, 1.0);
    }
  }

  uint32_t q[EPL];
  bool doubt = false;
  const float share = (float)(1.0 / total);
  auto fast_score = [&](float v) {
    return a.sigmoid ? __builtin_amdgcn_rcpf(1.0f + __expf(-v)) : __expf(v - top) * share;
  };
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = in * EPL + i;
    float c = l[i];
    if (!plain_key) {
      c = fast_score(l[i]) + bias[i];
      if (l[i] == -INFINITY || !(c == c)) c = -INFINITY;
      if (c != -INFINITY && !(fabsf(c) < 2.0f)) doubt = true;
    }
    q[i] = c == -INFINITY ? 0u : plain_key ? pack_float(c, e) : pack_fixed(fabsf(c) < 2.0f ? c : 0.0f, e);
  }
  // the lane's words, largest first
  auto order = [&](int i, int j) {
    const uint32_t hi = max(q[i], q[j]), lo = min(q[i], q[j]);
    q[i] = hi;
    q[j] = lo;
  };
  if (EPL == 8) {
    order(0, 1), order(2, 3), order(4, 5), order(6, 7);
    order(0, 2), order(1, 3), order(4, 6), order(5, 7);
    order(1, 2), order(5, 6), order(0, 4), order(3, 7);
    order(1, 5), order(2, 6);
    order(1, 4), order(3, 6);
    order(2, 4), order(3, 5);
    order(3, 4);
  } else {
    order(0, 1), order(2, 3), order(0, 2), order(1, 3), order(1, 2);
  }
  auto value = [&](uint32_t w) { return plain_key ? unpack_float(w) : unpack_fixed(w); };
  // how far apart two packed keys must be for their order to be certain
  const bool exact_keys = plain_key && F16;
  const float score_margin = a.sigmoid ? kSigmoidDoubt : kSoftmaxDoubt;
  auto margin = [&](float v) { return plain_key ? fabsf(v) * 0x1p-14f : score_margin; };

  if (a.groups > 1) {
    const int span = a.experts / a.groups / EPL;  // lanes of a group, a power of two
    uint32_t one = q[0], two = q[1];
    for (int d = 1; d < span; d <<= 1) {
      const uint32_t o1 = __shfl_xor(one, d), o2 = __shfl_xor(two, d);
      two = max(min(one, o1), max(two, o2));
      one = max(one, o1);
    }
    float sum = one ? value(one) : -INFINITY;
    // From the logits themselves: a word has dropped bits that a score may
    // hang on.
    if (score_sums) {
      float first_score = -INFINITY, second_score = -INFINITY;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const float v = l[i] == -INFINITY ? -INFINITY : fast_score(l[i]);
        second_score = fmaxf(second_score, fminf(first_score, v));
        first_score = fmaxf(first_score, v);
      }
      for (int d = 1; d < span; d <<= 1) {
        const float o1 = __shfl_xor(first_score, d), o2 = __shfl_xor(second_score, d);
        second_score = fmaxf(fminf(first_score, o1), fmaxf(second_score, o2));
        first_score = fmaxf(first_score, o1);
      }
      sum = second_score == -INFINITY ? first_score : first_score + second_score;
    } else if (a.best == 2 && two) {
      sum += value(two);
    }
    const int mine = in / span;
    int rank = 0;  // groups before this one
    for (int g = 0; g < a.groups; ++g) {
      const float v = __shfl(sum, lane - in + g * span);
      if (v > sum || (v == sum && g < mine)) ++rank;
    }
    if (!exact_keys || score_sums) {  // the last group kept, certainly before the next?
      const uint32_t b = __builtin_bit_cast(uint32_t, sum), w = (int32_t)b < 0 ? ~b : b | 0x80000000u;
      const bool kept = rank < a.keep && in < a.groups * span;
      const uint32_t least = ~lanes_max<LPR>(kept ? ~w : 0u), most = lanes_max<LPR>(kept || in >= a.groups * span ? 0u : w);
      auto back = [](uint32_t v) { return __builtin_bit_cast(float, v & 0x80000000u ? v & 0x7FFFFFFFu : ~v); };
      const float x = back(least), y = back(most);
      const bool unsure = most && y != -INFINITY && !(x - y > 2.0f * (score_sums ? score_margin : margin(x)));
      if (__ballot(unsure)) {
        if ((!plain_key || score_sums) && !a.sigmoid) {
          doubt = doubt || unsure;
        } else {  // the groups' FP64 sums
          double first_key = -INFINITY, second_key = -INFINITY;
          for (int i = 0; i < EPL; ++i) {
            const int e = in * EPL + i;
            const float v = e < a.experts ? load_logit<F16>(a.logits, base + e) : -INFINITY;
            double k = v;
            if ((!plain_key || score_sums) && v != -INFINITY) {
              k = score_of(v, 1, 0.f, 1.0) + (a.bias ? (double)a.bias[e] : 0.0);
              if (!(k == k)) k = -INFINITY;
            }
            second_key = fmax(second_key, fmin(first_key, k));
            first_key = fmax(first_key, k);
          }
          for (int d = 1; d < span; d <<= 1) {
            const double o1 = __shfl_xor(first_key, d), o2 = __shfl_xor(second_key, d);
            second_key = fmax(fmin(first_key, o1), fmax(second_key, o2));
            first_key = fmax(first_key, o1);
          }
          double total_key = first_key;
          if (a.best == 2 && second_key != -INFINITY) total_key += second_key;
          rank = 0;
          for (int g = 0; g < a.groups; ++g) {
            const double v = __shfl(total_key, lane - in + g * span);
            if (v > total_key || (v == total_key && g < mine)) ++rank;
          }
        }
      }
    }
    if (rank >= a.keep) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) q[i] = 0;
    }
  }

  // lane j keeps the j-th word taken, topk + 1 of them
  uint32_t kept = 0;
  auto take = [&](int j) {
    const uint32_t w = lanes_max<LPR>(q[0]);
    if (in == j) kept = w;
    const bool taken = q[0] == w;  // words differ, but for the zeros at the end
#pragma unroll
    for (int i = 0; i + 1 < EPL; ++i) q[i] = taken ? q[i + 1] : q[i];
    q[EPL - 1] = taken ? 0u : q[EPL - 1];
  };
  for (int j = 0; j <= a.topk; ++j) take(j);
  auto certain = [&]() {  // this lane's word is larger than the next in FP64 too
    const uint32_t next = __shfl_down(kept, 1);
    const float v = value(kept);
    return exact_keys || !next || v - value(next) > margin(v);
  };
  int at = in;  // where this lane's expert goes
  bool sure = certain();  // by every lane: a lane reads its neighbour's word
  if (__ballot(in < a.topk && !sure)) {
    // A few more words, up to a certain gap; the FP64 keys of those before it
    // give the order.
    for (int j = a.topk + 1; j < a.topk + kMore; ++j) take(j);
    sure = certain();
    const unsigned long long gap = __ballot(in >= a.topk - 1 && in < a.topk + kMore - 1 && sure) >> (lane - in) & kMine;
    if (!gap || (!plain_key && !a.sigmoid)) doubt = true;
    const int count = gap ? __ffsll(gap) : 0;  // words before the gap
    if (in >= count) kept = 0;
    const int e = kept ? 255 - (int)(kept & 255u) : -1;
    double key = -INFINITY;
    if (e >= 0) {
      const float v = load_logit<F16>(a.logits, base + e);
      key = plain_key ? (double)v : score_of(v, 1, 0.f, 1.0) + (a.bias ? (double)a.bias[e] : 0.0);
      at = 0;
    }
    for (int i = 0; i < a.topk + kMore; ++i) {
      const double k = __shfl(key, lane - in + i);
      const int o = __shfl(e, lane - in + i);
      if (e >= 0 && o >= 0 && (k > key || (k == key && o < e))) ++at;
    }
  } else if (in >= a.topk) {
    kept = 0;
  }
  const int mine = at < a.topk && kept ? 255 - (int)(kept & 255u) : -1;

  double g = 0.0;
  if (mine >= 0) g = score_of(load_logit<F16>(a.logits, base + mine), a.sigmoid, top, a.renorm ? 1.0 : total);
  if (a.renorm) {
    double sum = g;  // of the first lanes, a power of two of them
    for (int d = 1; d < a.topk + kMore; d <<= 1) sum += __shfl_xor(sum, d);
    g = sum > 0.0 ? g / sum : 0.0;
  }
  const unsigned long long again = __ballot(doubt);
  if (row < a.m && at < a.topk && !(again & (kMine << (lane - in)))) {
    a.ids[(size_t)row * a.topk + at] = mine;
    a.weights[(size_t)row * a.topk + at] = (float)(g * (double)a.scale);
  }
  if (again) {
    for (int t = 0; t < RPW; ++t)
      if (first + t < a.m && (again & (kMine << (t * LPR)))) exact_row<XPL, F16>(a, first + t, keys[wave]);
  }
}

template <int LPR, int EPL, int F16>
hipError_t launch(const RouteArgs& a, hipStream_t s) {
  constexpr int rows = kWaves * (64 / LPR);
  hipLaunchKernelGGL((route_kernel<LPR, EPL, F16>), dim3((unsigned)((a.m + rows - 1) / rows)), dim3(kWaves * 64), 0, s, a);
  return hipGetLastError();
}

template <int EPL, int F16>
hipError_t launch_exact(const RouteArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((route_exact_kernel<EPL, F16>), dim3((unsigned)((a.m + kWaves - 1) / kWaves)), dim3(kWaves * 64), 0, s, a);
  return hipGetLastError();
}

template <int F16>
hipError_t pick(const RouteArgs& a, hipStream_t s) {
  const int lpr = a.experts <= 128 ? 16 : 32, epl = a.experts <= 64 ? 4 : 8;
  const int size = a.experts / a.groups, span = size / epl;
  const bool packed = a.experts <= 256 && a.topk + kMore <= lpr && (a.groups == 1 || (size % epl == 0 && (span & (span - 1)) == 0));
  if (packed) {
    if (a.experts <= 64) return launch<16, 4, F16>(a, s);
    if (a.experts <= 128) return launch<16, 8, F16>(a, s);
    return launch<32, 8, F16>(a, s);
  }
  if (a.experts <= 64) return launch_exact<1, F16>(a, s);
  if (a.experts <= 128) return launch_exact<2, F16>(a, s);
  if (a.experts <= 256) return launch_exact<4, F16>(a, s);
  if (a.experts <= 512) return launch_exact<8, F16>(a, s);
  return launch_exact<16, F16>(a, s);
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, int f16, hipStream_t s) { return f16 ? pick<1>(a, s) : pick<0>(a, s); }

}  // namespace tern
