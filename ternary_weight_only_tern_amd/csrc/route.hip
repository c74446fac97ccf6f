// Routing of tokens to experts: scores (softmax or sigmoid), a selection key
// (score + bias), selection of groups, top-k, weights.  The definition
// stands at tern_route in tern.h.
//
// One wavefront per token; lane l holds the experts l, l + 64, ...  What is
// chosen hangs on the order of the keys alone, so they are FP64: FP32 scores
// near 1 (sigmoid) or tiny ones (softmax) tie where the exact ones do not.
// Without a bias both scores grow with the logit and the logit itself is the
// key.  A round of the top-k takes the largest key of the wavefront, the
// lowest expert among equals.
#include "q4.h"

namespace tern {
namespace {

constexpr int kRowsPerWg = 4;

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

template <int F16>
__device__ inline float load_logit(const void* logits, size_t i) {
  float v = F16 ? (float)reinterpret_cast<const _Float16*>(logits)[i] : reinterpret_cast<const float*>(logits)[i];
  if (!(v == v)) v = -INFINITY;
  return fminf(v, 3.4028234663852886e38f);
}

// The score of a logit that is not minus infinity (top, total: softmax's).
__device__ inline double score_of(float l, int sigmoid, float top, double total) {
  return sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - (double)top) / total;
}

template <int EPL, int F16>
__global__ __launch_bounds__(kRowsPerWg * 64) void route_kernel(const RouteArgs a) {
  __shared__ double keys[kRowsPerWg][EPL * 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int row = blockIdx.x * kRowsPerWg + wave;
  if (row >= a.m) return;  // no barrier below: a wavefront works alone
  const size_t base = (size_t)row * a.experts;

  float l[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = i * 64 + lane;
    l[i] = -INFINITY;
    if (e < a.experts) l[i] = load_logit<F16>(a.logits, base + e);
  }
  const bool plain_key = a.bias == nullptr && (a.groups == 1 || a.best == 1);
  float top = 0.f;
  double total = 1.0;
  if (!a.sigmoid) {
    top = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) top = fmaxf(top, l[i]);
    top = wave_max(top);
    if (top == -INFINITY) top = 0.f;
    if (!plain_key || !a.renorm) {
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (l[i] != -INFINITY) sum += exp((double)l[i] - (double)top);
      total = fmax(wave_sum(sum), 1.0);
    }
  }
  double key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = i * 64 + lane;
    key[i] = l[i];
    if (!plain_key && l[i] != -INFINITY) {
      key[i] = score_of(l[i], a.sigmoid, top, total);
      if (a.bias) key[i] += (double)a.bias[e];
      if (!(key[i] == key[i])) key[i] = -INFINITY;
    }
  }

  if (a.groups > 1) {
    const int size = a.experts / a.groups;
#pragma unroll
    for (int i = 0; i < EPL; ++i) keys[wave][i * 64 + lane] = key[i];
    __builtin_amdgcn_wave_barrier();
    __threadfence_block();
    double one = -INFINITY, two = -INFINITY;
    if (lane < a.groups)
      for (int i = 0; i < size; ++i) {
        const double v = keys[wave][lane * size + i];
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

  int mine = -1;
  for (int j = 0; j < a.topk; ++j) {
    double best = -INFINITY;
    int at = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i * 64 + lane;
      }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double v = __shfl_xor(best, d);
      const int w = __shfl_xor(at, d);
      if (v > best || (v == best && w < at)) {
        best = v;
        at = w;
      }
    }
    if (best == -INFINITY) break;
    if (lane == j) mine = at;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (at == i * 64 + lane) key[i] = -INFINITY;
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

template <int F16>
hipError_t pick(const RouteArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.m + kRowsPerWg - 1) / kRowsPerWg)), block(kRowsPerWg * 64);
  if (a.experts <= 64)
    hipLaunchKernelGGL((route_kernel<1, F16>), grid, block, 0, s, a);
  else if (a.experts <= 128)
    hipLaunchKernelGGL((route_kernel<2, F16>), grid, block, 0, s, a);
  else if (a.experts <= 256)
    hipLaunchKernelGGL((route_kernel<4, F16>), grid, block, 0, s, a);
  else if (a.experts <= 512)
    hipLaunchKernelGGL((route_kernel<8, F16>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((route_kernel<16, F16>), grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, int f16, hipStream_t s) { return f16 ? pick<1>(a, s) : pick<0>(a, s); }

}  // namespace tern
