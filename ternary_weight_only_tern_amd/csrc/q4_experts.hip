// The routed experts' bookkeeping around the products of q4_rows.hip and
// q4_tile.hip (which tile of rows belongs to which expert, the weighted sum
// of a token's slots), and the packing of 4-bit codes.
#include "q4.h"

namespace tern {
namespace {

constexpr int kPlanThreads = 1024, kBatch = 8;  // kBatch ids requested before any is used

// Sorts the slots by expert: order[position] = slot, place[slot] = position
// (-1 for a slot that names no expert), and cuts every expert's positions
// into tiles of at most `rows`.  One workgroup: 42 slots 3.1 us, 16384 slots
// 12 us, bound by the latency of reading the ids and of the LDS atomics.  Where inside its expert a
// slot lands depends on the order of the LDS atomics, but a row's result does
// not depend on its place: the matrix instructions' rows are independent.
__global__ __launch_bounds__(kPlanThreads) void q4_plan_kernel(const int32_t* ids, int slots, int experts, int rows,
                                                               int4* tiles, int32_t* ntiles, int32_t* order,
                                                               int32_t* place) {
  __shared__ int count[kPlanThreads], wave_rows[kPlanThreads / 64], wave_tiles[kPlanThreads / 64];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  int e[kBatch];  // the batch at hand; the last one counted is kept
  int s0 = t;
  auto fetch = [&](int from) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) e[i] = from + i * kPlanThreads < slots ? ids[from + i * kPlanThreads] : -1;
  };
  fetch(s0);
  count[t] = 0;
  __syncthreads();
  while (true) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if ((unsigned)e[i] < (unsigned)experts) atomicAdd(&count[e[i]], 1);
    if (s0 + kPlanThreads * kBatch >= slots) break;
    fetch(s0 += kPlanThreads * kBatch);
  }
  __syncthreads();
  // running sums over the experts: inside a wavefront, then over wavefronts
  const int mine = count[t], tl = (mine + rows - 1) / rows;
  int f = mine, q = tl;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int a = __shfl_up(f, d), b = __shfl_up(q, d);
    if (lane >= d) f += a, q += b;
  }
  if (lane == 63) wave_rows[wave] = f, wave_tiles[wave] = q;
  __syncthreads();
  for (int w = 0; w < wave; ++w) f += wave_rows[w], q += wave_tiles[w];
  if (t == kPlanThreads - 1) *ntiles = q;
  f -= mine;
  q -= tl;
  count[t] = f;
  for (int i = 0; i < tl; ++i) tiles[q + i] = make_int4(t, f + i * rows, min(rows, mine - i * rows), 0);
  __syncthreads();
  for (;; fetch(s0 -= kPlanThreads * kBatch)) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int s = s0 + i * kPlanThreads;
      int p = -1;
      if ((unsigned)e[i] < (unsigned)experts) {
        p = atomicAdd(&count[e[i]], 1);
        order[p] = s;
      }
      if (s < slots) place[s] = p;
    }
    if (s0 < kPlanThreads * kBatch) break;
  }
}

// y[token] = sum over its slots, in slot order, of gate * part[place]; four
// columns a thread (V = 4: n a multiple of four).  Bound by the reading of
// the partials: 16384 slots of 2560 columns 27.4 us, 6.5 TB/s.
template <int V>
__global__ __launch_bounds__(256) void q4_combine_kernel(const float* part, const int32_t* place, const float* gates,
                                                         int topk, int n, void* y, int y_f32) {
  const size_t first = (size_t)blockIdx.x * topk;
  for (uint32_t c = (blockIdx.y * 256 + threadIdx.x) * V; c < (uint32_t)n; c += gridDim.y * 256 * V) {
    float sum[V] = {};
#pragma unroll 4
    for (int j = 0; j < topk; ++j) {
      const int p = place[first + j];
      if (p < 0) continue;
      const float g = gates[first + j];
      const float* from = part + (size_t)p * n + c;
      if (V == 4) {
        const f4_t v = *reinterpret_cast<const f4_t*>(from);
#pragma unroll
        for (int i = 0; i < V; ++i) sum[i] += g * v[i];
      } else {
        sum[0] += g * from[0];
      }
    }
    const size_t dst = (size_t)blockIdx.x * n + c;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (y_f32)
        reinterpret_cast<float*>(y)[dst + i] = sum[i];
      else
        reinterpret_cast<_Float16*>(y)[dst + i] = (_Float16)sum[i];
    }
  }
}

// Eight codes (one byte each) to a word: offset o in bits 16 (o % 2) + 4 (o / 2).
__global__ __launch_bounds__(256) void q4_pack_kernel(const uint8_t* q, size_t words, uint8_t* codes, uint32_t* flag) {
  const size_t step = (size_t)gridDim.x * 256;
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < words; i += step) {
    const w2_t v = reinterpret_cast<const w2_t*>(q)[i];
    uint32_t word = 0;
#pragma unroll
    for (int o = 0; o < 8; ++o) word |= ((((o < 4 ? v.x : v.y) >> (8 * (o % 4))) & 15u)) << (16 * (o % 2) + 4 * (o / 2));
    if ((v.x | v.y) & 0xF0F0F0F0u) *flag = 1;
    reinterpret_cast<uint32_t*>(codes)[i] = word;
  }
}

__global__ __launch_bounds__(256) void q4_unpack_kernel(const uint8_t* codes, size_t words, uint8_t* q) {
  const size_t step = (size_t)gridDim.x * 256;
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < words; i += step) {
    const uint32_t word = reinterpret_cast<const uint32_t*>(codes)[i];
    uint32_t v[2] = {0, 0};
#pragma unroll
    for (int o = 0; o < 8; ++o) v[o / 4] |= ((word >> (16 * (o % 2) + 4 * (o / 2))) & 15u) << (8 * (o % 4));
    reinterpret_cast<w2_t*>(q)[i] = w2_t{v[0], v[1]};
  }
}

__global__ void q4_clear_kernel(uint32_t* flag) { *flag = 0; }

unsigned blocks_for(size_t items) {
  const size_t b = (items + 255) / 256;
  return (unsigned)(b < 8192 ? b : 8192);
}

}  // namespace

hipError_t launch_q4_plan(const int32_t* ids, int slots, int experts, int rows, int4* tiles, int32_t* ntiles,
                          int32_t* order, int32_t* place, hipStream_t s) {
  hipLaunchKernelGGL(q4_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, ids, slots, experts, rows, tiles, ntiles, order,
                     place);
  return hipGetLastError();
}

hipError_t launch_q4_combine(const float* part, const int32_t* place, const float* gates, int m, int topk, int n,
                             void* y, int y_f32, hipStream_t s) {
  const int v = n % 4 ? 1 : 4, blocks = (n + 256 * v - 1) / (256 * v);
  const dim3 grid((unsigned)m, (unsigned)(blocks < 64 ? blocks : 64));
  if (v == 4)
    hipLaunchKernelGGL((q4_combine_kernel<4>), grid, dim3(256), 0, s, part, place, gates, topk, n, y, y_f32);
  else
    hipLaunchKernelGGL((q4_combine_kernel<1>), grid, dim3(256), 0, s, part, place, gates, topk, n, y, y_f32);
  return hipGetLastError();
}

hipError_t launch_q4_pack(const uint8_t* q, size_t words, uint8_t* codes, uint32_t* flag, hipStream_t s) {
  hipLaunchKernelGGL(q4_clear_kernel, dim3(1), dim3(1), 0, s, flag);
  if (words) hipLaunchKernelGGL(q4_pack_kernel, dim3(blocks_for(words)), dim3(256), 0, s, q, words, codes, flag);
  return hipGetLastError();
}

hipError_t launch_q4_unpack(const uint8_t* codes, size_t words, uint8_t* q, hipStream_t s) {
  if (words) hipLaunchKernelGGL(q4_unpack_kernel, dim3(blocks_for(words)), dim3(256), 0, s, codes, words, q);
  return hipGetLastError();
}

}  // namespace tern
