// Attention of few rows over the 8-bit cache (tern_kv_attention in tern.h):
//   y = sum_t exp(z_t) v_t / sum_t exp(z_t),  z_t = scale q . k_t.
//
// The rows of a sequence and the query heads that share a cache head, R =
// rows * group of them, are the 16 columns of a matrix operand (NT of them).
// A workgroup's four wavefronts walk the pages of their part of the context,
// a page each at a time: 16-byte loads of codes in operand order (kv.h), K^T
// products in FP32 from exact FP16 codes, one page's softmax in registers, the
// weights rounded to FP16 (the only rounding; 2^-11 of a weight, as the
// output's own) against the value codes.  The keys' scale multiplies the
// scores, the values' scale the weights, in FP32.  The next page's keys are
// requested when this page's have been multiplied, the values likewise.  Then
// the wavefronts' sums meet in LDS, in order, and those of the parts in
// attn_join_kernel.
#include "kv_attn.h"

namespace tern {
namespace {

constexpr int kWaves = 4;

template <int D, int NT>
__global__ __launch_bounds__(64 * kWaves, NT <= 2 && D <= 128 ? 2 : 1) void attn_rows_kernel(const AttnArgs a) {
  constexpr int C = D / 64, DT = D / 16;
  constexpr int P = D + 4;  // pitch of a row in LDS: rows fall in other banks
  __shared__ float sums[kWaves * 16 * P];
  __shared__ float tops[kWaves][16 * NT], totals[kWaves][16 * NT];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, kq = lane >> 4;
  const int part = blockIdx.x % a.parts, head = blockIdx.x / a.parts % a.c.heads;
  const int s = blockIdx.x / a.parts / a.c.heads;
  const Span sp = span_of(a.b, s);
  const int total = sp.n * a.group;
  if (total <= 0) return;
  const Range all = range_of_rows(a, sp, 0, total - 1);
  const Parts parts = parts_of(a, all);
  if (part >= parts.count) return;
  const Range mine = part_of(all, parts, part);

  // rows of the operand: j * group + h
  kh8_t q[NT][C][2];
  Sees sees[NT];
  int low = 0, high = 0x7fffffff;  // tokens that every row sees
  Row row[NT];
  kf4_t o[NT][DT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = n * 16 + col, j = r / a.group, h = r % a.group;
    const bool there = r < total;
    sees[n] = sees_of(a, sp, sp.from + j, there);
    if (there) {
      low = max(low, sees[n].low);
      high = min(high, sees[n].high);
    }
    const uint16_t* const from = a.q + (int64_t)(sp.first + j) * a.q_stride + (head * a.group + h) * D;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        q[n][c][u] = kh8_t{0, 0, 0, 0, 0, 0, 0, 0};
        if (there) q[n][c][u] = *reinterpret_cast<const kh8_t*>(from + 64 * c + 16 * kq + 8 * u);
      }
    row[n] = {-INFINITY, 0.f, 0.f};
#pragma unroll
    for (int d = 0; d < DT; ++d) o[n][d] = kf4_t{0.f, 0.f, 0.f, 0.f};
  }
  for (int i = 1; i < 16; i <<= 1) {
    low = max(low, __shfl_xor(low, i));
    high = min(high, __shfl_xor(high, i));
  }
  low = __builtin_amdgcn_readfirstlane(low);
  high = __builtin_amdgcn_readfirstlane(high);

  kw4_t kr[C][4], vr[DT];
  // a page that is not there reads as zeros, and is masked
  auto page_at = [&](int p) { return p < mine.end ? __builtin_amdgcn_readfirstlane(page_of(a.b, a.c, s, p)) : -1; };
  auto load_keys = [&](int id) {
    const __amdgpu_buffer_rsrc_t from = kv_buffer(a.c.k + ((size_t)max(id, 0) * a.c.heads + head) * (kPage * D), id < 0 ? 0 : kPage * D);
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int t = 0; t < 4; ++t) kr[c][t] = kv_load16(from, ((4 * c + t) * 64 + lane) * 16);
  };
  auto load_values = [&](int id) {
    const __amdgpu_buffer_rsrc_t from = kv_buffer(a.c.v + ((size_t)max(id, 0) * a.c.heads + head) * (kPage * D), id < 0 ? 0 : kPage * D);
#pragma unroll
    for (int d = 0; d < DT; ++d) vr[d] = kv_load16(from, (d * 64 + lane) * 16);
  };

  // Page numbers are read two pages ahead, scales one: their use never waits.
  auto scale_at = [&](const float* scales, int id) { return scales[(size_t)max(id, 0) * a.c.heads + head]; };
  int p = mine.begin + wave;
  int id = page_at(p), next = page_at(p + kWaves);
  float ks_next = 0.f, vs_next = 0.f;
  if (p < mine.end) {
    load_keys(id);
    load_values(id);
    ks_next = scale_at(a.c.ks, id);
    vs_next = scale_at(a.c.vs, id);
  }
  for (; p < mine.end; p += kWaves) {
    const int later = page_at(p + 2 * kWaves);
    const float ks = ks_next * a.scale, vs = vs_next;
    ks_next = scale_at(a.c.ks, next);
    vs_next = scale_at(a.c.vs, next);
    kf4_t z[NT][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int n = 0; n < NT; ++n) z[n][t] = kf4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const kh8_t k = codes8(kr[c][t][2 * u], kr[c][t][2 * u + 1]);
#pragma unroll
          for (int n = 0; n < NT; ++n) z[n][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, q[n][c][u], z[n][t], 0, 0, 0);
        }
    }
    load_keys(next);
    const bool whole = id >= 0 && p * kPage >= low && p * kPage + kPage <= high;
    kh8_t w[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float best = -INFINITY;
#pragma unroll
      for (int t = 0; t < 4; ++t) z[n][t] *= ks;
      if (!whole) {
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const int token = p * kPage + 16 * kq + x;
          if (id < 0 || token < sees[n].low || token >= sees[n].high) z[n][x / 4][x % 4] = -INFINITY;
        }
      }
#pragma unroll
      for (int x = 0; x < 16; ++x) best = fmaxf(best, z[n][x / 4][x % 4]);
      best = fmaxf(best, __shfl_xor(best, 16));
      best = fmaxf(best, __shfl_xor(best, 32));
      float ratio;
      const float factor = step_row(row[n], best, vs, &ratio);
      if (__any(factor != 1.0f)) {
#pragma unroll
        for (int d = 0; d < DT; ++d) o[n][d] *= factor;
      }
      const float top = row[n].top == -INFINITY ? 0.f : row[n].top;
      float sum = 0.f;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float e = __builtin_amdgcn_exp2f(z[n][t][i] - top);
          sum += e;
          w[n][t / 2][t % 2 * 4 + i] = (_Float16)(e * ratio);
        }
      row[n].sum += sum;
    }
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const kh8_t v = codes8(vr[d][2 * u], vr[d][2 * u + 1]);
#pragma unroll
        for (int n = 0; n < NT; ++n) o[n][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, w[n][u], o[n][d], 0, 0, 0);
      }
    load_values(next);
    id = next;
    next = later;
  }

  // The wavefronts' sums: references first, then 16 rows at a time.
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float sum = row[n].sum;
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    row[n].sum = sum;
    if (kq == 0) {
      tops[wave][n * 16 + col] = row[n].top;
      totals[wave][n * 16 + col] = sum;
    }
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    if (n * 16 >= total) break;
    float top = tops[0][n * 16 + col];
    for (int i = 1; i < kWaves; ++i) top = fmaxf(top, tops[i][n * 16 + col]);
    const float own = row[n].top == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(row[n].top - top) * (row[n].unit / kLift);
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      const kf4_t v = o[n][d] * own;
      *reinterpret_cast<kf4_t*>(&sums[(wave * 16 + col) * P + d * 16 + 4 * kq]) = v;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * D / 4; i += 64 * kWaves) {
      const int c = i / (D / 4), d = i % (D / 4) * 4, r = n * 16 + c;
      if (r >= total) break;
      kf4_t v = *reinterpret_cast<const kf4_t*>(&sums[c * P + d]);
      float best = tops[0][r], sum = 0.f;
      for (int x = 1; x < kWaves; ++x) {
        v += *reinterpret_cast<const kf4_t*>(&sums[(x * 16 + c) * P + d]);
        best = fmaxf(best, tops[x][r]);
      }
      for (int x = 0; x < kWaves; ++x)
        sum += tops[x][r] == -INFINITY ? totals[x][r] : totals[x][r] * __builtin_amdgcn_exp2f(tops[x][r] - best);
      const size_t out = (size_t)(sp.first + r / a.group) * a.q_heads + head * a.group + r % a.group;
      store_row<D>(a, parts, part, out, d, v, best, sum);
    }
    __syncthreads();
  }
}

// y from the parts' sums, in their order: a workgroup has a row's head, its
// groups of lanes take turns at the parts.
template <int D>
__global__ __launch_bounds__(256) void attn_join_kernel(const AttnArgs a, int block_rows) {
  constexpr int L = D / 4, G = 256 / L;  // lanes of a row, groups
  __shared__ kf4_t sums[256];
  __shared__ float totals[G];
  const Span sp = span_of(a.b, blockIdx.x / a.b.max_rows);
  const int j = blockIdx.x % a.b.max_rows, head = blockIdx.y;
  if (j >= sp.n) return;
  const int block = (j * a.group + head % a.group) / block_rows * block_rows;
  const Parts p = parts_of(a, range_of_rows(a, sp, block, min(block + block_rows, sp.n * a.group) - 1));
  if (p.count == 1) return;  // written where it was computed
  const int lane = threadIdx.x & 63, g = threadIdx.x / L, d = threadIdx.x % L * 4;
  const size_t rows = (size_t)a.b.rows * a.q_heads, r = (size_t)(sp.first + j) * a.q_heads + head;
  const kw2_t* const tops = reinterpret_cast<const kw2_t*>(a.part + (size_t)a.parts * rows * D) + r;
  float top = -INFINITY;
  for (int i = lane; i < p.count; i += 64) top = fmaxf(top, __uint_as_float(tops[i * rows].x));
  for (int o = 32; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
  kf4_t v = {0.f, 0.f, 0.f, 0.f};
  float sum = 0.f;
#pragma unroll 4
  for (int i = g; i < p.count; i += G) {
    const kw2_t t = tops[i * rows];
    const float at = __uint_as_float(t.x), f = at == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(at - top);
    sum += __uint_as_float(t.y) * f;
    v += *reinterpret_cast<const kf4_t*>(a.part + (i * rows + r) * D + d) * f;
  }
  sums[threadIdx.x] = v;
  if (threadIdx.x % L == 0) totals[g] = sum;
  __syncthreads();
  if (threadIdx.x >= L) return;
  for (int i = 1; i < G; ++i) {
    v += sums[i * L + threadIdx.x];
    sum += totals[i];
  }
  finish_row(a, r * D + d, v, sum);
}

template <int D>
hipError_t rows(const AttnArgs& a, int blocks, long long grid, hipStream_t s) {
  if (blocks == 1)
    hipLaunchKernelGGL((attn_rows_kernel<D, 1>), dim3((unsigned)grid), dim3(64 * kWaves), 0, s, a);
  else if (blocks == 2)
    hipLaunchKernelGGL((attn_rows_kernel<D, 2>), dim3((unsigned)grid), dim3(64 * kWaves), 0, s, a);
  else if constexpr (D <= 128)
    hipLaunchKernelGGL((attn_rows_kernel<D, 4>), dim3((unsigned)grid), dim3(64 * kWaves), 0, s, a);
  return hipGetLastError();
}

template <int D>
hipError_t join(const AttnArgs& a, int block_rows, hipStream_t s) {
  const long long x = (long long)a.b.count * a.b.max_rows;
  if (a.q_heads > 65535 || !kv_grid_fits(x * a.q_heads, 256)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((attn_join_kernel<D>), dim3((unsigned)x, (unsigned)a.q_heads), dim3(256), 0, s, a, block_rows);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_rows(const AttnArgs& a, int dim, int blocks, hipStream_t s) {
  const long long grid = (long long)a.b.count * a.c.heads * a.parts;
  if (!kv_grid_fits(grid, 64 * kWaves)) return hipErrorInvalidConfiguration;
  if (dim == 64) return rows<64>(a, blocks, grid, s);
  return dim == 128 ? rows<128>(a, blocks, grid, s) : rows<256>(a, blocks, grid, s);
}

hipError_t launch_attn_join(const AttnArgs& a, int dim, int block_rows, hipStream_t s) {
  if (dim == 64) return join<64>(a, block_rows, s);
  return dim == 128 ? join<128>(a, block_rows, s) : join<256>(a, block_rows, s);
}

}  // namespace tern
