// Products with 4-bit weights for many activation rows, and the routed
// experts' products: y[m][n] = sum_g s[n][g] sum_{k in g} (q - z) x.
//
// A workgroup of four wavefronts (2 x 2) owns a 128 x 128 output tile and
// walks K in steps of 128.  The activations' 128 x 128 FP16 step is staged in
// LDS (16-byte chunks XOR-swizzled by row, so that the 32 rows of an operand
// read fall in distinct banks); the weights never pass through LDS: a lane
// loads 16 bytes of one row's codes, decodes them in registers and feeds
// v_mfma_f32_32x32x16_f16 as the B operand (32 weight rows).  Each
// wavefront's 64 x 64 part keeps one FP32 sum of the current group, which is
// scaled and added to the running FP32 sum when the group ends: 64 FMAs per
// lane against 1,024 matrix cycles at group 128.
#include "q4.h"

namespace tern {
namespace {

constexpr int BM = 128, BN = 128, BK = 128;

template <int G, bool Z, int MODE>
__global__ __launch_bounds__(256, 2) void q4_tile_kernel(const Q4Args a) {
  __shared__ h8_t xs[BM * BK / 8];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1;
  const int c32 = lane & 31, kq = lane >> 5;
  const int k = a.k, ng = k / G;
  constexpr bool up = MODE == kQ4Up;
  const int width = up ? a.n / 2 : a.n;
  const int cols = up ? BN / 2 : BN;
  const int tn = (width + cols - 1) / cols;

  int bid = blockIdx.x;
  const int n0 = bid % tn * cols;
  bid /= tn;
  int e = 0, pos, rows, t0 = 0, t1 = (k + BK - 1) / BK, split = 0;
  if (MODE == kQ4Plain) {
    split = bid % a.splits;
    pos = bid / a.splits * BM;
    rows = min(a.m - pos, BM);
    t0 = split * a.tps;
    t1 = min(t1, t0 + a.tps);
  } else {
    if (bid >= *a.ntiles) return;
    const int4 tile = a.tiles[bid];
    e = tile.x;
    pos = tile.y;
    rows = tile.z;
  }

  // activation rows this thread stages: (tid >> 4) + 16 j, chunk tid & 15
  const int sc = tid & 15;
  const uint16_t* xr[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int row = min((tid >> 4) + 16 * j, rows - 1);
    size_t src = (size_t)pos + row;
    if (MODE == kQ4Up) src = (size_t)(a.slots[pos + row] / a.topk);
    xr[j] = a.x + src * k;
  }
  // weight rows of this lane
  const uint8_t* cr[2];
  const uint16_t* sr[2];
  const uint8_t* zr[2];
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int col = up ? min(n0 + wn * 32 + c32, width - 1) + b * width : min(n0 + wn * 64 + b * 32 + c32, width - 1);
    const size_t row = (size_t)e * a.n + col;
    cr[b] = a.codes + row * (size_t)(k / 2);
    sr[b] = a.scale + row * ng;
    zr[b] = Z ? a.zero + row * ng : nullptr;
  }

  h8_t xv[8];
  w4_t cv[2][2];
  auto load = [&](int t) {
    const int kx = t * BK + sc * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      xv[j] = h8_t{};
      if (kx < k) xv[j] = *reinterpret_cast<const h8_t*>(xr[j] + kx);
    }
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        cv[b][c] = w4_t{0, 0, 0, 0};
        if (t * BK + c * 64 + kq * 32 < k)
          cv[b][c] = *reinterpret_cast<const w4_t*>(cr[b] + (size_t)t * (BK / 2) + c * 32 + kq * 16);
      }
  };

  f16_t acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][b][v] = 0.f;

  constexpr int SPG = G / 16;  // instructions of 16 k per group
  if (t0 < t1) load(t0);
  for (int t = t0; t < t1; ++t) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int row = (tid >> 4) + 16 * j;
      xs[row * 16 + (sc ^ (row & 15))] = xv[j];
    }
    w4_t cw[2][2];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int c = 0; c < 2; ++c) cw[b][c] = cv[b][c];
    __syncthreads();
    if (t + 1 < t1) load(t + 1);
    f16_t sum[2][2];
    Q4Bias bias[2];
    float sc32[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t w[2][4];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        w[b][0] = cw[b][c].x;
        w[b][1] = cw[b][c].y;
        w[b][2] = cw[b][c].z;
        w[b][3] = cw[b][c].w;
        if (G == 32) {  // words in k order: both lane halves inside one group
          const auto p = __builtin_amdgcn_permlane32_swap(w[b][0], w[b][1], false, false);
          const auto q = __builtin_amdgcn_permlane32_swap(w[b][2], w[b][3], false, false);
          w[b][0] = p[0];
          w[b][1] = q[0];
          w[b][2] = p[1];
          w[b][3] = q[1];
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int step = c * 4 + i;
        if (step % SPG == 0) {
          const int g = min(t * (BK / G) + step / SPG, ng - 1);
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            sc32[b] = half_bits(sr[b][g]);
            bias[b] = q4_bias(Z ? zr[b][g] : 8);
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int v = 0; v < 16; ++v) sum[x][b][v] = 0.f;
          }
        }
        const int chunk = G == 32 ? c * 8 + i * 2 + kq : c * 8 + kq * 4 + i;
        h8_t xa[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int row = wm * 64 + x * 32 + c32;
          xa[x] = xs[row * 16 + (chunk ^ (row & 15))];
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const h8_t wv = q4_decode(w[b][i], bias[b]);
#pragma unroll
          for (int x = 0; x < 2; ++x) sum[x][b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(xa[x], wv, sum[x][b], 0, 0, 0);
        }
        if (step % SPG == SPG - 1) {
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int v = 0; v < 16; ++v) acc[x][b][v] += sc32[b] * sum[x][b][v];
        }
      }
    }
  }

#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int b = 0; b < (up ? 1 : 2); ++b)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int row = wm * 64 + x * 32 + 8 * (v / 4) + 4 * kq + v % 4;
        const int col = up ? n0 + wn * 32 + c32 : n0 + wn * 64 + b * 32 + c32;
        if (row >= rows || col >= width) continue;
        const size_t dst = ((size_t)pos + row) * width + col;
        if (up)
          reinterpret_cast<_Float16*>(a.y)[dst] = (_Float16)q4_swiglu(acc[x][0][v], acc[x][1][v]);
        else if (MODE == kQ4Plain && a.splits > 1)
          a.partial[(size_t)split * a.m * a.n + dst] = acc[x][b][v];
        else if (MODE == kQ4Down || a.y_f32)
          reinterpret_cast<float*>(a.y)[dst] = acc[x][b][v];
        else
          reinterpret_cast<_Float16*>(a.y)[dst] = (_Float16)acc[x][b][v];
      }
}

// y = the sum of the K parts' partials, in part order.
__global__ __launch_bounds__(256) void q4_reduce_kernel(const float* part, int splits, size_t count, void* y, int y_f32) {
  const size_t step = (size_t)gridDim.x * 256;
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < count; i += step) {
    float sum = 0.f;
    for (int s = 0; s < splits; ++s) sum += part[(size_t)s * count + i];
    if (y_f32)
      reinterpret_cast<float*>(y)[i] = sum;
    else
      reinterpret_cast<_Float16*>(y)[i] = (_Float16)sum;
  }
}

template <int G, bool Z, int MODE>
hipError_t launch(const Q4Args& a, int tiles, hipStream_t s) {
  const int width = MODE == kQ4Up ? a.n / 2 : a.n, cols = MODE == kQ4Up ? BN / 2 : BN;
  const long long tn = (width + cols - 1) / cols;
  const long long tm = MODE == kQ4Plain ? (long long)((a.m + BM - 1) / BM) * a.splits : tiles;
  if (tn * tm > 0x7fffffffll) return hipErrorInvalidValue;
  hipLaunchKernelGGL((q4_tile_kernel<G, Z, MODE>), dim3((unsigned)(tn * tm)), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <int G, bool Z>
hipError_t pick(int mode, const Q4Args& a, int tiles, hipStream_t s) {
  switch (mode) {
    case kQ4Up: return launch<G, Z, kQ4Up>(a, tiles, s);
    case kQ4Down: return launch<G, Z, kQ4Down>(a, tiles, s);
    default: return launch<G, Z, kQ4Plain>(a, tiles, s);
  }
}

}  // namespace

hipError_t launch_q4_tile(int mode, int group, const Q4Args& a, int tiles, hipStream_t s) {
  const bool z = a.zero != nullptr;
  switch (group) {
    case 32: return z ? pick<32, true>(mode, a, tiles, s) : pick<32, false>(mode, a, tiles, s);
    case 64: return z ? pick<64, true>(mode, a, tiles, s) : pick<64, false>(mode, a, tiles, s);
    default: return z ? pick<128, true>(mode, a, tiles, s) : pick<128, false>(mode, a, tiles, s);
  }
}

hipError_t launch_q4_reduce(const Q4Args& a, hipStream_t s) {
  const size_t count = (size_t)a.m * a.n;
  const size_t blocks = (count + 255) / 256;
  hipLaunchKernelGGL(q4_reduce_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, s, a.partial, a.splits,
                     count, a.y, a.y_f32);
  return hipGetLastError();
}

}  // namespace tern
