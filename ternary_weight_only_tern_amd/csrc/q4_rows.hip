// Products with 4-bit weights for few activation rows (up to 64; the routed
// experts' 16-row tiles): y[m][n] = sum_g s[n][g] sum_{k in g} (q - z) x.
//
// A workgroup owns 16 weight rows (a panel, contiguous in memory; NB panels)
// and its wavefronts share the panel's K: wavefront w takes the 128-wide K
// tiles w, w + W, ...  A lane loads 16 bytes of one row (32 codes), decodes
// them to FP16 and feeds four v_mfma_f32_16x16x32_f16 with the activations
// as A (16 rows) and the weights as B (16 columns); a group's sum, FP32, is
// scaled and added to the running FP32 sum.  At group 128 the four lanes
// that hold one row's tile multiply 32 consecutive k each.  Smaller groups
// need every instruction's 32 k inside one group, so the four lanes' words
// are transposed first (v_permlane32_swap, v_permlane16_swap: four
// operations per 16 bytes).  The wavefronts' sums are added in LDS in
// wavefront order: results do not depend on timing.
//
// At one row the bound is the reading of the codes from memory.
#include "q4.h"

namespace tern {
namespace {

template <int G, int MT, int NB>
struct Frag {
  w4_t c[NB];
  uint16_t s[NB][128 / G];
  uint8_t z[NB][128 / G];
  h8_t x[MT][4];
};

// The rows a lane reads: weight rows (clamped into the matrix) and
// activation rows (NULL: none, counted as zeros).
template <int MT, int NB>
struct Rows {
  const uint8_t* c[NB];
  const uint16_t* s[NB];
  const uint8_t* z[NB];
  const uint16_t* x[MT];
};

template <int G, int MT, int NB, bool Z>
__device__ inline void load_tile(Frag<G, MT, NB>& f, const Rows<MT, NB>& r, int t, int k, int kq) {
  constexpr int SG = 128 / G;
  const int ng = k / G;
  const bool in = t * 128 + kq * 32 < k;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    f.c[b] = w4_t{0, 0, 0, 0};
    if (in) f.c[b] = *reinterpret_cast<const w4_t*>(r.c[b] + (size_t)t * 64 + kq * 16);
#pragma unroll
    for (int j = 0; j < SG; ++j) {
      const int g = min(t * SG + j, ng - 1);  // a tile past the end of K has zero activations there
      f.s[b][j] = r.s[b][g];
      f.z[b][j] = Z ? r.z[b][g] : (uint8_t)8;
    }
  }
#pragma unroll
  for (int a = 0; a < MT; ++a)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int kx = t * 128 + (G == 128 ? kq * 32 + i * 8 : i * 32 + kq * 8);
      f.x[a][i] = h8_t{};
      if (r.x[a] != nullptr && kx < k) f.x[a][i] = *reinterpret_cast<const h8_t*>(r.x[a] + kx);
    }
}

template <int G, int MT, int NB, bool Z>
__device__ inline void multiply_tile(const Frag<G, MT, NB>& f, float mul, f4_t (&acc)[MT][NB]) {
  constexpr int SG = 128 / G;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    uint32_t w[4] = {f.c[b].x, f.c[b].y, f.c[b].z, f.c[b].w};
    if (G < 128) {  // word i of lane quarter q <- word q of lane quarter i
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const auto p = __builtin_amdgcn_permlane32_swap(w[i], w[i + 2], false, false);
        w[i] = p[0];
        w[i + 2] = p[1];
      }
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const auto p = __builtin_amdgcn_permlane16_swap(w[i], w[i + 1], false, false);
        w[i] = p[0];
        w[i + 1] = p[1];
      }
    }
#pragma unroll
    for (int j = 0; j < SG; ++j) {
      const Q4Bias bias = q4_bias(Z ? f.z[b][j] : 8);
      f4_t sum[MT];
#pragma unroll
      for (int a = 0; a < MT; ++a) sum[a] = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 4 / SG; ++i) {
        const h8_t wv = q4_decode(w[j * (4 / SG) + i], bias);
#pragma unroll
        for (int a = 0; a < MT; ++a)
          sum[a] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f.x[a][j * (4 / SG) + i], wv, sum[a], 0, 0, 0);
      }
      const float s = half_bits(f.s[b][j]) * mul;
#pragma unroll
      for (int a = 0; a < MT; ++a) acc[a][b] += s * sum[a];
    }
  }
}

template <int G, int MT, int NB, bool Z, int W, int MODE>
__global__ __launch_bounds__(W * 64) void q4_rows_kernel(const Q4Args a) {
  __shared__ float red[W][MT * NB][4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, kq = lane >> 4;
  const int k = a.k, ng = k / G, T = (k + 127) / 128;
  constexpr bool up = MODE == kQ4Up || MODE == kQ4UpSlot;
  const int width = up ? a.n / 2 : a.n;  // output columns
  const int n0 = blockIdx.x * 16 * (up ? 1 : NB);

  int e = 0, rows = a.m, pos = 0;
  if (MODE == kQ4Up || MODE == kQ4Down) {
    if ((int)blockIdx.y >= *a.ntiles) return;
    const int4 tile = a.tiles[blockIdx.y];
    e = tile.x;
    pos = tile.y;
    rows = tile.z;
  } else if (MODE == kQ4UpSlot) {
    e = a.ids[blockIdx.y];
    if ((unsigned)e >= (unsigned)a.experts) return;
    pos = blockIdx.y;
    rows = 1;
  } else if (MODE == kQ4Plain) {
    pos = blockIdx.y * 16 * MT;
    rows = min(rows - pos, 16 * MT);
  } else {
    pos = blockIdx.y;
    rows = 1;
  }

  Rows<MT, NB> at;
  auto weights = [&](int expert) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int col = min(n0 + (up ? 0 : b * 16) + r, width - 1) + (up && b ? width : 0);
      const size_t row = (size_t)expert * a.n + col;
      at.c[b] = a.codes + row * (size_t)(k / 2);
      at.s[b] = a.scale + row * ng;
      at.z[b] = Z ? a.zero + row * ng : nullptr;
    }
  };
  f4_t acc[MT][NB];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[i][b] = f4_t{0.f, 0.f, 0.f, 0.f};

  if (MODE == kQ4DownToken) {
    // the token's slots one after another along the wavefronts' K tiles
    for (int u = wave; u < a.topk * T; u += W) {
      const int j = u / T, t = u - j * T;
      const int slot = pos * a.topk + j;
      const int ex = a.ids[slot];
      if ((unsigned)ex >= (unsigned)a.experts) continue;
      weights(ex);
      at.x[0] = r == 0 ? a.x + (size_t)slot * k : nullptr;
      Frag<G, MT, NB> f;
      load_tile<G, MT, NB, Z>(f, at, t, k, kq);
      multiply_tile<G, MT, NB, Z>(f, a.gates[slot], acc);
    }
  } else {
    weights(e);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int row = i * 16 + r;
      at.x[i] = nullptr;
      if (row < rows) {
        size_t src = (size_t)pos + row;
        if (MODE == kQ4Up) src = (size_t)(a.slots[pos + row] / a.topk);
        if (MODE == kQ4UpSlot) src = (size_t)(pos / a.topk);
        at.x[i] = a.x + src * k;
      }
    }
    Frag<G, MT, NB> f, next;
    if (wave < T) load_tile<G, MT, NB, Z>(f, at, wave, k, kq);
    for (int t = wave; t < T; t += W) {
      if (t + W < T) load_tile<G, MT, NB, Z>(next, at, t + W, k, kq);
      multiply_tile<G, MT, NB, Z>(f, 1.0f, acc);
      f = next;
    }
  }

#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int v = 0; v < 4; ++v) red[wave][i * NB + b][v][lane] = acc[i][b][v];
  __syncthreads();
  constexpr int OUT = MT * (up ? 1 : NB) * 256;
  for (int o = threadIdx.x; o < OUT; o += W * 64) {
    const int l = o & 63, v = (o >> 6) & 3, tile = o >> 8;
    const int i = up ? tile : tile / NB, b = up ? 0 : tile % NB;
    const int row = i * 16 + (l >> 4) * 4 + v, col = n0 + b * 16 + (l & 15);
    float sum = 0.f, gate = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (up) {
        gate += red[w][i * NB][v][l];
        sum += red[w][i * NB + NB - 1][v][l];
      } else {
        sum += red[w][tile][v][l];
      }
    }
    if (row >= rows || col >= width) continue;
    const size_t dst = ((size_t)pos + row) * width + col;
    if (up)
      reinterpret_cast<_Float16*>(a.y)[dst] = (_Float16)q4_swiglu(gate, sum);
    else if (MODE == kQ4Down || a.y_f32)
      reinterpret_cast<float*>(a.y)[dst] = sum;
    else
      reinterpret_cast<_Float16*>(a.y)[dst] = (_Float16)sum;
  }
}

template <int G, int MT, int NB, bool Z, int W, int MODE>
hipError_t launch(const Q4Args& a, int tiles, hipStream_t s) {
  constexpr bool up = MODE == kQ4Up || MODE == kQ4UpSlot;
  const int width = up ? a.n / 2 : a.n;
  const int cols = 16 * (up ? 1 : NB);
  const int gy = MODE == kQ4Plain ? (a.m + 16 * MT - 1) / (16 * MT) : tiles;
  const dim3 grid((unsigned)((width + cols - 1) / cols), (unsigned)gy);
  hipLaunchKernelGGL((q4_rows_kernel<G, MT, NB, Z, W, MODE>), grid, dim3(W * 64), 0, s, a);
  return hipGetLastError();
}

template <int G, bool Z>
hipError_t pick(int mode, const Q4Args& a, int tiles, hipStream_t s) {
  switch (mode) {
    case kQ4Up: return launch<G, 1, 2, Z, 8, kQ4Up>(a, tiles, s);
    case kQ4Down: return launch<G, 1, 1, Z, 8, kQ4Down>(a, tiles, s);
    case kQ4UpSlot: return launch<G, 1, 2, Z, 8, kQ4UpSlot>(a, tiles, s);
    case kQ4DownToken: return launch<G, 1, 1, Z, 8, kQ4DownToken>(a, tiles, s);
    default: break;
  }
  if (a.m <= 16) return launch<G, 1, 1, Z, 8, kQ4Plain>(a, tiles, s);
  if (a.m <= 32) return launch<G, 2, 1, Z, 8, kQ4Plain>(a, tiles, s);
  return launch<G, 4, 1, Z, 4, kQ4Plain>(a, tiles, s);
}

}  // namespace

hipError_t launch_q4_rows(int mode, int group, const Q4Args& a, int tiles, hipStream_t s) {
  const bool z = a.zero != nullptr;
  switch (group) {
    case 32: return z ? pick<32, true>(mode, a, tiles, s) : pick<32, false>(mode, a, tiles, s);
    case 64: return z ? pick<64, true>(mode, a, tiles, s) : pick<64, false>(mode, a, tiles, s);
    default: return z ? pick<128, true>(mode, a, tiles, s) : pick<128, false>(mode, a, tiles, s);
  }
}

}  // namespace tern
