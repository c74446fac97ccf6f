// Products with 4-bit weights for many activation rows, and the routed
// experts' products: y[m][n] = sum_g s[n][g] sum_{k in g} (q - z) x.
//
// A workgroup of four wavefronts (2 x 2) owns a 128 x 128 output tile and
// walks K in steps of 128, the next step's activations (32 KiB) and codes (8
// KiB) loaded straight into the other half of LDS meanwhile; 16-byte chunks
// are XOR-swizzled by row, so that the 32 rows of an operand read fall in
// distinct banks.  Only codes are staged, never decoded weights: a wavefront
// decodes its 64 weight rows in registers and feeds
// v_mfma_f32_32x32x16_f16 as the B operand.  Its 64 x 64 part keeps one FP32
// sum of the current group, which is scaled and added to the running FP32
// sum when the group ends (64 FMAs per lane against 1,024 matrix cycles at
// group 128).  Workgroups of one XCD take consecutive tiles, so that its L2
// reads each weight once.
#include "q4_rows.h"

namespace tern {
namespace {

constexpr int BM = 128, BN = 128, BK = 128;
constexpr int kXcds = 8;

template <int G, bool Z, int MODE>
__global__ __launch_bounds__(256, 2) void q4_tile_kernel(const Q4Args a) {
  constexpr bool up = MODE == kQ4Up;
  constexpr int NS = BK / G, SPG = G / 16;  // groups in a step, instructions (16 k) in a group
  // separate arrays: the compiler then knows that reading one does not wait
  // for loads into the other
  __shared__ w4_t xs0[BM * 16], xs1[BM * 16], cs0[BN * 4], cs1[BN * 4];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int c32 = lane & 31, kq = lane >> 5;
  const int k = a.k, ng = k / G;
  const int width = up ? a.n / 2 : a.n, cols = up ? BN / 2 : BN;
  const int tn = (width + cols - 1) / cols;

  // this workgroup's tile: XCD i (blockIdx % 8) has the i-th eighth of them
  const int tm = MODE == kQ4Plain ? (a.m + BM - 1) / BM : *a.ntiles;
  const int total = tn * tm * (MODE == kQ4Plain ? a.splits : 1), per = (total + kXcds - 1) / kXcds;
  int bid = blockIdx.x % kXcds * per + blockIdx.x / kXcds;
  if ((int)(blockIdx.x / kXcds) >= per || bid >= total) return;
  int e = 0, pos, rows, n0, t0 = 0, t1 = (k + BK - 1) / BK, split = 0;
  if (MODE == kQ4Plain) {
    pos = bid % tm * BM;
    bid /= tm;
    split = bid % a.splits;
    n0 = bid / a.splits * cols;
    rows = min(a.m - pos, BM);
    t0 = split * a.tps;
    t1 = min(t1, t0 + a.tps);
  } else {
    const int4 tile = a.tiles[bid / tn];
    n0 = bid % tn * cols;
    e = tile.x;
    pos = tile.y;
    rows = tile.z;
  }

  // Staging: wavefront w loads rows 32 w + 4 j + (lane >> 4), j < 8, of x and
  // rows 32 w + 16 j + (lane >> 2), j < 2, of the codes (a wavefront pair's 64
  // columns are two blocks of 32; up: 32 of the gate, 32 of the up projection).
  const uint8_t *xr[8], *cr[2];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int row = min(wave * 32 + j * 4 + (lane >> 4), rows - 1);
    size_t src = (size_t)pos + row;
    if (MODE == kQ4Up) src = (size_t)(a.slots[pos + row] / a.topk);
    xr[j] = reinterpret_cast<const uint8_t*>(a.x + src * k);
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int lr = wave * 32 + j * 16 + (lane >> 2);
    const int col = up ? min(n0 + lr / 64 * 32 + lr % 32, width - 1) + lr % 64 / 32 * width : min(n0 + lr, width - 1);
    cr[j] = a.codes + ((size_t)e * a.n + col) * (size_t)(k / 2);
  }
  const uint16_t* sr[2];
  const uint8_t* zr[2];
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int col = up ? min(n0 + wn * 32 + c32, width - 1) + b * width : min(n0 + wn * 64 + b * 32 + c32, width - 1);
    const size_t row = (size_t)e * a.n + col;
    sr[b] = a.scale + row * ng;
    zr[b] = Z ? a.zero + row * ng : nullptr;
  }
  // Scales (zero points) four groups at a time where rows start on multiples
  // of four, one step's otherwise.
  const bool vec = ng % 4 == 0 && !((uintptr_t)a.scale & 7) && (!Z || !((uintptr_t)a.zero & 3));
  w2_t sv[2], sn[2];
  uint32_t zv[2], zn[2];

  auto issue = [&](int t, w4_t* xd, w4_t* cd) {
    const int g0 = t * NS;
    if (vec) {
      if (t == t0 || g0 % 4 == 0) {
        const int g = g0 / 4 * 4;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          sn[b] = *reinterpret_cast<const w2_t*>(sr[b] + g);
          if (Z) zn[b] = *reinterpret_cast<const uint32_t*>(zr[b] + g);
        }
      }
    } else {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        uint32_t s[4] = {0, 0, 0, 0}, z = 0;
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          const int g = min(g0 + j, ng - 1);
          s[j] = sr[b][g];
          if (Z) z |= (uint32_t)zr[b][g] << (8 * j);
        }
        sn[b] = w2_t{s[0] | s[1] << 16, s[2] | s[3] << 16};
        zn[b] = z;
      }
    }
    const bool full = G == 128 || t * BK + BK <= k;  // chunks behind k: any that exist, not multiplied
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int lr = wave * 32 + j * 4 + (lane >> 4);
      int c = (lane ^ lr) & 15;
      if (!full && t * BK + c * 8 >= k) c = 0;
      __builtin_amdgcn_global_load_lds(xr[j] + (size_t)t * 256 + c * 16,
                                       (__attribute__((address_space(3))) void*)(xd + (wave * 8 + j) * 64), 16, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      int c = code_chunk(wave * 32 + j * 16 + (lane >> 2), lane & 3) & 3;
      if (!full && t * BK + c * 32 >= k) c = 0;
      __builtin_amdgcn_global_load_lds(cr[j] + (size_t)t * 64 + c * 16,
                                       (__attribute__((address_space(3))) void*)(cd + (wave * 2 + j) * 64), 16, 0, 0);
    }
  };

  const Q4Masks masks;
  a16_t acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][b][v] = 0.f;

  // one step; the loads of the next are in flight
  auto compute = [&](int t, const w4_t* xd, const w4_t* cd) {
    const int left = min(NS, ng - t * NS);  // groups in this step
    const int at = vec ? t * NS % 4 : 0;
    w4_t w[2];
    a16_t sum[2][2];
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      if (j && j >= left) break;
      float sc[2];
      Q4Bias bias[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        sc[b] = half_bits((uint16_t)((at + j < 2 ? sv[b].x : sv[b].y) >> (16 * ((at + j) & 1))));
        bias[b] = q4_bias(Z ? (zv[b] >> (8 * (at + j))) & 255u : 8u);
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int v = 0; v < 16; ++v) sum[x][b][v] = 0.f;
      }
#pragma unroll
      for (int q = 0; q < SPG; ++q) {
        const int step = j * SPG + q, c = step / 4, i = step % 4;  // 64 k chunk, instruction in it
        if (i == 0) {
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            w[b] = cd[code_chunk(wn * 64 + b * 32 + c32, c * 2 + kq)];
            if (G == 32) {  // words in k order: both lane halves inside one group
              const auto p = __builtin_amdgcn_permlane32_swap(w[b].x, w[b].y, false, false);
              const auto o = __builtin_amdgcn_permlane32_swap(w[b].z, w[b].w, false, false);
              w[b] = w4_t{p[0], o[0], p[1], o[1]};
            }
          }
        }
        const int chunk = G == 32 ? c * 8 + i * 2 + kq : c * 8 + kq * 4 + i;
        h8_t xa[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int row = wm * 64 + x * 32 + c32;
          xa[x] = __builtin_bit_cast(h8_t, xd[row * 16 + ((chunk ^ row) & 15)]);
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const h8_t wv = q4_decode(w[b][i], bias[b], masks);
#pragma unroll
          for (int x = 0; x < 2; ++x) sum[x][b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(xa[x], wv, sum[x][b], 0, 0, 0);
        }
      }
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int v = 0; v < 16; ++v) acc[x][b][v] += sc[b] * sum[x][b][v];
    }
  };
  auto arrive = [&](int t) {
    q4_loads_done();
    if (!vec || t == t0 || t * NS % 4 == 0) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        sv[b] = sn[b];
        zv[b] = zn[b];
      }
    }
    __syncthreads();
  };

  if (t0 < t1) issue(t0, xs0, cs0);
  for (int t = t0; t < t1; t += 2) {
    arrive(t);
    if (t + 1 < t1) issue(t + 1, xs1, cs1);
    compute(t, xs0, cs0);
    if (t + 1 >= t1) break;
    arrive(t + 1);
    if (t + 2 < t1) issue(t + 2, xs0, cs0);
    compute(t + 1, xs1, cs1);
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
  const long long grid = (tn * tm + kXcds - 1) / kXcds * kXcds;
  if (grid > 0x7fffffffll) return hipErrorInvalidValue;
  hipLaunchKernelGGL((q4_tile_kernel<G, Z, MODE>), dim3((unsigned)grid), dim3(256), 0, s, a);
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
