// Products with 4-bit weights for many activation rows, and the routed
// experts' products: y[m][n] = sum_g s[n][g] sum_{k in g} (q - z) x.
//
// A workgroup of WM x WN wavefronts owns an output tile and walks K in steps
// of 128, the next step's activations and codes loaded straight into the
// other half of LDS meanwhile; 16-byte chunks are XOR-swizzled by row, so
// that the 32 rows of an operand read fall in distinct banks.  Only codes are
// staged, never decoded weights: a wavefront decodes its weight rows in
// registers and feeds v_mfma_f32_32x32x16_f16 as the B operand (the experts'
// down products the BF16 form, once for each of an inner value's two parts: as
// many operations as the gate and up products, 226 against 251 us at 2048
// tokens, 8 of 64 experts of 2560 x 1024; with one part, in FP16, 128 us, but
// FP16's range and 11 bits).  It keeps one FP32 sum of the current group, which
// is scaled and added to the running FP32 sum when the group ends (at group 128
// one FMA per lane for every 16 matrix cycles).  Workgroups of one XCD take
// consecutive tiles, so that its L2 reads each weight once.
//
// Bound by the matrix and vector instructions together, and by what the power
// leaves of the clock: 512 x 12288 x 4096 62.8 us, 820 TFLOP/s (the library's
// FP16 product of that size 58-60 us); 8192 x 4096 x 4096 286 us, 960
// TFLOP/s.  Per 32 x 32 x 16 block the vector units decode eight codes a lane
// once for MW instructions: larger tiles decode less and fill fewer CUs.
#include "q4_rows.h"

namespace tern {
namespace {

constexpr int BK = 128;
constexpr int kXcds = 8;

// WM x WN wavefronts, MW x NW blocks of 32 x 32 each.
template <int G, bool Z, int MODE, int WM, int WN, int MW, int NW>
__global__ __launch_bounds__(WM * WN * 64) void q4_tile_kernel(const Q4Args a) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass drops the kernel's stub when it has to look at the LDS loads
  constexpr int BM = 32 * WM * MW, BN = 32 * WN * NW, WAVES = WM * WN;
  constexpr bool up = MODE == kQ4Up, inner = MODE == kQ4Down;
  constexpr int P = inner ? kInnerTile : 1;  // rows of x that make an operand's row
  constexpr int NS = BK / G, SPG = G / 16;  // groups in a step, instructions (16 k) in a group
  // Two steps' staging, in separate arrays: the compiler then knows that
  // reading one does not wait for loads into the other.  (A third step in
  // flight gained nothing: 2048 x 4096 x 4096 77.7 against 74.4 us.)
  __shared__ w4_t xs0[BM * P * 16], xs1[BM * P * 16], cs0[BN * 4], cs1[BN * 4];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
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

  // Staging: wavefront w loads rows 4 XJ w + 4 j + (lane >> 4) of x and rows
  // 16 CJ w + 16 j + (lane >> 2) of the codes.  Columns come in blocks of 32;
  // up: 16 of the gate, then the same 16 of the up projection.  Rows behind
  // the last lie past the buffers' ends.
  constexpr int XJ = BM * P / 4 / WAVES, CJ = BN / 16 / WAVES;
  static_assert(XJ > 0 && CJ > 0 && XJ * 4 * WAVES == BM * P && CJ * 16 * WAVES == BN, "every wavefront stages");
  // half blocks of 16 rows: first row, and how many exist
  auto half_row = [&](int h) {
    const int col = n0 + (up ? h / 2 : h) * 16;
    return (col < width ? col : 0) + (up ? h % 2 * width : 0);
  };
  auto half_rows = [&](int h) { return max(0, min(16, width - n0 - (up ? h / 2 : h) * 16)); };
  const size_t row_bytes = (size_t)k * 2;
  const __amdgpu_buffer_rsrc_t fx = MODE == kQ4Up ? q4_buffer(a.x, (uint32_t)(a.m * row_bytes))
                                                  : q4_buffer(a.x + (size_t)pos * P * k, (uint32_t)(rows * P * row_bytes));
  uint32_t xo[XJ];
#pragma unroll
  for (int j = 0; j < XJ; ++j) {
    const int row = wave * 4 * XJ + j * 4 + (lane >> 4);
    xo[j] = kFar;
    if (row < rows * P)
      xo[j] = (uint32_t)(MODE == kQ4Up ? a.slots[pos + row] / a.topk : row) * (uint32_t)row_bytes + ((lane ^ (row / P)) & 15) * 16;
  }
  __amdgpu_buffer_rsrc_t fc[CJ];
  uint32_t co[CJ];
#pragma unroll
  for (int j = 0; j < CJ; ++j) {
    const int h = wave * CJ + j, row = lane >> 2;
    fc[j] = q4_buffer(a.codes + ((size_t)e * a.n + half_row(h)) * (size_t)(k / 2), (uint32_t)half_rows(h) * (uint32_t)(k / 2));
    co[j] = (uint32_t)row * (uint32_t)(k / 2) + (code_chunk(row, lane & 3) & 3) * 16;
  }
  // Scales (zero points) four groups at a time where rows start on multiples
  // of four, one step's otherwise.
  const bool vec = ng % 4 == 0 && !((uintptr_t)a.scale & 7) && (!Z || !((uintptr_t)a.zero & 3));
  const __amdgpu_buffer_rsrc_t fs = q4_buffer(a.scale + (size_t)e * a.n * ng, (uint32_t)a.n * (uint32_t)ng * 2);
  const __amdgpu_buffer_rsrc_t fz = q4_buffer(Z ? a.zero + (size_t)e * a.n * ng : nullptr, (uint32_t)a.n * (uint32_t)ng);
  uint32_t so[NW];
#pragma unroll
  for (int b = 0; b < NW; ++b) {
    const int blk = wn * NW + b;
    const int col = up ? min(n0 + blk * 16 + c32 % 16, width - 1) + c32 / 16 * width : min(n0 + blk * 32 + c32, width - 1);
    so[b] = (uint32_t)col * (uint32_t)ng;
  }
  w2_t sv[NW], sn[NW];
  uint32_t zv[NW], zn[NW];

  auto load_scales = [&](int t) {
    const int g0 = t * NS;
    if (vec) {
      if (t == t0 || g0 % 4 == 0) {
#pragma unroll
        for (int b = 0; b < NW; ++b) {
          sn[b] = __builtin_bit_cast(w2_t, __builtin_amdgcn_raw_buffer_load_b64(fs, (so[b] + g0 / 4 * 4) * 2, 0, 0));
          if (Z) zn[b] = __builtin_amdgcn_raw_buffer_load_b32(fz, so[b] + g0 / 4 * 4, 0, 0);
        }
      }
    } else {
#pragma unroll
      for (int b = 0; b < NW; ++b) {
        uint32_t s[4] = {0, 0, 0, 0}, z = 0;
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          const uint32_t g = so[b] + min(g0 + j, ng - 1);
          s[j] = __builtin_amdgcn_raw_buffer_load_b16(fs, g * 2, 0, 0);
          if (Z) z |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(fz, g, 0, 0) << (8 * j);
        }
        sn[b] = w2_t{s[0] | s[1] << 16, s[2] | s[3] << 16};
        zn[b] = z;
      }
    }
  };
  // chunks behind k are the next row's, or nothing: they are not multiplied
  auto stage = [&](int t, w4_t* xd, w4_t* cd) {
#pragma unroll
    for (int j = 0; j < XJ; ++j) q4_stage16(fx, xd + (wave * XJ + j) * 64, xo[j] + (uint32_t)t * 256);
#pragma unroll
    for (int j = 0; j < CJ; ++j) q4_stage16(fc[j], cd + (wave * CJ + j) * 64, co[j] + (uint32_t)t * 64);
  };

  const Q4Masks masks;
  a16_t acc[MW][NW];
#pragma unroll
  for (int i = 0; i < MW; ++i)
#pragma unroll
    for (int b = 0; b < NW; ++b)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][b][v] = 0.f;

  // One step; the loads of the next are in flight.  An instruction's operands
  // of x are read one instruction ahead.
  auto compute = [&](int t, const w4_t* xd, const w4_t* cd) {
    const int left = min(NS, ng - t * NS);  // groups in this step
    const int at = vec ? t * NS % 4 : 0;
    w4_t w[2][NW];
    w4_t xa[2][P][MW];
    a16_t sum[MW][NW];
    auto read_x = [&](int step) {
      const int c = step / 4, i = step % 4;  // 64 k chunk, instruction in it
      const int chunk = G == 32 ? c * 8 + i * 2 + kq : c * 8 + kq * 4 + i;
#pragma unroll
      for (int x = 0; x < MW; ++x) {
        const int row = (wm * MW + x) * 32 + c32;
#pragma unroll
        for (int o = 0; o < P; ++o) xa[step % 2][o][x] = xd[(row * P + o) * 16 + ((chunk ^ row) & 15)];
      }
    };
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int b = 0; b < NW; ++b) w[c][b] = cd[code_chunk((wn * NW + b) * 32 + c32, c * 2 + kq)];
    read_x(0);
    if (G == 32) {  // words in k order: both lane halves inside one group
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int b = 0; b < NW; ++b) {
          const auto p = __builtin_amdgcn_permlane32_swap(w[c][b].x, w[c][b].y, false, false);
          const auto o = __builtin_amdgcn_permlane32_swap(w[c][b].z, w[c][b].w, false, false);
          w[c][b] = w4_t{p[0], o[0], p[1], o[1]};
        }
    }
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      if (j && j >= left) break;
      float sc[NW];
      Q4Bias bias[NW];
#pragma unroll
      for (int b = 0; b < NW; ++b) {
        sc[b] = half_bits((uint16_t)((at + j < 2 ? sv[b].x : sv[b].y) >> (16 * ((at + j) & 1)))) * (inner ? kInnerScale : 1.0f);
        bias[b] = q4_bias(Z ? (zv[b] >> (8 * (at + j))) & 255u : 8u);
#pragma unroll
        for (int x = 0; x < MW; ++x)
#pragma unroll
          for (int v = 0; v < 16; ++v) sum[x][b][v] = 0.f;
      }
#pragma unroll
      for (int q = 0; q < SPG; ++q) {
        const int step = j * SPG + q;
        if (step < 7) read_x(step + 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int b = 0; b < NW; ++b) {
          const w4_t wv = q4_weights<inner>(w[step / 4][b][step % 4], bias[b], masks);
#pragma unroll
          for (int o = 0; o < P; ++o)
#pragma unroll
            for (int x = 0; x < MW; ++x) sum[x][b] = q4_mfma32<inner>(xa[step % 2][o][x], wv, sum[x][b]);
        }
      }
#pragma unroll
      for (int b = 0; b < NW; ++b)
#pragma unroll
        for (int x = 0; x < MW; ++x)
#pragma unroll
          for (int v = 0; v < 16; ++v) acc[x][b][v] += sc[b] * sum[x][b][v];
    }
  };
  // Step t: its staged loads have arrived and everyone has read step t - 1;
  // then the loads of t + 1 go where that was.
  auto step = [&](int t, const w4_t* xd, const w4_t* cd, w4_t* xn, w4_t* cn) {
    q4_loads_done();
    if (!vec || t == t0 || t * NS % 4 == 0) {
#pragma unroll
      for (int b = 0; b < NW; ++b) {
        sv[b] = sn[b];
        zv[b] = zn[b];
      }
    }
    __syncthreads();
    if (t + 1 < t1) {
      load_scales(t + 1);
      stage(t + 1, xn, cn);
    }
    compute(t, xd, cd);
  };
  if (t0 < t1) {
    load_scales(t0);
    stage(t0, xs0, cs0);
  }
  for (int t = t0; t < t1; t += 2) {
    step(t, xs0, cs0, xs1, cs1);
    if (t + 1 >= t1) break;
    step(t + 1, xs1, cs1, xs0, cs0);
  }

#pragma unroll
  for (int x = 0; x < MW; ++x)
#pragma unroll
    for (int b = 0; b < NW; ++b)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int row = (wm * MW + x) * 32 + 8 * (v / 4) + 4 * kq + v % 4;
        const float value = acc[x][b][v];
        if (up) {  // the up projection's value is 16 lanes on
          const float other = __shfl_xor(value, 16);
          const int col = n0 + (wn * NW + b) * 16 + c32;
          if (c32 < 16 && row < rows && col < width)
            q4_store_inner<kInnerTile>(a.y, ((size_t)pos + row) * kInnerTile * width + col, width, q4_swiglu(value, other));
          continue;
        }
        const int col = n0 + (wn * NW + b) * 32 + c32;
        if (row >= rows || col >= width) continue;
        const size_t dst = ((size_t)pos + row) * width + col;
        if (MODE == kQ4Plain && a.splits > 1)
          a.partial[(size_t)split * a.m * a.n + dst] = value;
        else if (MODE == kQ4Down || a.y_f32)
          reinterpret_cast<float*>(a.y)[dst] = value;
        else
          reinterpret_cast<_Float16*>(a.y)[dst] = (_Float16)value;
      }
#endif
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

template <int G, bool Z, int MODE, int WM, int WN, int MW, int NW>
hipError_t launch(const Q4Args& a, int tiles, hipStream_t s) {
  constexpr int BM = 32 * WM * MW, BN = 32 * WN * NW;
  const int width = MODE == kQ4Up ? a.n / 2 : a.n, cols = MODE == kQ4Up ? BN / 2 : BN;
  const long long tn = (width + cols - 1) / cols;
  const long long tm = MODE == kQ4Plain ? (long long)((a.m + BM - 1) / BM) * a.splits : tiles;
  const long long grid = (tn * tm + kXcds - 1) / kXcds * kXcds;
  if (!grid_fits(grid, WM * WN * 64)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((q4_tile_kernel<G, Z, MODE, WM, WN, MW, NW>), dim3((unsigned)grid), dim3(WM * WN * 64), 0, s, a);
  return hipGetLastError();
}

template <int G, bool Z, int MODE>
hipError_t pick(const Q4Args& a, int tiles, int rows, hipStream_t s) {
  if constexpr (MODE == kQ4Plain) {
    if (rows == kQ4TileLarge) return launch<G, Z, MODE, 1, 8, 4, 1>(a, tiles, s);
    if (rows == kQ4TileMid) return launch<G, Z, MODE, 1, 8, 3, 1>(a, tiles, s);
  }
  if (rows == kQ4TileTiny) return launch<G, Z, MODE, 1, 4, 1, 1>(a, tiles, s);
  return launch<G, Z, MODE, 1, 4, 2, 1>(a, tiles, s);
}

template <int G, bool Z>
hipError_t pick_mode(int mode, const Q4Args& a, int tiles, int rows, hipStream_t s) {
  switch (mode) {
    case kQ4Up: return pick<G, Z, kQ4Up>(a, tiles, rows, s);
    case kQ4Down: return pick<G, Z, kQ4Down>(a, tiles, rows, s);
    default: return pick<G, Z, kQ4Plain>(a, tiles, rows, s);
  }
}

}  // namespace

hipError_t launch_q4_tile(int mode, int group, const Q4Args& a, int tiles, int rows, hipStream_t s) {
  const bool z = a.zero != nullptr;
  switch (group) {
    case 32: return z ? pick_mode<32, true>(mode, a, tiles, rows, s) : pick_mode<32, false>(mode, a, tiles, rows, s);
    case 64: return z ? pick_mode<64, true>(mode, a, tiles, rows, s) : pick_mode<64, false>(mode, a, tiles, rows, s);
    default: return z ? pick_mode<128, true>(mode, a, tiles, rows, s) : pick_mode<128, false>(mode, a, tiles, rows, s);
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
