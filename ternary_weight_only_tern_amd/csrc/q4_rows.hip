// Products with 4-bit weights for a few to some hundred activation rows, and
// the routed experts' slots and 16-row tiles: y[m][n] = sum_g s[n][g] sum_{k in g} (q - z) x.
//
// A workgroup of W wavefronts owns NB panels of 16 weight rows (a panel is
// contiguous in memory) and shares their K: wavefront w takes the 128-wide K
// tiles w, w + W, ...  A tile's codes and activations are loaded straight
// into the wavefront's own LDS in memory order (a load in the matrix
// operand's order, lane = row, would touch a line per lane), read back in the
// operands' order, and the next tile's loads are in flight while they are
// decoded and fed to v_mfma_f32_16x16x32_f16 (activations as A, 16 rows;
// weights as B, 16 columns; the experts' down products to the BF16 form, an
// inner value's parts in rows of their own).  A group's FP32 sum is scaled and added to the
// running FP32 sum.  The panels' scales and zero points are staged once, for
// the whole workgroup.  The wavefronts' sums are added in LDS in wavefront
// order: results do not depend on timing.  Loads go through buffer
// descriptors, whose bounds checks stand in for branches; what they leave in
// LDS behind the last row or behind k reaches no stored output.
//
// One row is bound by the reading of the codes where they are many (131072 x
// 2560, zero points, group 128: 33.8 us, 5.2 TB/s; a plain read of the bytes
// 26.7 us) and by one trip to memory where they are few (4096 x 4096: 4.2 us;
// the plain read 2.5 us).  From some ten rows on the waits of each wavefront's
// K tiles for the next, and then the decoding, repeated for every 16 or 32
// rows, bound it (13 x 12288 x 4096, group 64, zero points 8.8 us, 3.1 TB/s; 77
// x 2560 x 9728, group 32 16.3 us).
#include "q4_rows.h"

namespace tern {
namespace {

// LDS of a workgroup behind the wavefronts' staging: the scales and zero
// points of `panels` panels over `groups` groups.  Rows are padded to an odd
// number of dwords: a tile's 16 rows are read at once.
__host__ __device__ constexpr int scale_pitch(int groups) { return (groups + 7) / 8 * 8 + 2; }  // halves
__host__ __device__ constexpr int zero_pitch(int groups) { return (groups + 7) / 8 * 8 + 4; }   // bytes
constexpr size_t scale_bytes(int groups, int panels, bool z) {
  return (size_t)panels * 16 * (scale_pitch(groups) * 2 + (z ? zero_pitch(groups) : 0)) + 16;
}
constexpr size_t kLdsMost = 100 * 1024, kScaleMost = 32 * 1024;

// XR: rows of x at most (4, 16 or 32; kQ4Down: of inner values' parts).  ct: K tiles whose scales are staged
// at a time (all of them unless K is very long).
template <int G, bool Z, int XR, int NB, int W, int MODE>
__global__ __launch_bounds__(W * 64) void q4_rows_kernel(const Q4Args a, const int ct) {
  constexpr bool up = MODE == kQ4Up || MODE == kQ4UpSlot, token = MODE == kQ4DownToken;
  static_assert(!up || NB == 2, "gate and up panels go together");
  static_assert(!token || NB == 1, "one panel");
  constexpr bool inner = MODE == kQ4Down || token;    // x holds inner values in BF16
  // rows of x (of the operands) whose products make one row of the output
  constexpr int P = MODE == kQ4Down ? kInnerTile : token ? kInnerSlot : 1;
  constexpr int NBO = up ? 1 : NB;                    // panels of the output
  constexpr int XI = XR / 4, MT = (XR + 15) / 16;     // staging loads and operands of a tile's x
  constexpr int SG = 128 / G, S = (NB + XI) * 64;     // 16-byte chunks of a wavefront's staging
  extern __shared__ w4_t lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, kq = lane >> 4;
  const int k = a.k, ng = k / G, T = (k + 127) / 128;
  const int width = up ? a.n / 2 : a.n;  // output columns
  // Plain: the row chunks of one panel follow each other on one XCD
  // (blockIdx % 8), whose L2 then reads the panel once.
  const int chunks = MODE == kQ4Plain ? (a.m + XR - 1) / XR : 1;
  const int panel = MODE == kQ4Plain ? (int)blockIdx.x / 8 / chunks * 8 + (int)blockIdx.x % 8 : (int)blockIdx.x;
  const int n0 = panel * 16 * NBO;
  if (MODE == kQ4Plain && n0 >= width) return;
  w4_t* const cl = lds + wave * S;
  w4_t* const xl = cl + NB * 64;
  // scales [panel][16][sp], then zero points [panel][16][zp], of cg groups
  const int cg = min(ct * SG, ng), sp = scale_pitch(cg), zp = zero_pitch(cg), panels = token ? a.topk : NB;
  uint16_t* const sl = reinterpret_cast<uint16_t*>(lds + W * S);
  uint8_t* const zl = reinterpret_cast<uint8_t*>(sl + panels * 16 * sp);

  int e = 0, rows = 1, pos = blockIdx.y;  // output rows
  if (MODE == kQ4Up || MODE == kQ4Down) {
    if ((int)blockIdx.y >= *a.ntiles) return;
    const int4 tile = a.tiles[blockIdx.y];
    e = tile.x;
    pos = tile.y;
    rows = tile.z;
  } else if (MODE == kQ4UpSlot) {
    e = a.ids[blockIdx.y];
    if ((unsigned)e >= (unsigned)a.experts) return;
  } else if (MODE == kQ4Plain) {
    pos = (int)blockIdx.x / 8 % chunks * XR;
    rows = min(a.m - pos, XR);
  }

  const int xrows = rows * P;

  // panel b: 16 rows from row0(b), as many as exist
  auto row0 = [&](int b) {
    const int col = n0 + (up ? 0 : b * 16);
    return (col < width ? col : 0) + (up && b ? width : 0);
  };
  auto count = [&](int b) { return max(0, min(16, width - n0 - (up ? 0 : b * 16))); };
  __amdgpu_buffer_rsrc_t fc[NB], fx;
  auto aim = [&](int expert) {
#pragma unroll
    for (int b = 0; b < NB; ++b)
      fc[b] = q4_buffer(a.codes + ((size_t)expert * a.n + row0(b)) * (size_t)(k / 2), (uint32_t)count(b) * (uint32_t)(k / 2));
  };
  // The scales (zero points) of the workgroup's panels, groups g0 and on.  A
  // panel's 16 rows lie one behind the other: 16 bytes a load where they
  // start on a multiple of 16.  All panels (a token: its slots') in one pass;
  // one after another, their latencies would add up.
  auto stage_scales = [&](int expert, int g0) {
    const int want = min(cg, ng - g0);
    auto first = [&](int p) {  // the panel's first row's offset, or -1
      int ex = expert;
      if (token) {
        ex = a.ids[(size_t)pos * a.topk + p];
        if ((unsigned)ex >= (unsigned)a.experts) return (int64_t)-1;
      }
      return ((int64_t)ex * a.n + row0(token ? 0 : p)) * ng;
    };
    auto quotient = [](int i, int d) { return (int)(((float)i + 0.5f) / (float)d); };  // below 2^20, exact
    auto copy = [&](auto* dst, const auto* src, int pitch) {
      constexpr int E = 16 / sizeof(*src), D = E / 4;  // elements in 16 bytes, in a dword
      const bool full = count(0) == 16 && count(token ? 0 : panels - 1) == 16;
      if (full && want == ng && !((uintptr_t)src & 15) && (size_t)a.n * ng % E == 0) {
        const int per = 16 * ng / E;
        const float inv = 1.0f / (float)ng;
        for (int i = threadIdx.x; i < panels * per; i += W * 64) {
          const int p = token ? quotient(i, per) : NB == 1 ? 0 : (int)(i >= per), c = (i - p * per) * E;
          const int64_t at = first(p);
          if (at < 0) continue;
          const w4_t v = *reinterpret_cast<const w4_t*>(src + at + c);
          int row = (int)(((float)c + 0.5f) * inv), col = c - row * ng;
          row += p * 16;
          if (ng % D == 0) {
#pragma unroll
            for (int d = 0; d < 4; ++d) {
              *reinterpret_cast<uint32_t*>(dst + row * pitch + col) = v[d];
              if ((col += D) == ng) col = 0, ++row;
            }
          } else {  // dwords straddle rows
#pragma unroll
            for (int d = 0; d < E; ++d) {
              dst[row * pitch + col] = v[d / D] >> (32 / D * (d % D));
              if (++col == ng) col = 0, ++row;
            }
          }
        }
      } else {
        const int per = 16 * want;
        for (int i = threadIdx.x; i < panels * per; i += W * 64) {
          const int p = i / per, row = i % per / want, g = i % want;
          const int64_t at = first(p);
          if (at >= 0 && row < count(token ? 0 : p)) dst[(p * 16 + row) * pitch + g] = src[at + (int64_t)row * ng + g0 + g];
        }
      }
    };
    copy(sl, a.scale, sp);
    if (Z) copy(zl, a.zero, zp);
  };

  // the chunks of x this lane stages: row, chunk (swizzled by row like the codes)
  uint32_t xo[XI];
  if (MODE == kQ4Up) {
    fx = q4_buffer(a.x, (uint32_t)a.m * (uint32_t)k * 2);  // below 2 GiB (host)
  } else if (!token) {
    const size_t first = MODE == kQ4UpSlot ? pos / a.topk : pos;
    fx = q4_buffer(a.x + first * P * k, (uint32_t)xrows * (uint32_t)k * 2);
  }
#pragma unroll
  for (int j = 0; j < XI; ++j) {
    const int row = j * 4 + (lane >> 4);
    xo[j] = kFar;
    if (row < xrows)
      xo[j] = (uint32_t)(MODE == kQ4Up ? a.slots[pos + row] / a.topk : row) * (uint32_t)k * 2 + ((lane ^ row) & 15) * 16;
  }
  const int cr = lane >> 2;  // the chunk of the codes this lane stages
  const uint32_t co = (uint32_t)cr * (uint32_t)(k / 2) + (uint32_t)(code_chunk(cr, lane & 3) & 3) * 16;

  const Q4Masks masks;
  f4_t acc[MT][NB];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[i][b] = f4_t{0.f, 0.f, 0.f, 0.f};
  int slot_id = -1, slot_gate = 0;  // token: lane j holds slot j's expert and gate (topk <= 32, host)
  if (token && lane < a.topk) {
    slot_id = a.ids[(size_t)pos * a.topk + lane];
    slot_gate = __builtin_bit_cast(int, a.gates[(size_t)pos * a.topk + lane]);
  }
  if (!token) aim(e);

  for (int c0 = 0; c0 < T || c0 == 0; c0 += ct) {
    const int c1 = min(T, c0 + ct);
    // work unit v: tile c0 + v (a token: its slots' tiles one after another)
    const int tiles = c1 - c0, work = token ? a.topk * tiles : tiles;
    int t = 0, p = 0;
    float mul = 1.0f;
    auto issue = [&](int v) {
      t = c0 + v;
      if (token) {
        p = v / tiles;
        t = c0 + v - p * tiles;
        const size_t slot = (size_t)pos * a.topk + p;
        const int ex = __builtin_amdgcn_readlane(slot_id, p);
        if ((unsigned)ex >= (unsigned)a.experts) return false;
        mul = __builtin_bit_cast(float, __builtin_amdgcn_readlane(slot_gate, p));
        aim(ex);
        fx = q4_buffer(a.x + slot * P * k, (uint32_t)P * (uint32_t)k * 2);
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) q4_stage16(fc[b], cl + b * 64, co + (uint32_t)t * 64);
#pragma unroll
      for (int j = 0; j < XI; ++j)
        if (j == 0 || j * 4 < xrows) q4_stage16(fx, xl + j * 64, xo[j] + (uint32_t)t * 256);
      return true;
    };
    bool have = false;
    int v = wave;
    for (; v < work && !(have = issue(v)); v += W) {
    }
    if (c0) __syncthreads();  // the scales before these are in use until here
    stage_scales(e, c0 * SG);
    __syncthreads();
    while (have) {
      q4_loads_done();
      w4_t words[NB];
      w4_t x[MT][4];
#pragma unroll
      for (int b = 0; b < NB; ++b) words[b] = cl[b * 64 + code_chunk(r, kq)];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int row = min(i * 16 + r, xrows - 1);  // rows behind the last: a copy, not stored
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] = xl[row * 16 + ((x_chunk<G>(j, kq) ^ row) & 15)];
      }
      // this tile's scales and zero points of the lane's row; behind the last
      // group whatever lies there, not used
      uint16_t s[NB][SG];
      uint8_t z[NB][SG];
      const int left = min(SG, (k - t * 128) / G);  // groups in this tile
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int row = (token ? p : b) * 16 + r;
        const uint16_t* from = sl + row * sp + (t - c0) * SG;
        const uint8_t* zero = zl + row * zp + (t - c0) * SG;
#pragma unroll
        for (int j = 0; j < SG; j += 2) {
          if (SG == 1) {
            s[b][0] = from[0];
          } else {
            const uint32_t v = reinterpret_cast<const uint32_t*>(from)[j / 2];
            s[b][j] = (uint16_t)v;
            s[b][j + (SG > 1 ? 1 : 0)] = (uint16_t)(v >> 16);
          }
        }
        uint32_t v = 0x08080808u;
        if (Z) v = SG == 4 ? *reinterpret_cast<const uint32_t*>(zero) : SG == 2 ? *reinterpret_cast<const uint16_t*>(zero) : *zero;
#pragma unroll
        for (int j = 0; j < SG; ++j) z[b][j] = (uint8_t)(v >> (8 * j));
      }
      const float factor = mul;
      q4_reads_done();
      have = false;
      for (v += W; v < work && !(have = issue(v)); v += W) {
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const w4_t w = in_order<G>(words[b]);
#pragma unroll
        for (int j = 0; j < SG; ++j) {
          if (j && j >= left) break;
          const Q4Bias bias = q4_bias(z[b][j]);
          f4_t sum[MT];
#pragma unroll
          for (int i = 0; i < MT; ++i) sum[i] = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int q = j * (4 / SG); q < (j + 1) * (4 / SG); ++q) {
            const w4_t wv = q4_weights<inner>(w[q], bias, masks);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              if (MODE == kQ4Down && i * 16 >= xrows) break;
              sum[i] = q4_mfma16<inner>(x[i][q], wv, sum[i]);
            }
          }
          const float f = half_bits(s[b][j]) * (inner ? kInnerScale : 1.0f);
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            if (token)  // the slot's weight last: with kInnerScale alone it could leave FP32's range
              acc[i][b] += factor * (f * sum[i]);
            else
              acc[i][b] += f * sum[i];
          }
        }
      }
    }
  }

  // every wavefront's sums to its own staging, [operand][panel][lane]
  f4_t* const red = reinterpret_cast<f4_t*>(lds);
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int b = 0; b < NB; ++b)
      if (i * 16 + kq * 4 < xrows) red[wave * S + (i * NB + b) * 64 + lane] = acc[i][b];
  __syncthreads();
  for (int o = threadIdx.x; o < rows * NBO * 16; o += W * 64) {
    const int row = o / (NBO * 16), c = o % (NBO * 16), b = c / 16, col = n0 + c;
    float sum = 0.f, gate = 0.f;
#pragma unroll
    for (int i = P - 1; i >= 0; --i) {  // the smallest parts first
      const int xr = row * P + i, l = (xr / 16 * NB + b) * 64 + xr % 16 / 4 * 16 + c % 16;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        if (up) gate += red[w * S + l][xr % 4];
        sum += red[w * S + l + (up ? 64 : 0)][xr % 4];
      }
    }
    if (col >= width) continue;
    const size_t at = (size_t)pos + row, dst = at * width + col;
    if (MODE == kQ4UpSlot)
      q4_store_inner<kInnerSlot>(a.y, at * kInnerSlot * width + col, width, q4_swiglu(gate, sum));
    else if (MODE == kQ4Up)
      q4_store_inner<kInnerTile>(a.y, at * kInnerTile * width + col, width, q4_swiglu(gate, sum));
    else if (MODE == kQ4Down || a.y_f32)
      reinterpret_cast<float*>(a.y)[dst] = sum;
    else
      reinterpret_cast<_Float16*>(a.y)[dst] = (_Float16)sum;
  }
}

template <int G, bool Z, int XR, int NB, int W, int MODE>
hipError_t launch(const Q4Args& a, int tiles, hipStream_t s) {
  constexpr bool up = MODE == kQ4Up || MODE == kQ4UpSlot;
  constexpr int SG = 128 / G, S = (NB + XR / 4) * 64;
  const int width = up ? a.n / 2 : a.n, cols = 16 * (up ? 1 : NB);
  const int T = (a.k + 127) / 128, panels = MODE == kQ4DownToken ? a.topk : NB;
  constexpr size_t staging = (size_t)W * S * 16;
  const size_t most = kLdsMost - staging < kScaleMost ? kLdsMost - staging : kScaleMost;
  int ct = T > 0 ? T : 1;
  while (scale_bytes(ct * SG, panels, Z) > most && ct > 1) ct = (ct + 1) / 2;
  const size_t bytes = staging + scale_bytes(ct * SG, panels, Z);
  if (bytes > kLdsMost) return hipErrorInvalidValue;
  long long blocks = (width + cols - 1) / cols;
  if (MODE == kQ4Plain) blocks = (blocks + 7) / 8 * 8 * ((a.m + XR - 1) / XR);
  if (!grid_fits(blocks, W * 64)) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks, MODE == kQ4Plain ? 1u : (unsigned)tiles);
  if (bytes > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(q4_rows_kernel<G, Z, XR, NB, W, MODE>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)kLdsMost);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((q4_rows_kernel<G, Z, XR, NB, W, MODE>), grid, dim3(W * 64), bytes, s, a, ct);
  return hipGetLastError();
}

template <int G, bool Z>
hipError_t pick(int mode, const Q4Args& a, int tiles, int rows, hipStream_t s) {
  // Wavefronts of a panel that share K.  us of whole calls at 4, 8, 16: gate and
  // up, 64 experts of 2560 x 1024, top 8, one token 15.1, 15.1, 17.1, four tokens
  // 33.4, 34.2, 43.7; 16 of 4096 x 1056 at group 32, top 2, one token 16.1, 13.9,
  // 13.9; down, the same, one token 18.4, 15.5, 14.7, four tokens 35.8, 33.7, 37.1;
  // 8 of 4096 x 14336, one token 71, 54, 48.
  if (mode == kQ4UpSlot) return launch<G, Z, 4, 2, kUpSlotWaves, kQ4UpSlot>(a, tiles, s);
  if (mode == kQ4DownToken) {
    if (tiles == 1) return launch<G, Z, 4, 1, kDownOneTokenWaves, kQ4DownToken>(a, tiles, s);
    return launch<G, Z, 4, 1, kDownTokenWaves, kQ4DownToken>(a, tiles, s);
  }
  if (mode == kQ4Up) return launch<G, Z, 16, 2, kUpWaves, kQ4Up>(a, tiles, s);
  // Two panels of two wavefronts; one of four was slower (us of whole calls:
  // 64 experts of 2560 x 1024, 64 slots 52 against 49, 512 slots 103 against 90).
  if (mode == kQ4Down) {
    if (rows == kQ4TileFew) return launch<G, Z, 16, kDownPanels, kDownWaves, kQ4Down>(a, tiles, s);
    return launch<G, Z, 32, kDownPanels, kDownWaves, kQ4Down>(a, tiles, s);
  }
  // Wavefronts a panel: 4 where there are panels enough to fill the card, 16
  // where few panels have long rows; two or four panels at a time where there
  // are thousands.  us at W = 4, 8, 16 (m = 1, group 128): 12288 x 4096 6.9, 7.0,
  // 8.5; 4096 x 4096 4.3, 3.7, 4.2; 2560 x 9728 9.8, 6.6, 5.6; 131072 x 2560
  // 38.9, 51.6, 95.9, with two panels at W = 4 34.9; at W = 4, 8 (m = 16):
  // 12288 x 4096 8.4, 9.5; 4096 x 12288 13.7, 9.6; 131072 x 2560 with two, four
  // panels at W = 4 52, 43.
  const int panels = (a.n + 15) / 16, T = (a.k + 127) / 128;
  if (a.m <= 4) {
    if (panels >= 2048) return launch<G, Z, 4, 2, 4, kQ4Plain>(a, tiles, s);
    if (panels >= 512) return launch<G, Z, 4, 1, 4, kQ4Plain>(a, tiles, s);
    if (panels < 256 && T >= 64) return launch<G, Z, 4, 1, 16, kQ4Plain>(a, tiles, s);
    return launch<G, Z, 4, 1, 8, kQ4Plain>(a, tiles, s);
  }
  if (a.m <= 16) {
    if (panels >= 2048) return launch<G, Z, 16, 4, 4, kQ4Plain>(a, tiles, s);
    if (panels >= 512) return launch<G, Z, 16, 1, 4, kQ4Plain>(a, tiles, s);
    return launch<G, Z, 16, 1, 8, kQ4Plain>(a, tiles, s);
  }
  // Chunks of 32 rows decode the codes least often, several panels share the
  // activations' way from the L2; both leave fewer wavefronts.  us at 32 rows
  // with four panels (W = 4), two (W = 4, 7), one (W = 6), at 16 rows with two
  // (W = 8), by panels x chunks: m = 128, 12288 x 4096 (3.1 thousand) 23.6,
  // 27.8, 33.1, -, 33.7; m = 96, 9728 x 2560 (1824) 13.1, 15.2, 16.1, -, 17.6;
  // m = 64, 12288 x 4096 (1536) 17.2, 16.3, 16.9, -, 18.6; m = 128, 4096 x 4096
  // at group 64 (1024) 16.6, 15.3, 13.9, 23.5, 17.1; m = 64, 4096 x 12288 (512)
  // -, 18.8, 16.6, 23.5, 18.7; at group 32, 2560 x 9728: m = 77 (480) -, 24.9,
  // 17.9, 20.1, 18.7; m = 48 (320) -, 23.4, 16.5, 17.7, 12.2; m = 24 (160) -,
  // 22.6, -, 11.1, 11.8.
  // Seven wavefronts want K tiles: below two each four of 16 rows take less (7
  // of 32 rows / 4 of 16, group 128, group 32: m = 32, 12288 x 256 5.4 / 4.4, 6.0
  // / 4.6, x 1024 6.9 / 5.5, 7.4 / 6.4; m = 128, 4096 x 128 5.5 / 4.7, 5.7 / 4.9, x
  // 1024 7.0 / 6.3, 7.3 / 7.0; m = 64, 4096 x 512 4.7 / 4.2, 5.0 / 4.4).  The
  // other choices lie within 1.3 us of the best shape measured at K from 128 to
  // 2048, but for m = 64, 32768 rows, where four panels of two wavefronts take 7.2
  // against 9.4 at K = 128 and 26.2 against 29.4 at K = 2048 of group 32, and m =
  // 128, 12288 x 2048 of group 32 (two panels of four 20.8 against 23.6).
  const long long work = (long long)panels * ((a.m + 31) / 32);
  if (work >= 1792) return launch<G, Z, 32, 4, 4, kQ4Plain>(a, tiles, s);
  if (work >= 1152) return launch<G, Z, 32, 2, 4, kQ4Plain>(a, tiles, s);
  if (work >= 448 && T < 14) return launch<G, Z, 16, 2, 4, kQ4Plain>(a, tiles, s);
  if (work >= 448) return launch<G, Z, 32, 2, 7, kQ4Plain>(a, tiles, s);
  if (a.m <= 32) return launch<G, Z, 32, 1, 6, kQ4Plain>(a, tiles, s);
  return launch<G, Z, 16, 2, 8, kQ4Plain>(a, tiles, s);
}

}  // namespace

hipError_t launch_q4_rows(int mode, int group, const Q4Args& a, int tiles, int rows, hipStream_t s) {
  const bool z = a.zero != nullptr;
  switch (group) {
    case 32: return z ? pick<32, true>(mode, a, tiles, rows, s) : pick<32, false>(mode, a, tiles, rows, s);
    case 64: return z ? pick<64, true>(mode, a, tiles, rows, s) : pick<64, false>(mode, a, tiles, rows, s);
    default: return z ? pick<128, true>(mode, a, tiles, rows, s) : pick<128, false>(mode, a, tiles, rows, s);
  }
}

}  // namespace tern
