// Declarations and device code shared by the 4-bit kernels (q4_*.hip).  Not
// part of the public ABI.
//
// A 4-bit weight is W[n][k] = s[n][g] (q[n][k] - z[n][g]), g = k / G.  The
// code q - z (0..15 minus 0..255) is an exact FP16 integer, so every kernel
// here multiplies q - z with the FP16 activations on the matrix cores, sums
// one group in FP32, and applies the group's scale to that FP32 sum: no
// weight is ever rounded, and a scale's size costs neither range nor
// precision.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "tern.h"

namespace tern {

typedef _Float16 h2_t __attribute__((ext_vector_type(2)));
typedef _Float16 h8_t __attribute__((ext_vector_type(8)));
typedef __bf16 b8_t __attribute__((ext_vector_type(8)));
typedef short s2_t __attribute__((ext_vector_type(2)));
typedef float f4_t __attribute__((ext_vector_type(4)));
typedef float a16_t __attribute__((ext_vector_type(16)));
typedef uint32_t w2_t __attribute__((ext_vector_type(2)));
typedef uint32_t w4_t __attribute__((ext_vector_type(4)));

// One product, or the products of the slots that were routed to experts.
struct Q4Args {
  const uint8_t* codes;
  const uint16_t* scale;
  const uint8_t* zero;  // NULL: 8 everywhere
  const uint16_t* x;
  void* y;
  int32_t n, k, m;      // m: rows of x (plain product)
  int32_t y_f32;
  // split K (plain tiles): FP32 partials [splits][m][n], tiles of K per part
  float* partial;
  int32_t splits, tps;
  // experts
  const int4* tiles;     // {expert, first position, rows, 0}, sorted by expert
  const int32_t* ntiles;
  const int32_t* slots;  // position -> slot (token * topk + j)
  const int32_t* ids;    // [m][topk]
  const float* gates;    // [m][topk]
  int32_t topk, experts;
};

enum Q4Mode {
  kQ4Plain = 0,       // y[m][n]
  kQ4Up = 1,          // h[position][kInnerTile][n / 2] = silu(gate) * up, rows gathered from x
  kQ4Down = 2,        // part[position][n] (FP32) from h[position][kInnerTile][k]
  kQ4UpSlot = 3,      // as kQ4Up, one slot per tile: position = slot, expert = ids[slot]; h[slot][kInnerSlot][n / 2]
  kQ4DownToken = 4    // y[token][n] = sum over its slots from kQ4UpSlot's h
};

// An inner value is held as the sum of BF16 values, each what the ones before
// leave (q4_store_inner): two have 17 bits and cost the down product twice the
// matrix instructions; three have FP32's bits and are free for single slots,
// which fill three rows of an operand of sixteen.  BF16 because it has FP32's
// range: inner values are products of two projections, whose size a model
// bounds nowhere.
constexpr int kInnerTile = 2, kInnerSlot = 3;

// A grid's threads have to be countable in 32 bits.
inline bool grid_fits(long long blocks, int threads) { return blocks * threads < (1ll << 32); }

// Rows of the tile kernel's output tiles: 128 x 256 (one workgroup a CU), 96 x
// 256 (two), 64 x 128 (three) and 32 x 128 (five).
constexpr int kQ4TileLarge = 128, kQ4TileMid = 96, kQ4TileSmall = 64, kQ4TileTiny = 32;
// Rows of an experts' tile on the rows kernel.
constexpr int kQ4TileRows = 16, kQ4TileFew = 8;
// Wavefronts of its workgroups in the expert modes (their choice: q4_rows.hip),
// and the down tiles' panels of 16 columns.
constexpr int kUpSlotWaves = 8, kDownTokenWaves = 8, kDownOneTokenWaves = 16, kUpWaves = 4, kDownWaves = 2, kDownPanels = 2;
// max_tiles: experts' tiles at most (expert modes); rows: one of the
// four above, kQ4TileTiny or kQ4TileSmall in the expert modes; one of the two
// above on the rows kernel's tiles.
hipError_t launch_q4_rows(int mode, int group, const Q4Args& a, int max_tiles, int rows, hipStream_t s);
hipError_t launch_q4_tile(int mode, int group, const Q4Args& a, int max_tiles, int rows, hipStream_t s);
hipError_t launch_q4_reduce(const Q4Args& a, hipStream_t s);
hipError_t launch_q4_plan(const int32_t* ids, int slots, int experts, int rows, int4* tiles, int32_t* ntiles,
                          int32_t* order, int32_t* place, hipStream_t s);
hipError_t launch_q4_combine(const float* part, const int32_t* place, const float* gates, int m, int topk, int n,
                             void* y, int y_f32, hipStream_t s);
hipError_t launch_q4_pack(const uint8_t* q, size_t words, uint8_t* codes, uint32_t* flag, hipStream_t s);
hipError_t launch_q4_unpack(const uint8_t* codes, size_t words, uint8_t* q, hipStream_t s);

struct RouteArgs {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* weights;
  int32_t m, experts, topk, groups, best, keep, renorm, sigmoid;
  float scale;
};
hipError_t launch_route(const RouteArgs& a, int f16, hipStream_t s);


// ---------------------------------------------------------------- device code
__device__ inline h2_t as_h2(uint32_t v) { return __builtin_bit_cast(h2_t, v); }

// What turns 1024 + q and 1024 + 16 q into q - z, and the two bit patterns of
// q4_decode, kept in registers: v_and_or_b32 takes no literal.
struct Q4Bias {
  h2_t lo, hi;  // -(1024 + z), -(64 + z)
};
__device__ inline Q4Bias q4_bias(uint32_t z) {  // 0..255
  const _Float16 l = __builtin_bit_cast(_Float16, (uint16_t)(0xE400u | z));
  const _Float16 h = l + (_Float16)960.0f;
  return {h2_t{l, l}, h2_t{h, h}};
}
struct Q4Masks {
  uint32_t lo = 0x000F000Fu, hi = 0x00F000F0u, one = 0x64006400u;
  __device__ inline Q4Masks() { asm("" : "+v"(lo), "+v"(hi), "+s"(one)); }
};

// Eight codes of a word to FP16 q - z, in k order.  A code ORed into the low
// mantissa bits of 1024.0 is 1024 + q, into bits 4..7 1024 + 16 q; both
// steps back are exact.  Nine VALU operations per word.
__device__ inline h8_t q4_decode(uint32_t w, const Q4Bias& b, const Q4Masks& m) {
  const h2_t six = {(_Float16)0.0625f, (_Float16)0.0625f};
  const uint32_t v = w >> 8;
  const h2_t p0 = as_h2((w & m.lo) | m.one) + b.lo;
  const h2_t p1 = as_h2((w & m.hi) | m.one) * six + b.hi;
  const h2_t p2 = as_h2((v & m.lo) | m.one) + b.lo;
  const h2_t p3 = as_h2((v & m.hi) | m.one) * six + b.hi;
  return h8_t{p0.x, p0.y, p1.x, p1.y, p2.x, p2.y, p3.x, p3.y};
}

// The same as BF16 (q - z) 2^-112, the down product's operand: FP16's bits of
// an integer below 256 end in three zeros, so that a shift by three leaves
// BF16's seven bits of mantissa and FP16's exponent where BF16's is read, its
// bias 112 larger.  The inner values are held 2^56 times as large, the sums'
// scales too: products lie 2^-56 below their value, in FP32's range for inner
// values from 2^-50 to 2^71, and every factor is exact.  Eight more operations
// per word.
constexpr float kInnerScale = 0x1p56f;
__device__ inline b8_t q4_decode_inner(uint32_t w, const Q4Bias& b, const Q4Masks& m) {
  w4_t v = __builtin_bit_cast(w4_t, q4_decode(w, b, m));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t pair = v[i];  // a bit cast of v[i] itself would read v[0]
    v[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(s2_t, pair) >> 3) & 0x8FFF8FFFu;
  }
  return __builtin_bit_cast(b8_t, v);
}

// Weights of a word as the B operand and its product with A, 16 bytes of x
// (FP16) or of inner values (BF16).
template <bool INNER>
__device__ inline w4_t q4_weights(uint32_t w, const Q4Bias& b, const Q4Masks& m) {
  if constexpr (INNER) return __builtin_bit_cast(w4_t, q4_decode_inner(w, b, m));
  return __builtin_bit_cast(w4_t, q4_decode(w, b, m));
}
template <bool INNER>
__device__ inline f4_t q4_mfma16(w4_t x, w4_t w, f4_t c) {
  if constexpr (INNER)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8_t, x), __builtin_bit_cast(b8_t, w), c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8_t, x), __builtin_bit_cast(h8_t, w), c, 0, 0, 0);
}
template <bool INNER>
__device__ inline a16_t q4_mfma32(w4_t x, w4_t w, a16_t c) {
  if constexpr (INNER)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b8_t, x), __builtin_bit_cast(b8_t, w), c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8_t, x), __builtin_bit_cast(h8_t, w), c, 0, 0, 0);
}

// An inner value to PARTS rows of BF16 values, `pitch` apart.
template <int PARTS>
__device__ inline void q4_store_inner(void* y, size_t at, size_t pitch, float h) {
  __bf16* const to = reinterpret_cast<__bf16*>(y) + at;
  float rest = h * kInnerScale;
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    const __bf16 v = (__bf16)rest;
    to[i * pitch] = v;
    rest = fabsf((float)v) < INFINITY ? rest - (float)v : 0.0f;  // exact; nothing beside an infinity or a NaN
  }
}

__device__ inline float half_bits(uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }

__device__ inline float q4_swiglu(float gate, float up) { return gate / (1.0f + __expf(-gate)) * up; }

}  // namespace tern
