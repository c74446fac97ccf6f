// Declarations and device code shared by the kernels of rotary positions, the
// 8-bit cache and attention over it (rope.hip, kv_*.hip).  Not part of the
// public ABI.
//
// A page holds 64 tokens of one head, 64 D bytes of keys and as many of
// values, in the order in which the matrix cores' operands take them: a
// wavefront that loads 16 consecutive bytes a lane has the operand of
// v_mfma_f32_16x16x32_f16 in its registers, without LDS or shuffles.
//   keys    token 16a + 4t + i, dimension 64c + 16r + b  at  ((4c + t) 64 + 16r + 4a + i) 16 + b
//   values  token 16a + j, dimension 16c + e             at  ((4c + a) 16 + e) 16 + j
// (c for a chunk of dimensions).  The product of keys and queries leaves lane
// group a of a row with the scores of tokens 16a + 4t + i, and the same lane
// group holds the values of tokens 16a .. 16a + 15: the weights go from the
// first product into the second without leaving their lane.
// A byte is code + 128, so that 0x6400 | byte is the FP16 number 1024 + 128 +
// code: decoding is one byte permutation and one packed subtraction for two
// codes, exact.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <type_traits>

#include "tern.h"

namespace tern {

constexpr int kPage = TERN_KV_PAGE;
// Positions and rows stay below these, so that their sums fit 32 bits.
constexpr int kMaxTokens = 1 << 30, kMaxRows = 1 << 29;
constexpr int kMaxStride = 1 << 23;  // of q in attention: 64 rows lie in one buffer

// Turning and norm of a head's values (tern_rotary).
struct Rotary {
  const double* freq;
  const uint16_t* norm;
  float amp, eps;
  int32_t rot, inter;
  int32_t on;  // 0: values pass unchanged
};

struct RopeArgs {
  const uint16_t* x;
  uint16_t* out;
  int64_t x_stride, out_stride;
  const int32_t* pos;
  Rotary r;
  int32_t m, heads, dim;
};

// Which rows belong to which sequence (tern_kv_batch).
struct Batch {
  const int32_t *start, *len, *pages;
  int32_t count, rows, max_rows, max_pages;
};

struct Cache {
  uint8_t *k, *v;
  float *ks, *vs;
  int32_t heads, pages;
};

struct WriteArgs {
  Cache c;
  Batch b;
  const uint16_t *k, *v, *q;
  uint16_t* q_out;
  int64_t k_stride, v_stride, q_stride;
  Rotary rk, rq;
  int32_t q_heads;
  int32_t items;       // pages that a sequence's rows may lie in
  int32_t kv_blocks;   // workgroups before those of q
  int32_t q_waves;     // wavefronts for a row of q
};

struct ReadArgs {
  Cache c;
  Batch b;
  void *k, *v;
  int32_t f32, items;
};

struct AttnArgs {
  Cache c;
  Batch b;
  const uint16_t* q;
  int64_t q_stride;
  uint16_t* y;         // [rows][q_heads][dim]
  // Few rows: pieces of the line of all pages (whole: units), `per` pages each
  // at least; their sums [pieces][2][max_rows * group][dim] and references and
  // sums of weights [pieces][2][max_rows * group][2] in part; info: a unit's first
  // piece and how many it has.  Tiles (tiles > 0): parts of the context at most,
  // `per` pages each at least; part: [tiles][count][heads][parts][128][dim] in an order of the
  // kernel's own, then [tiles][count][heads][parts][128][2].
  float* part;
  int2* info;
  float scale;         // times log2(e)
  int32_t q_heads, group, window, causal;
  int32_t pieces, whole, parts, per, tiles;
};

// Rows (of a sequence, times the query heads of one cache head) of one
// workgroup: the kernel for few rows, by blocks of 16, and the tiles.
constexpr int kAttnFew = 16, kAttnMid = 64, kAttnTile = 128;

hipError_t launch_rope(const RopeArgs& a, hipStream_t s);
hipError_t launch_kv_write(WriteArgs a, int dim, hipStream_t s);
hipError_t launch_kv_read(const ReadArgs& a, int dim, hipStream_t s);
// blocks: of 16 rows, 1 or 2; shares: wavefronts of a whole unit
hipError_t launch_attn_rows(const AttnArgs& a, int dim, int blocks, int shares, hipStream_t s);
hipError_t launch_attn_tile(const AttnArgs& a, int dim, hipStream_t s);
hipError_t launch_attn_join_rows(const AttnArgs& a, int dim, hipStream_t s);
hipError_t launch_attn_mid(const AttnArgs& a, int dim, hipStream_t s);
// rows: of a tile
hipError_t launch_attn_join_tile(const AttnArgs& a, int dim, int rows, hipStream_t s);

// Wavefronts that share a row's heads: one where there are rows enough to fill
// the card, as many as have heads where there are few.
inline int kv_waves(long long rows, int heads, int lanes) {
  const int most = (heads * lanes + 63) / 64;
  int waves = 1;
  while (waves < most && rows * waves < 2048) waves *= 2;
  return waves < most ? waves : most;
}

// A launch without the <<<>>> form, which sets its shape aside first and copies the
// arguments once more (a write 3.85 -> 3.1 us of host time, attention's two 6.7 ->
// 5.4).  The arguments are of the kernel's own types.
template <typename... A>
hipError_t kv_launch(void (*kernel)(A...), dim3 grid, int threads, hipStream_t s, const std::common_type_t<A>&... args) {
  const void* p[] = {&args...};
  const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(threads), const_cast<void**>(p), 0, s);
  if (e != hipSuccess) (void)hipGetLastError();
  return e;
}

// A grid's threads have to be countable in 32 bits.
inline bool kv_grid_fits(long long blocks, int threads) { return blocks * threads < (1ll << 32); }

// ---------------------------------------------------------------- device code
#ifdef __HIPCC__
typedef _Float16 kh2_t __attribute__((ext_vector_type(2)));
typedef _Float16 kh4_t __attribute__((ext_vector_type(4)));
typedef _Float16 kh8_t __attribute__((ext_vector_type(8)));
typedef float kf4_t __attribute__((ext_vector_type(4)));
typedef float kf16_t __attribute__((ext_vector_type(16)));
typedef uint32_t kw2_t __attribute__((ext_vector_type(2)));
typedef uint32_t kw4_t __attribute__((ext_vector_type(4)));

// An element of an array that nothing writes while the kernel runs: with an
// index that is the same in every lane a scalar load, which does not queue
// behind the vector loads in flight, whatever the kernel stores elsewhere.
template <class T>
__device__ inline T kv_const(const T* p, size_t i) {
  return ((const __attribute__((address_space(4))) T*)p)[i];
}

// A sequence's rows in the arrays of rows and its place in the cache.  Rows
// beyond max_rows or behind the arrays' end are left out, whatever start says.
struct Span {
  int first, n;  // rows that are there
  int from;      // position of the first row; negative: rows before the sequence's beginning
  int len;       // tokens, 0 at least
};
__device__ inline Span span_of(const Batch& b, int s) {
  Span r;
  int n = b.max_rows;
  r.first = s * b.max_rows;
  if (b.start) {
    r.first = min(max(kv_const(b.start, s), 0), b.rows);
    n = min(max(kv_const(b.start, s + 1) - r.first, 0), b.rows - r.first);
  }
  r.n = min(n, b.max_rows);
  r.len = min(max(kv_const(b.len, s), 0), kMaxTokens);
  r.from = r.len - n;
  return r;
}

// The page of a sequence's tokens 64 p ..; -1: none.
__device__ inline int page_of(const Batch& b, const Cache& c, int s, int p) {
  if (p >= b.max_pages) return -1;
  const int id = kv_const(b.pages, (size_t)s * b.max_pages + p);
  return id >= 0 && id < c.pages ? id : -1;
}

// Four bytes code + 128 to FP16 codes.
__device__ inline void codes4(uint32_t w, kh2_t& lo, kh2_t& hi) {
  const kh2_t bias = {(_Float16)-1152.0f, (_Float16)-1152.0f};
  lo = __builtin_bit_cast(kh2_t, __builtin_amdgcn_perm(0x64646464u, w, 0x04010400u)) + bias;
  hi = __builtin_bit_cast(kh2_t, __builtin_amdgcn_perm(0x64646464u, w, 0x04030402u)) + bias;
}
__device__ inline kh8_t codes8(uint32_t w0, uint32_t w1) {
  kh2_t a, b, c, d;
  codes4(w0, a, b);
  codes4(w1, c, d);
  return kh8_t{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// A buffer of bytes at p, the same in every lane (said so explicitly: a
// descriptor that the compiler cannot prove uniform costs a loop around every
// load).  A load past its end gives zeros and moves nothing, which stands in
// for branches around loads.
__device__ inline __amdgpu_buffer_rsrc_t kv_buffer(const void* p, int bytes) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>((uint64_t)hi << 32 | lo), (short)0,
                                           __builtin_amdgcn_readfirstlane(bytes), 0x00020000);
}
constexpr int kFarAway = (int)0x80000000;  // an offset past every buffer
constexpr int kv_stream = 2;  // bytes that are read once pass the caches by
template <int AUX = 0>
__device__ inline kw4_t kv_load16(__amdgpu_buffer_rsrc_t r, int offset) {
  return __builtin_bit_cast(kw4_t, __builtin_amdgcn_raw_buffer_load_b128(r, offset, 0, AUX));
}

// Bits of the FP16 value nearest to v.
__device__ inline uint16_t kv_bits(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
__device__ inline float kv_half(uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }

// cos and sin of the angle pos * freq, times amp.  The angle is taken to a
// turn in FP64 (2^31 turns would still leave 2^-22 of a turn).
__device__ inline void angle_of(double pos, double freq, float amp, float& c, float& s) {
  const double turns = pos * freq * 0.15915494309189533577;
  const float t = (float)(turns - rint(turns));
  c = amp * __builtin_amdgcn_cosf(t);
  s = amp * __builtin_amdgcn_sinf(t);
}

// The eight values of a head that a lane holds, four pairs (y[e], y[4 + e])
// from pair i0 on in the half layout, four neighbours of dimension a and four
// of b elsewhere.  Pair i is dimensions (i, i + rot / 2) where it turns, and
// (2i, 2i + 1) behind that: one lane of a head may hold both kinds (mixed).
struct Place {
  int a, b, i0;
  bool mixed;
};
__device__ inline bool sided(const Rotary& r) { return !r.inter && r.rot > 0; }
__device__ inline Place place_of(const Rotary& r, int lane) {
  const int half = r.rot / 2, i0 = 4 * lane;
  if (!sided(r) || i0 >= half) return {8 * lane, 8 * lane + 4, i0, false};
  return {i0, i0 + half, i0, i0 + 4 > half};
}
__device__ inline int dim_of(const Rotary& r, const Place& at, int e) {
  if (!at.mixed) return e < 4 ? at.a + e : at.b + e - 4;
  const int i = at.i0 + e % 4;
  return i < r.rot / 2 ? (e < 4 ? i : i + r.rot / 2) : 2 * i + e / 4;
}

// The frequencies of the lane's four pairs (0 for those that do not turn), and
// cos and sin of their angles at position pos.
struct Freqs {
  double f[4];
};
struct Angles {
  float c[4], s[4];
};
__device__ inline Freqs freqs_of(const Rotary& r, const Place& at) {
  Freqs q;
#pragma unroll
  for (int e = 0; e < 4; ++e) q.f[e] = at.i0 + e < r.rot / 2 ? r.freq[at.i0 + e] : 0.0;
  return q;
}
__device__ inline Angles angles_of(const Rotary& r, const Freqs& q, int pos) {
  Angles g;
#pragma unroll
  for (int e = 0; e < 4; ++e) angle_of((double)pos, q.f[e], r.amp, g.c[e], g.s[e]);
  return g;
}

union Eight {
  kw2_t w[2];
  uint16_t h[8];
};
typedef kw2_t kw2u_t __attribute__((aligned(2)));  // the pairs' second side lies anywhere
__device__ inline Eight load_eight(const uint16_t* x, const Rotary& r, const Place& at) {
  Eight v;
  if (at.mixed) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v.h[e] = x[dim_of(r, at, e)];
    return v;
  }
  v.w[0] = *reinterpret_cast<const kw2_t*>(x + at.a);
  v.w[1] = *reinterpret_cast<const kw2u_t*>(x + at.b);
  return v;
}
__device__ inline void store_eight(uint16_t* x, const Rotary& r, const Place& at, const Eight& v) {
  if (at.mixed) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[dim_of(r, at, e)] = v.h[e];
    return;
  }
  *reinterpret_cast<kw2_t*>(x + at.a) = v.w[0];
  *reinterpret_cast<kw2u_t*>(x + at.b) = v.w[1];
}

// A lane's values v of a head, normed (by the weights w at its place) and
// turned, rounded to FP16.  All lanes of the head (`lanes` of them, a power of
// two, neighbours) call it together; those without values hold zeros.  Every
// product and sum is spelled out, so that all kernels round alike.
__device__ inline Eight turn_eight(Eight v, const Eight& w, const Place& at, int dim, int lanes, const Rotary& r, const Angles& g) {
  if (!r.on) return v;
  float y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = kv_half(v.h[e]);
  if (r.norm) {
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(y[e], y[e], sum);
    for (int o = 1; o < lanes; o <<= 1) sum += __shfl_xor(sum, o);
    const float inv = 1.0f / sqrtf(sum / dim + r.eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = (inv * kv_half(w.h[e])) * y[e];
  }
  const int pairs = r.rot / 2 - at.i0;  // that turn
  auto turn = [&](int e, float& p, float& q) {
    const float a = p, b = q;
    if (e < pairs) {
      p = __builtin_fmaf(a, g.c[e], -(b * g.s[e]));
      q = __builtin_fmaf(b, g.c[e], a * g.s[e]);
    }
  };
  if (r.inter) {
#pragma unroll
    for (int e = 0; e < 4; ++e) turn(e, y[2 * e], y[2 * e + 1]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) turn(e, y[e], y[4 + e]);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v.h[e] = kv_bits(y[e]);
  return v;
}

// A wavefront turns heads first, first + step, .. of a row, several at a time.
__device__ inline void turn_row(const uint16_t* x, uint16_t* out, int heads, int dim, int lanes, int first, int step,
                                const Rotary& r, int pos) {
  const int lane = threadIdx.x % lanes;
  const bool live = lane * 8 < dim;
  const Place at = place_of(r, lane);
  const Angles g = angles_of(r, freqs_of(r, at), pos);
  Eight w = {};
  if (live && r.norm) w = load_eight(r.norm, r, at);
  // the next heads are read while these are turned (out may be x: they are others)
  int h = first + (threadIdx.x & 63) / lanes;
  Eight v = {};
  if (live && h < heads) v = load_eight(x + (int64_t)h * dim, r, at);
  for (int h0 = first; h0 < heads; h0 += step, h += step) {
    Eight next = {};
    if (live && h + step < heads) next = load_eight(x + (int64_t)(h + step) * dim, r, at);
    const Eight y = turn_eight(v, w, at, dim, lanes, r, g);
    if (live && h < heads) store_eight(out + (int64_t)h * dim, r, at, y);
    v = next;
  }
}

#endif

}  // namespace tern
