// Writing rows of keys and values into the 8-bit cache and reading them back
// (tern_kv_write and tern_kv_read in tern.h).
//
// A page's scale s has 8 significant bits and the values 11 (the keys are
// rounded to FP16 after they are turned, as if a call of tern_rope had done
// it): codes are the exact quotients' roundings (byte_of), and the growth's
// comparison with 127 s is exact.
//
// One workgroup has a (page, head) of the keys or of the values, so that a
// scale has one writer.  A thread owns pieces of the page: of the
// keys two words of four dimensions of a token, of the values 16 tokens of four
// dimensions.  It alone reads, rounds
// again and writes those bytes; nothing is shared but the largest value.  q's
// rows are turned by further workgroups of the same launch (rope.hip's way).
//
// Bound by vector instructions and bytes: a prompt of 4096 tokens, 8 heads of
// 128 with 32 of q, takes 26-28 us (92 MB read and written, 3.4 TB/s; the vector
// units are busy for 72 % of the cycles: norms, FP64 angles of every head's keys,
// codes).  Prefixes of 96000 tokens, 8 heads, are read back as FP32 in 124 us (4.6
// TB/s), as FP16 in 79.  A token each of 48 sequences takes 5.8-6.1 us, a chain of
// four trips to memory: lengths, page number, scale, the page's other codes.
#include "kv.h"

namespace tern {
namespace {

// Scale of 8 significant bits, the smallest with most <= 127 s.
__device__ inline float least_scale(float most) {
  return __uint_as_float((__float_as_uint(most / 127.0f) + 0xFFFFu) & 0xFFFF0000u);
}

// The byte of x in steps of s, inv = 1 / s (0 beside a scale that is 0 or NaN).
// x inv is off by 2^-23 of the quotient.  A quotient that is no tie is 2^-16 of
// itself away from one: |2X 2^a - (2n+1) S 2^b|, with X of 11 bits and S of 8, is
// 2^b at least, against (2n+1) S 2^b with 2n+1 < 256, or 2^(a+1), against 2X 2^a.
// So with 18 bits left a tie is one again and nothing else becomes one.
// The sum with 1.5 2^23 + 128 rounds to a whole number, whose low byte is it + 128;
// nothing is past 127 steps of its page's scale.
__device__ inline float steps_of(float s) { return s > 0.f ? 1.0f / s : 0.f; }
constexpr float kToByte = 12583040.0f;
__device__ inline uint32_t byte_of(float x, float inv) {
  return __float_as_uint(__uint_as_float((__float_as_uint(x * inv) + 0x20u) & ~0x3Fu) + kToByte);
}

// The low bytes of four words.
__device__ inline uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_amdgcn_perm(b, a, 0x0c0c0400u) | __builtin_amdgcn_perm(d, c, 0x04000c0cu);
}

// Four bytes rounded again to steps that are 1 / shrink times as large.
__device__ inline uint32_t again4(uint32_t w, float shrink) {
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(__builtin_fmaf((float)((w >> (8 * i)) & 255u) - 128.f, shrink, kToByte));
  return pack4(b[0], b[1], b[2], b[3]);
}

// 4 x 4 bytes: out[j] has byte j of every in.
__device__ inline void transpose4(const uint32_t in[4], uint32_t out[4]) {
  const uint32_t a = __builtin_amdgcn_perm(in[1], in[0], 0x05010400u), b = __builtin_amdgcn_perm(in[1], in[0], 0x07030602u);
  const uint32_t c = __builtin_amdgcn_perm(in[3], in[2], 0x05010400u), d = __builtin_amdgcn_perm(in[3], in[2], 0x07030602u);
  out[0] = __builtin_amdgcn_perm(c, a, 0x05040100u);
  out[1] = __builtin_amdgcn_perm(c, a, 0x07060302u);
  out[2] = __builtin_amdgcn_perm(d, b, 0x05040100u);
  out[3] = __builtin_amdgcn_perm(d, b, 0x07060302u);
}

// The page's new scale, from the largest magnitude's FP16 bits that each
// thread has seen, and what old codes shrink by.
struct Grown {
  float s, shrink;
  bool keep;  // old codes stay as they are
};
__device__ inline Grown grow(uint32_t bits, bool fresh, float old) {
  __shared__ uint32_t seen[4];
  for (int o = 32; o; o >>= 1) bits = max(bits, (uint32_t)__shfl_xor((int)bits, o));
  if (threadIdx.x % 64 == 0) seen[threadIdx.x / 64] = bits;
  __syncthreads();
  bits = max(max(seen[0], seen[1]), max(seen[2], seen[3]));
  Grown g = {old, 1.0f, true};
  if (bits >= 0x7C00u) {  // an infinity or a NaN
    g.s = NAN;
    return g;
  }
  const float most = kv_half((uint16_t)bits);
  if (fresh || old == 0.f) {
    g.s = least_scale(most);
    return g;
  }
  for (int i = 0; i < 300 && most > 127.0f * g.s; ++i) {  // 41 times at most between FP16 values
    g.s *= 2.0f;
    g.shrink *= 0.5f;
    g.keep = false;
  }
  return g;
}

// Of the keys a thread owns, token by token, what a lane holds of a head (kv.h),
// two words of the page.
template <int D>
__device__ void write_keys(const WriteArgs& a, const Span& sp, int s, int page, int head, int t0, int t1) {
  constexpr int kLanes = D / 8, kRound = 256 / kLanes, kRounds = kPage / kRound;
  const int lane = threadIdx.x % kLanes;
  const Place place = place_of(a.rk, lane);
  Eight v[kRounds], weight = {};
  const int first = threadIdx.x / kLanes;  // tokens of a round
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const int token = i * kRound + first;
    v[i] = {};
    if (token >= t0 && token < t1)
      v[i] = load_eight(a.k + (sp.first + page * kPage + token - sp.from) * a.k_stride + head * D, a.rk, place);
  }
  if (a.rk.norm) weight = load_eight(a.rk.norm, a.rk, place);
  const Freqs freqs = freqs_of(a.rk, place);
  const int id = page_of(a.b, a.c, s, page);
  if (id < 0) return;
  const size_t at = (size_t)id * a.c.heads + head;
  const float old = fabsf(a.c.ks[at]);
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const int token = i * kRound + first;
    if (i * kRound >= t1 || i * kRound + kRound <= t0) continue;  // the same for all: no token of this round
    const Angles g = angles_of(a.rk, freqs, page * kPage + token);
    v[i] = turn_eight(v[i], weight, place, D, kLanes, a.rk, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) bits = max(bits, (uint32_t)v[i].h[e] & 0x7FFFu);
  }
  const Grown g = grow(bits, t0 == 0, old);
  if (threadIdx.x == 0) a.c.ks[at] = g.s;
  uint8_t* const base = a.c.k + at * (kPage * D);
  const float inv = steps_of(g.s);
  if (!(inv > 0.f))  // codes 0, whatever the values
#pragma unroll
    for (int i = 0; i < kRounds; ++i) v[i] = {};
  const bool words = !sided(a.rk) || a.rk.rot % 8 == 0;  // four dimensions are a word of the page
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const int token = i * kRound + first;
    const bool live = token >= t0 && token < t1;
    if (!live && g.keep) continue;
    auto byte_at = [&](int d) {
      return base + ((d / 64 * 4 + token / 4 % 4) * 64 + d / 16 % 4 * 16 + token / 16 * 4 + token % 4) * 16 + d % 16;
    };
    if (words) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t* const to = reinterpret_cast<uint32_t*>(byte_at(q ? place.b : place.a));
        auto byte = [&](int e) { return byte_of(kv_half(v[i].h[4 * q + e]), inv); };
        *to = live ? pack4(byte(0), byte(1), byte(2), byte(3)) : again4(*to, g.shrink);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        uint8_t* const to = byte_at(dim_of(a.rk, place, e));
        *to = (uint8_t)(live ? byte_of(kv_half(v[i].h[e]), inv) : again4(*to, g.shrink));
      }
    }
  }
}

// Of the values a thread owns 16 tokens of four dimensions, 64 contiguous bytes.
template <int D>
__device__ void write_values(const WriteArgs& a, const Span& sp, int s, int page, int head, int t0, int t1) {
  const int part = threadIdx.x / (D / 4), d0 = threadIdx.x % (D / 4) * 4;  // D = 256: four parts, else idle threads
  kh4_t y[16];
  uint32_t bits = 0;
  const bool some = part < 4 && t0 < part * 16 + 16 && t1 > part * 16;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const int token = part * 16 + j;
    y[j] = kh4_t{0, 0, 0, 0};
    if (some && token >= t0 && token < t1)
      y[j] = *reinterpret_cast<const kh4_t*>(a.v + (sp.first + page * kPage + token - sp.from) * a.v_stride + head * D + d0);
  }
  const int id = page_of(a.b, a.c, s, page);
  if (id < 0) return;
  const size_t at = (size_t)id * a.c.heads + head;
  const float old = fabsf(a.c.vs[at]);
#pragma unroll
  for (int j = 0; j < 16; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const _Float16 x = y[j][e];  // a bit cast of the element itself would read the first
      bits = max(bits, (uint32_t)__builtin_bit_cast(uint16_t, x) & 0x7FFFu);
    }
  // the bytes of other tokens are read before it is known whether they grow
  const bool all = t0 <= part * 16 && t1 >= part * 16 + 16;
  kw4_t* const to = reinterpret_cast<kw4_t*>(a.c.v + at * (kPage * D) + ((d0 / 16 * 4 + part % 4) * 16 + d0 % 16) * 16);
  kw4_t o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = all || part >= 4 || (!some && t0 == 0) ? kw4_t{0, 0, 0, 0} : to[e];
  const Grown g = grow(bits, t0 == 0, old);
  if (threadIdx.x == 0) a.c.vs[at] = g.s;
  if (part >= 4 || (g.keep && !some)) return;
  if (!g.keep)
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int q = 0; q < 4; ++q) o[e][q] = again4(o[e][q], g.shrink);
  const float inv = steps_of(g.s);
  if (!(inv > 0.f))
#pragma unroll
    for (int j = 0; j < 16; ++j) y[j] = kh4_t{0, 0, 0, 0};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (t1 <= part * 16 + q * 4 || t0 >= part * 16 + q * 4 + 4) continue;
    uint32_t mask = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (part * 16 + q * 4 + i >= t0 && part * 16 + q * 4 + i < t1) mask |= 255u << (8 * i);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      auto byte = [&](int i) { return byte_of((float)y[q * 4 + i][e], inv); };
      o[e][q] = (o[e][q] & ~mask) | (pack4(byte(0), byte(1), byte(2), byte(3)) & mask);
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) to[e] = o[e];
}

template <int D>
__global__ __launch_bounds__(256) void kv_write_kernel(const WriteArgs a) {
  int bid = blockIdx.x;
  if (bid >= a.kv_blocks) {  // wavefronts of rows of q
    constexpr int lanes = D / 8, per = 64 / lanes;
    const int64_t wave = (int64_t)(bid - a.kv_blocks) * 4 + threadIdx.x / 64;
    const int64_t r = wave / a.q_waves;
    const int s = (int)(r / a.b.max_rows), j = (int)(r % a.b.max_rows);
    if (s >= a.b.count) return;
    const Span sp = span_of(a.b, s);
    if (j >= sp.n) return;
    const int64_t row = sp.first + j;
    turn_row(a.q + row * a.q_stride, a.q_out + row * a.q_heads * D, a.q_heads, D, lanes, (int)(wave % a.q_waves) * per,
             a.q_waves * per, a.rq, sp.from + j);
    return;
  }
  const bool values = bid & 1;
  bid >>= 1;
  const int head = bid % a.c.heads;
  bid /= a.c.heads;
  const int s = bid / a.items;
  const Span sp = span_of(a.b, s);
  const int begin = max(sp.from, 0), end = sp.from + sp.n;  // positions of the rows that are there
  const int page = begin / kPage + bid % a.items;
  const int t0 = max(begin - page * kPage, 0), t1 = min(end - page * kPage, kPage);
  if (t0 >= t1) return;
  if (values)
    write_values<D>(a, sp, s, page, head, t0, t1);
  else
    write_keys<D>(a, sp, s, page, head, t0, t1);
}

constexpr kw4_t kNone = {0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u};  // codes 0

// One workgroup has a (page, head), its keys or its values.
template <int D, bool F32>
__global__ __launch_bounds__(256) void kv_read_kernel(const ReadArgs a) {
  int bid = blockIdx.x;
  const bool values = bid & 1;
  bid >>= 1;
  const int head = bid % a.c.heads;
  bid /= a.c.heads;
  const int s = bid / a.items;
  const Span sp = span_of(a.b, s);
  void* const out = values ? a.v : a.k;
  if (!out) return;
  const int begin = sp.from, end = sp.from + sp.n;
  // pages of the rows before the sequence's beginning count as negative ones
  const int page = (begin >= 0 ? begin / kPage : -((-begin + kPage - 1) / kPage)) + bid % a.items;
  const int t0 = max(begin - page * kPage, 0), t1 = min(end - page * kPage, kPage);
  if (t0 >= t1) return;
  const int id = page < 0 ? -1 : page_of(a.b, a.c, s, page);
  const size_t at = (size_t)max(id, 0) * a.c.heads + head;
  const float scale = id < 0 ? 0.f : (values ? a.c.vs : a.c.ks)[at];
  const int64_t row0 = (int64_t)sp.first + page * kPage - sp.from;  // of token 0
  auto place = [&](int token, int d) { return ((row0 + token) * a.c.heads + head) * D + d; };
  if (values) {
    const int part = threadIdx.x / (D / 4), d0 = threadIdx.x % (D / 4) * 4;
    if (part >= 4) return;
    const kw4_t* const from = reinterpret_cast<const kw4_t*>(a.c.v + at * (kPage * D) + ((d0 / 16 * 4 + part) * 16 + d0 % 16) * 16);
    kw4_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = id < 0 ? kNone : from[e];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t in[4] = {w[0][q], w[1][q], w[2][q], w[3][q]};
      uint32_t tok[4];
      transpose4(in, tok);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int token = part * 16 + q * 4 + i;
        if (token < t0 || token >= t1) continue;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = (float)((int)((tok[i] >> (8 * e)) & 255u) - 128) * scale;
        if (F32)
          __builtin_nontemporal_store(kf4_t{v[0], v[1], v[2], v[3]}, reinterpret_cast<kf4_t*>((float*)out + place(token, d0)));
        else
          __builtin_nontemporal_store(kh4_t{(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]},
                                      reinterpret_cast<kh4_t*>((_Float16*)out + place(token, d0)));
      }
    }
    return;
  }
  constexpr int E = F32 ? 4 : 8;  // 16 bytes of a row a lane
  constexpr int kLanes = D / E, kRound = 256 / kLanes;
  const int d = threadIdx.x % kLanes * E;
#pragma unroll
  for (int i = 0; i < kPage / kRound; ++i) {
    const int token = i * kRound + threadIdx.x / kLanes;
    if (token < t0 || token >= t1) continue;
    const uint32_t* const from = reinterpret_cast<const uint32_t*>(
        a.c.k + at * (kPage * D) + ((d / 64 * 4 + token / 4 % 4) * 64 + d / 16 % 4 * 16 + token / 16 * 4 + token % 4) * 16 + d % 16);
    uint32_t w[E / 4];
#pragma unroll
    for (int q = 0; q < E / 4; ++q) w[q] = id < 0 ? kNone.x : from[q];
    float v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = (float)((int)((w[e / 4] >> (8 * (e % 4))) & 255u) - 128) * scale;
    if constexpr (F32) {
      __builtin_nontemporal_store(kf4_t{v[0], v[1], v[2], v[3]}, reinterpret_cast<kf4_t*>((float*)out + place(token, d)));
    } else {
      kh8_t h;
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = (_Float16)v[e];
      __builtin_nontemporal_store(h, reinterpret_cast<kh8_t*>((_Float16*)out + place(token, d)));
    }
  }
}

template <int D>
hipError_t write(const WriteArgs& a, long long blocks, hipStream_t s) {
  return kv_launch(kv_write_kernel<D>, dim3((unsigned)blocks), 256, s, a);
}
template <int D>
hipError_t read(const ReadArgs& a, long long blocks, hipStream_t s) {
  if (a.f32) return kv_launch(kv_read_kernel<D, true>, dim3((unsigned)blocks), 256, s, a);
  return kv_launch(kv_read_kernel<D, false>, dim3((unsigned)blocks), 256, s, a);
}

}  // namespace

hipError_t launch_kv_write(WriteArgs a, int dim, hipStream_t s) {
  a.q_waves = kv_waves((long long)a.b.count * a.b.max_rows, a.q_heads, dim / 8);
  const long long blocks = a.kv_blocks + (a.q ? ((long long)a.b.count * a.b.max_rows * a.q_waves + 3) / 4 : 0);
  if (!kv_grid_fits(blocks, 256)) return hipErrorInvalidConfiguration;
  if (dim == 64) return write<64>(a, blocks, s);
  return dim == 128 ? write<128>(a, blocks, s) : write<256>(a, blocks, s);
}

hipError_t launch_kv_read(const ReadArgs& a, int dim, hipStream_t s) {
  const long long blocks = 2ll * a.b.count * a.items * a.c.heads;
  if (!kv_grid_fits(blocks, 256)) return hipErrorInvalidConfiguration;
  if (dim == 64) return read<64>(a, blocks, s);
  return dim == 128 ? read<128>(a, blocks, s) : read<256>(a, blocks, s);
}

}  // namespace tern
