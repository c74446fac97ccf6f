// Device code of the 4-bit products for few activation rows: staging and
// multiplying K tiles.
#pragma once

#include "q4.h"

namespace tern {

constexpr uint32_t kFar = 0x80000000u;  // an offset past every buffer here (2 GiB at most)

// p and bytes are the same in every lane; said so explicitly, or a descriptor
// that the compiler cannot prove uniform costs a loop around every load.
__device__ inline __amdgpu_buffer_rsrc_t q4_buffer(const void* p, uint32_t bytes) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>((uint64_t)hi << 32 | lo), (short)0,
                                           __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000);
}

// 16 bytes per lane from a buffer straight into LDS: lane l writes dst + l.
__device__ inline void q4_stage16(__amdgpu_buffer_rsrc_t r, w4_t* dst, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 16, off, 0, 0, 0);
}

// A wavefront's staging buffer is its own: no barrier, but its staged loads
// must have arrived before they are read, and its reads have returned before
// the next loads are issued.
__device__ inline void q4_loads_done() {
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}
__device__ inline void q4_reads_done() {
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
}

// Row r's 16-byte chunk c of a staged K tile's codes lies at 4 r + (c ^
// swizzle), so that the 16 rows of an operand read fall in distinct banks.
__device__ inline int code_chunk(int r, int c) { return r * 4 + (c ^ ((r >> 1) & 3)); }

// The 16-byte chunk of a K tile of x that instruction i multiplies on a lane.
template <int G>
__device__ inline int x_chunk(int i, int kq) {
  return G == 128 ? kq * 4 + i : i * 4 + kq;
}

// This lane's codes of one K tile, word i for instruction i.  Group 128: the
// four lanes that hold a row's tile multiply 32 consecutive k each.  Smaller
// groups need every instruction's 32 k inside one group, so the four lanes'
// words are transposed: four operations per 16 bytes.
template <int G>
__device__ inline w4_t in_order(w4_t v) {
  if (G == 128) return v;
  uint32_t w[4] = {v.x, v.y, v.z, v.w};  // word i of lane quarter q <- word q of lane quarter i
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
  return w4_t{w[0], w[1], w[2], w[3]};
}

}  // namespace tern
