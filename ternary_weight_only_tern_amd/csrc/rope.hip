// Rotary positions: pairs of a head's values turned by pos * freq, after an
// optional norm of the head (tern_rope in tern.h).
//
// Eight values (16 bytes) a lane; a head's lanes are neighbours in one
// wavefront, so that the norm's sum needs shuffles alone and out may equal x:
// the wavefront has read a head before it writes it.  In the half layout the
// pair's other value is read a second time (from the cache) instead of
// shuffled.  A workgroup of many rows walks the heads of its row, its angles
// computed once; for few rows every head has its own lanes.
#include "kv.h"

namespace tern {
namespace {

__global__ __launch_bounds__(256) void rope_kernel(const RopeArgs a, int lanes) {
  const int row = blockIdx.x, slots = 256 / lanes;
  const int lane = threadIdx.x % lanes, d0 = lane * 8;
  const bool live = d0 < a.dim;
  const int pos = a.pos[row];
  for (int h0 = blockIdx.y * slots; h0 < a.heads; h0 += gridDim.y * slots) {
    const int h = h0 + threadIdx.x / lanes;
    const bool there = live && h < a.heads;
    float y[8];
    turned<8>(a.x + row * a.x_stride + (int64_t)h * a.dim, d0, a.dim, there, lanes, a.r, pos, y);
    kh8_t o;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = (_Float16)y[e];
    if (there) *reinterpret_cast<kh8_t*>(a.out + row * a.out_stride + (int64_t)h * a.dim + d0) = o;
  }
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, hipStream_t s) {
  int lanes = 1;
  while (lanes * 8 < a.dim) lanes *= 2;
  const int groups = (a.heads * lanes + 255) / 256;
  const int y = a.m < 512 ? groups : 1;
  if (!kv_grid_fits((long long)a.m * y, 256)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(rope_kernel, dim3((unsigned)a.m, (unsigned)y), dim3(256), 0, s, a, lanes);
  return hipGetLastError();
}

}  // namespace tern
