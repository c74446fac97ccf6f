// Rotary positions: pairs of a head's values turned by pos * freq, after an
// optional norm of the head (tern_rope in tern.h).
//
// A lane holds eight values, in the half layout both sides of four pairs (kv.h);
// a head's lanes are neighbours in one wavefront, so that the norm's sum needs
// shuffles alone and out may equal x: the wavefront has read a head before it
// writes it.  A wavefront walks the heads of a row, its angles computed once;
// for few rows the heads are spread over more wavefronts.
//
// Bound by the bytes of x and out where rows are many: 5000 rows of 32 heads of
// 128, half of each turned, 14.7 us, 5.6 TB/s read and written.  One row of 40
// heads: 3.0-3.2 us, a trip to memory and the angles' FP64 behind an empty kernel's 1.9.
#include "kv.h"

namespace tern {
namespace {

__global__ __launch_bounds__(256) void rope_kernel(const RopeArgs a, int lanes, int waves) {
  const int64_t wave = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
  const int64_t row = wave / waves;
  if (row >= a.m) return;
  const int per = 64 / lanes;
  turn_row(a.x + row * a.x_stride, a.out + row * a.out_stride, a.heads, a.dim, lanes, (int)(wave % waves) * per, waves * per, a.r,
           a.pos[row]);
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, hipStream_t s) {
  int lanes = 1;
  while (lanes * 8 < a.dim) lanes *= 2;
  const int waves = kv_waves(a.m, a.heads, lanes);
  const long long blocks = ((long long)a.m * waves + 3) / 4;
  if (!kv_grid_fits(blocks, 256)) return hipErrorInvalidConfiguration;
  return kv_launch(rope_kernel, dim3((unsigned)blocks), 256, s, a, lanes, waves);
}

}  // namespace tern
