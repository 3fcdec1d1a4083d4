// Scale atoms of the microscaled formats (MXFP8, MXFP4): the scales of 128
// rows x 128 columns form 512 bytes, row i's four blocks of 32 columns at byte
// 16 (i % 32) + 4 (i / 32); atoms are ordered (128-row tile, 128 columns),
// columns fastest, and a group's (expert's) rows start a new tile.
#pragma once

#include "common.cuh"

namespace moe {
namespace mx {

constexpr int ATOM = 512;

// Byte offset of row i's scale word (blocks j = 0..3) in atom (tile, kb).
MOE_HD int64_t atom_word(int64_t tile, int KB, int kb, int i) {
  return (tile * KB + kb) * ATOM + 16 * (i & 31) + 4 * (i >> 5);
}

// E8M0 code c -> 2^(c - 127) (255 is NaN, 0 the subnormal 2^-127).
MOE_D float e8m0_value(uint32_t c) {
  return __uint_as_float(c == 255u ? 0x7fc00000u : (c ? c << 23 : 0x00400000u));
}

// The group boundaries off[0 .. G] in shared memory, kept within the rows, and
// the 128-row tiles before each group, rt[0 .. G] (an exclusive scan of
// ceil(rows_g / 128)).  Every thread of the block calls it.
MOE_D void load_groups(const int32_t* __restrict__ offsets, int G, int rows, int* off, int* rt) {
  for (int g = threadIdx.x; g <= G; g += blockDim.x) off[g] = min(max(__ldg(offsets + g), 0), rows);
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int running = 0;
    for (int g0 = 0; g0 < G; g0 += 32) {
      const int g = g0 + lane;
      const int v = g < G ? (max(off[g + 1] - off[g], 0) + 127) / 128 : 0;
      int incl = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      if (g < G) rt[g] = running + incl - v;
      running += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) rt[G] = running;
  }
  __syncthreads();
}

}  // namespace mx
}  // namespace moe
