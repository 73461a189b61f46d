// Sums over the 64 lanes of a wave by data-parallel moves.
#pragma once

#include <hip/hip_runtime.h>

namespace ep {
namespace wave {

template <int CTRL, int ROWS>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xf, false));
}
// The sum over a wave, in lane 63: pairs, quads, halves and whole rows of 16 lanes, then the rows.
__device__ __forceinline__ float add_wave(float v) {
  v = add_dpp<0xb1, 0xf>(v);    // lanes 1 0 3 2 of each quad
  v = add_dpp<0x4e, 0xf>(v);    // lanes 2 3 0 1
  v = add_dpp<0x141, 0xf>(v);   // half rows mirrored
  v = add_dpp<0x140, 0xf>(v);   // rows mirrored
  v = add_dpp<0x142, 0xa>(v);   // each row's last lane to the next row
  return add_dpp<0x143, 0xc>(v);   // lane 31 to the upper rows
}

}  // namespace wave
}  // namespace ep
