// w4.h -- what the kernels of the 4-bit products share (w4.cu has the packed
// layout).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace proj {

struct W4Params {
  const uint4* codes;      // [E][RB][KU][32 lanes] of 16 bytes
  const uint16_t* scales;  // [E][RB][NGp][8]{row g, row g + 8}
  const uint8_t* zeros;    // the same in bytes, or null: all 8
  uint32_t* status;
  const void* x;
  void* out;
  const int32_t* offsets;  // [E + 1], or null: one matrix
  int64_t ldx, ldo, m;
  int E, N, K;
  int group;
  int RB;   // blocks of 16 rows
  int KU;   // units of 64 columns
  int NGp;  // groups per row block in the packed scales
};

}  // namespace proj
