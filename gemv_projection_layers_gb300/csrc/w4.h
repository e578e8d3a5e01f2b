// w4.h -- what the kernels of the 4-bit products share (w4.cu has the packed
// layout).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace proj {

constexpr int kW4MaxExperts = 1024;
constexpr int kW4UnitBytes = 4096;  // codes of 128 rows x 64 columns

struct W4Params {
  const uint4* codes;      // [E][RT][KU][8 blocks][32 lanes] of 16 bytes
  const uint16_t* scales;  // [E][RT][NGp][8 blocks][8]{row g, row g + 8}
  const uint8_t* zeros;    // the same in bytes, or null: all 8
  uint32_t* status;
  const void* x;
  void* out;
  const int32_t* offsets;  // [E + 1], or null: one matrix
  int64_t ldx, ldo, m;
  int E, N, K;
  int group;
  int RB;   // blocks of 16 rows
  int RT;   // tiles of 128 rows
  int KU;   // units of 64 columns
  int NGp;  // groups per row block in the packed scales
  // ceil(2^31 / d) for the d = group / 64 units of a group: exact quotients
  // while u and d are at most 2^14, without a division.
  uint32_t group_magic;
  __device__ int group_of(int u) const {  // groups of 64 columns or more
    return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(u)) * group_magic) >> 31);
  }
};

// The tensor-core kernel (w4_tc.cu): token tiles of tn = 64, 128 or, without
// offsets, 256; clusters of C CTAs along K (C > 1: grid = C times the most items
// that a call of that size can have).
cudaError_t w4_tc_launch(bool fp16, int tn, const W4Params& p, int64_t grid, int C,
                         cudaStream_t s);

int w4_tc_max_clusters(int C);  // that run at once (occupancy query)

// api.cu
bool make_rows_map(CUtensorMap* map, const void* base, int64_t rows, int64_t K, int64_t ld,
                   bool fp16, int box_rows);

}  // namespace proj
