// kv_num.cuh -- the cache's 8-bit codes: fp32 to codes, and codes to pairs of
// fp16, which holds every one of them exactly.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

#include "../../include/proj.h"

namespace proj {

// Four codes, the first in the low byte; to nearest even, held to the range.
template <int kFormat>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  if constexpr (kFormat == PROJ_KV_E4M3) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
  } else {
    // 1.5 2^23 leaves whole numbers in the low bits, rounded to nearest even
    constexpr float kWhole = 12582912.f;
    const uint32_t x = __float_as_uint(a + kWhole), y = __float_as_uint(b + kWhole);
    const uint32_t z = __float_as_uint(c + kWhole), w = __float_as_uint(d + kWhole);
    return __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
  }
}

// Two codes of the low 16 bits, the lower byte to the lower half.
__device__ __forceinline__ uint32_t e4m3_pair(uint16_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(codes));
  return r;
}

// Signed bytes, taken by `pick` from word ^ 0x80808080 under the high byte
// 0x64: the fp16 number 1024 + byte + 128, less 1152.
__device__ __forceinline__ uint32_t int8_pair(uint32_t word, uint32_t pick) {
  uint32_t u;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(u) : "r"(word ^ 0x80808080u), "r"(0x64u), "r"(pick));
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&u), __half2half2(__ushort_as_half(0x6480)));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Bytes 0, 1 (which = 0) or 2, 3 (which = 1) of a word as fp16.
template <int kFormat>
__device__ __forceinline__ uint32_t decode_pair(uint32_t word, int which) {
  if constexpr (kFormat == PROJ_KV_E4M3)
    return e4m3_pair(static_cast<uint16_t>(which ? word >> 16 : word));
  else
    return int8_pair(word, which ? 0x4342u : 0x4140u);
}

// Bytes 0, 2 and bytes 1, 3.
template <int kFormat>
__device__ __forceinline__ void decode_cross(uint32_t word, uint32_t& even, uint32_t& odd) {
  if constexpr (kFormat == PROJ_KV_E4M3) {
    uint32_t s;
    asm("prmt.b32 %0, %1, %1, 0x3120;" : "=r"(s) : "r"(word));
    even = e4m3_pair(static_cast<uint16_t>(s));
    odd = e4m3_pair(static_cast<uint16_t>(s >> 16));
  } else {
    even = int8_pair(word, 0x4240u);
    odd = int8_pair(word, 0x4341u);
  }
}

}  // namespace proj
