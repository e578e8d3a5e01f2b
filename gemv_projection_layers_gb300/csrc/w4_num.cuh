// w4_num.cuh -- 4-bit numbers to pairs of bf16 or fp16, and their products.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace proj {

// A pair of 16-bit floats with q in the low mantissa bits of a power of two
// (128 for bf16, 1024 for fp16: one unit of the last place is 1) is that
// power + q; subtracting power + z leaves q - z exactly.
template <typename T>
struct Num;

template <>
struct Num<__nv_bfloat16> {
  static constexpr uint32_t kPower = 0x4300u;
  static constexpr uint32_t kIdescType = (1u << 7) | (1u << 10);  // A and B bf16
  static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ uint32_t mul(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  static __device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4],
                                                   uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
  }
};

template <>
struct Num<__half> {
  static constexpr uint32_t kPower = 0x6400u;
  static constexpr uint32_t kIdescType = 0u;  // A and B fp16
  static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ uint32_t mul(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  static __device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4],
                                                   uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
  }
};

// power + z in both halves of a pair, z the byte `which` of `zeros` (the
// power's low byte is zero, so this is one byte permutation).
template <typename T>
__device__ __forceinline__ uint32_t zero_pair(uint32_t zeros, int which) {
  return __byte_perm(zeros, Num<T>::kPower >> 8, which ? 0x4141 : 0x4040);
}

// Columns 2 i and 2 i + 1 of a packed word as the pair q - z.
template <typename T>
__device__ __forceinline__ uint32_t code_pair(uint32_t word, int i, uint32_t zero) {
  return Num<T>::sub(((word >> (4 * i)) & 0x000F000Fu) | (Num<T>::kPower * 0x10001u), zero);
}

// What a lane loads of the scales and zeros of a unit of 64 columns: one pair
// (rows g and g + 8), or one for each half where groups have 32 columns.
template <bool kG32>
struct ScaleOf {
  using Pair = uint32_t;
  using Bytes = uint16_t;
  static __device__ __forceinline__ uint32_t pair(uint32_t v, int) { return v; }
  static __device__ __forceinline__ uint32_t bytes(uint16_t v, int) { return v; }
};
template <>
struct ScaleOf<true> {
  using Pair = uint2;
  using Bytes = uint32_t;
  static __device__ __forceinline__ uint32_t pair(uint2 v, int h) { return h ? v.y : v.x; }
  static __device__ __forceinline__ uint32_t bytes(uint32_t v, int h) { return h ? v >> 16 : v; }
};

}  // namespace proj
