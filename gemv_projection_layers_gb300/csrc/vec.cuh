// vec.cuh -- 16-byte vectors of bf16, fp16 or fp32 widened to fp32 and back,
// and block sums, shared by the norm and expert-sort kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace proj {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

// Round to nearest even, as every output of these kernels.
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// V consecutive elements: one 16-byte access where V fills it, else V = 1.
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T e[V];
};

template <typename T>
constexpr int kFullVec = 16 / static_cast<int>(sizeof(T));

template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load_vec(const T* p) {
  return *reinterpret_cast<const Vec<T, V>*>(p);
}

// Two values rounded at once, the first in the low half.
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[V]) {
  if constexpr (sizeof(T) == 2 && V >= 2) {
    Vec<uint32_t, V / 2> o;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) o.e[i] = pack2(v[2 * i], v[2 * i + 1], T());
    *reinterpret_cast<Vec<uint32_t, V / 2>*>(p) = o;
  } else {
    Vec<T, V> o;
#pragma unroll
    for (int i = 0; i < V; ++i) o.e[i] = from_f32<T>(v[i]);
    *reinterpret_cast<Vec<T, V>*>(p) = o;
  }
}

// The two values of a word, the low half first: one instruction each.
__device__ __forceinline__ void widen2(uint32_t w, float& x, float& y, __nv_bfloat16) {
  x = __uint_as_float(w << 16);
  y = __uint_as_float(w & 0xFFFF0000u);
}
__device__ __forceinline__ void widen2(uint32_t w, float& x, float& y, __half) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  x = f.x;
  y = f.y;
}

template <typename T, int V>
__device__ __forceinline__ void widen(const Vec<T, V>& a, float (&v)[V]) {
  if constexpr (sizeof(T) == 2 && V >= 2) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&a);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) widen2(w[i], v[2 * i], v[2 * i + 1], T());
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = to_f32(a.e[i]);
  }
}

// A pair of fp32 that one instruction multiplies and adds.
struct F2 {
  unsigned long long b;
};
__device__ __forceinline__ F2 f2(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.b) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ F2 f2(float x) { return f2(x, x); }
__device__ __forceinline__ void parts(F2 a, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a.b));
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.b) : "l"(a.b), "l"(b.b));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.b) : "l"(a.b), "l"(b.b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.b) : "l"(a.b), "l"(b.b), "l"(c.b));
  return r;
}
template <int E>
__device__ __forceinline__ void pairs(const float (&v)[E], F2 (&p)[E / 2]) {
#pragma unroll
  for (int i = 0; i < E / 2; ++i) p[i] = f2(v[2 * i], v[2 * i + 1]);
}
template <int E>
__device__ __forceinline__ void unpair(const F2 (&p)[E / 2], float (&v)[E]) {
#pragma unroll
  for (int i = 0; i < E / 2; ++i) parts(p[i], v[2 * i], v[2 * i + 1]);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Sums of NV values over the TPR threads that share a row: a warp's by
// shuffles, several warps' through `room` (2 x NV x 32 floats; `turn`
// alternates its halves, so one barrier per call is enough).  Every thread
// gets the same sums, in an order that depends on TPR alone.
template <int TPR, int NV>
__device__ __forceinline__ void row_sums(float (&v)[NV], float* room, int& turn) {
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = warp_sum(v[i]);
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    float* half = room + turn * NV * 32;
    turn ^= 1;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) half[i * 32 + warp] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float s = lane < W ? half[i * 32 + lane] : 0.f;
#pragma unroll
      for (int o = W >= 32 ? 16 : W / 2; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
      // lanes of every aligned group of W hold the group's sum; lane 0's is the row's
      v[i] = __shfl_sync(0xFFFFFFFFu, s, 0);
    }
  }
}

}  // namespace proj
