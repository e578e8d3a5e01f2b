// w4.cu -- products with 4-bit weights and group scales, for one matrix or a
// stack of experts: packing, and the weight-streaming kernel.
//
//   out[i, n] = sum_g s[n, g] sum_{k in g} (q[n, k] - z[n, g]) x[i, k]
//
// The weights are read once, as 4 bits; the kernel's floor is their bytes.
// Each product is one step of the warp-level MMA m16n8k16 with 16 weight rows
// on its M side and 8 tokens on its N side.  The integers q - z (at most five
// bits) are exact in bf16 and fp16, so a group's sum is the exact products'
// fp32 sum, and s multiplies that sum in fp32.
//
// Packed layout.  Rows in blocks of 16, columns in units of 64.  Lane
// l = 4 g + t of the warp that reads unit (rb, u) holds columns
// 64 u + 32 h + 8 t + 0..7 (h = 0, 1) of rows 16 rb + g and + 8: 16 bytes,
// [h0 row g][h0 row g + 8][h1 row g][h1 row g + 8], at (rb KU + u) 512 + 16 l.
// One load of a lane is four A fragments: the order of columns within a unit
// is free as long as x follows it, and with this one the B fragments of two
// steps are 16 consecutive bytes of an x row.  In each 32-bit word column
// 2 i stands at bit 4 i and column 2 i + 1 at bit 16 + 4 i, so one shift and
// one mask give a pair of 16-bit lanes.  Scales and zeros: [rb][group][g]{row
// g, row g + 8}.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdio>
#include <new>

#include "../../include/proj.h"
#include "kernels.h"
#include "ptx.cuh"
#include "vec.cuh"
#include "w4.h"

namespace proj {
namespace {

// ---------------------------------------------------------------- packing --

__device__ __forceinline__ uint32_t code_at(const uint8_t* row, int64_t k, int64_t K) {
  if (k >= K) return 0u;  // meets x = 0
  const uint32_t b = row[k >> 1];
  return (k & 1) ? b >> 4 : b & 15u;
}

// One thread per 16-byte lane record.
__global__ void pack_codes_kernel(const uint8_t* __restrict__ codes, uint4* __restrict__ dst,
                                  int64_t E, int64_t N, int64_t K, int64_t RB, int64_t KU) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= E * RB * KU * 32) return;
  const int lane = static_cast<int>(i & 31);
  const int64_t u = (i >> 5) % KU;
  const int64_t rb = (i >> 5) / KU % RB;
  const int64_t e = (i >> 5) / KU / RB;
  const int g = lane >> 2, t = lane & 3;
  const int64_t bytes = (K + 1) / 2;
  uint32_t w[4];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int hi = 0; hi < 2; ++hi) {
      const int64_t n = rb * 16 + g + 8 * hi;
      uint32_t v = 0;
      if (n < N) {
        const uint8_t* row = codes + (e * N + n) * bytes;
        const int64_t k0 = u * 64 + 32 * h + 8 * t;
#pragma unroll
        for (int c = 0; c < 8; ++c)
          v |= code_at(row, k0 + c, K) << ((c & 1) * 16 + (c >> 1) * 4);
      }
      w[2 * h + hi] = v;
    }
  dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
}

// One thread per packed scale.  Groups beyond K and rows beyond N get 0.
__global__ void pack_scales_kernel(const uint16_t* __restrict__ scales,
                                   const uint8_t* __restrict__ zeros, uint16_t* __restrict__ ds,
                                   uint8_t* __restrict__ dz, int64_t E, int64_t N, int64_t NG,
                                   int64_t NGp, int64_t RB) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= E * RB * NGp * 16) return;
  const int r = static_cast<int>(i & 15);
  const int64_t grp = (i >> 4) % NGp;
  const int64_t rb = (i >> 4) / NGp % RB;
  const int64_t e = (i >> 4) / NGp / RB;
  const int64_t n = rb * 16 + (r >> 1) + 8 * (r & 1);
  const bool in = n < N && grp < NG;
  const int64_t src = (e * N + n) * NG + grp;
  ds[i] = in ? scales[src] : 0;
  if (dz) dz[i] = in ? static_cast<uint8_t>(zeros[src] & 15) : 0;
}

// ------------------------------------------------------ streaming kernel --

template <typename T>
struct Num;
template <>
struct Num<__nv_bfloat16> {
  static constexpr uint32_t kMagic = 0x43004300u;  // 128 + q in a pair's low mantissa bits
  static __device__ __forceinline__ uint32_t offset(uint32_t z) {  // 128 + z, twice
    return (0x4300u + z) * 0x10001u;
  }
  static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};
template <>
struct Num<__half> {
  static constexpr uint32_t kMagic = 0x64006400u;  // 1024 + q
  static __device__ __forceinline__ uint32_t offset(uint32_t z) {
    return (0x6400u + z) * 0x10001u;
  }
  static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

// Eight consecutive x values of a row from column c; zeros from K on.
template <typename T>
__device__ __forceinline__ uint4 load_x8(const T* row, int c, int K) {
  if (c + 8 <= K) return *reinterpret_cast<const uint4*>(row + c);
  uint4 v = make_uint4(0, 0, 0, 0);
  uint32_t* w = reinterpret_cast<uint32_t*>(&v);
  const uint16_t* r = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < K) w[i >> 1] |= static_cast<uint32_t>(r[c + i]) << (16 * (i & 1));
  return v;
}

struct Tile {
  int expert;
  int64_t row0;
  int rows;
};

// Token tile `index` of the experts' rows (tiles of T rows, expert by
// expert).  Offsets are clamped to 0 .. m and taken as not decreasing, so no
// row outside x is ever named.  Returns rows = 0 beyond the last tile.  All
// threads of the block call it.
template <int kThreads>
__device__ __forceinline__ Tile find_tile(const int32_t* __restrict__ offsets, int E, int64_t m,
                                          int T, int index) {
  __shared__ int s_sum[32];
  __shared__ int s_found[3];
  constexpr int W = kThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lim = static_cast<int>(m);
  if (threadIdx.x == 0) s_found[2] = 0;
  int carry = 0;
  for (int e0 = 0; e0 < E; e0 += kThreads) {
    const int e = e0 + threadIdx.x;
    int lo = 0, hi = 0;
    if (e < E) {
      lo = min(max(__ldg(offsets + e), 0), lim);
      hi = min(max(__ldg(offsets + e + 1), lo), lim);
    }
    const int tiles = (hi - lo + T - 1) / T;
    int inc = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += v;
    }
    __syncthreads();
    if (lane == 31) s_sum[warp] = inc;
    __syncthreads();
    int before = carry;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const int v = s_sum[w];
      if (w < warp) before += v;
      carry += v;
    }
    const int first = before + inc - tiles;
    if (index >= first && index < first + tiles) {
      const int r0 = lo + (index - first) * T;
      s_found[0] = e;
      s_found[1] = r0;
      s_found[2] = min(T, hi - r0);
    }
  }
  __syncthreads();
  return {s_found[0], s_found[1], s_found[2]};
}

// A CTA takes one block of 16 weight rows and one tile of 8 NT tokens; its W
// warps split the units of K (warp w: units w, w + W, ...) and meet in
// shared memory.
template <typename T, bool kG32, bool kZeros, int NT, int W>
__global__ void __launch_bounds__(32 * W) w4_stream_kernel(const W4Params p) {
  __shared__ alignas(16) float s_red[W][NT][32][4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int rb = blockIdx.x;
  griddep_launch_dependents();
  griddep_wait();
  Tile tile;
  if (p.offsets) {
    tile = find_tile<32 * W>(p.offsets, p.E, p.m, 8 * NT, blockIdx.y);
    if (tile.rows == 0) return;
  } else {
    tile.expert = 0;
    tile.row0 = static_cast<int64_t>(blockIdx.y) * 8 * NT;
    tile.rows = static_cast<int>(min(static_cast<int64_t>(8 * NT), p.m - tile.row0));
  }
  const int64_t block = static_cast<int64_t>(tile.expert) * p.RB + rb;
  const uint4* codes = p.codes + block * p.KU * 32 + lane;
  const uint32_t* scales = reinterpret_cast<const uint32_t*>(p.scales) + block * p.NGp * 8 + g;
  const uint16_t* zeros = reinterpret_cast<const uint16_t*>(p.zeros) + block * p.NGp * 8 + g;
  const T* x = static_cast<const T*>(p.x) + tile.row0 * p.ldx;

  float acc[NT][4] = {};
  const int upg = kG32 ? 1 : p.group / 64;  // units per group
#pragma unroll 4
  for (int u = warp; u < p.KU; u += W) {
    const uint4 q = ld_stream_v4(codes + static_cast<int64_t>(u) * 32);
    const uint32_t word[4] = {q.x, q.y, q.z, q.w};
    float part[NT][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int grp = kG32 ? 2 * u + h : u / upg;
      uint32_t off[2] = {Num<T>::offset(8), Num<T>::offset(8)};
      if (kZeros) {
        const uint32_t z = __ldg(zeros + grp * 8);
        off[0] = Num<T>::offset(z & 255u);
        off[1] = Num<T>::offset(z >> 8);
      }
      uint32_t a[2][4];
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int hi = i & 1, pair = 2 * s + (i >> 1);
          a[s][i] = Num<T>::sub(((word[2 * h + hi] >> (4 * pair)) & 0x000F000Fu) | Num<T>::kMagic,
                                off[hi]);
        }
      if (kG32 || h == 0) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) part[j][i] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        uint4 b = make_uint4(0, 0, 0, 0);
        if (8 * j + g < tile.rows)
          b = load_x8(x + static_cast<int64_t>(8 * j + g) * p.ldx, u * 64 + 32 * h + 8 * t, p.K);
        Num<T>::mma(part[j], a[0], b.x, b.y);
        Num<T>::mma(part[j], a[1], b.z, b.w);
      }
      if (kG32 || h == 1) {
        const uint32_t sp = __ldg(scales + grp * 8);
        const float s0 = to_f32(reinterpret_cast<const T*>(&sp)[0]);
        const float s1 = to_f32(reinterpret_cast<const T*>(&sp)[1]);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          acc[j][0] = fmaf(s0, part[j][0], acc[j][0]);
          acc[j][1] = fmaf(s0, part[j][1], acc[j][1]);
          acc[j][2] = fmaf(s1, part[j][2], acc[j][2]);
          acc[j][3] = fmaf(s1, part[j][3], acc[j][3]);
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j)
    *reinterpret_cast<float4*>(s_red[warp][j][lane]) =
        make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
  __syncthreads();
  // sum the warps' partials in order; element i of lane l is row g + 8 (i / 2),
  // token 2 t + i % 2
  T* out = static_cast<T*>(p.out);
  for (int i = threadIdx.x; i < NT * 128; i += 32 * W) {
    const int n16 = i & 15, tok = i >> 4;
    const int l = (n16 & 7) * 4 + ((tok & 7) >> 1);
    const int c = (n16 >> 3) * 2 + (tok & 1);
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) s += s_red[w][tok >> 3][l][c];
    const int64_t n = static_cast<int64_t>(rb) * 16 + n16;
    if (tok < tile.rows && n < p.N) out[(tile.row0 + tok) * p.ldo + n] = from_f32<T>(s);
  }
}

template <typename T, bool kG32, bool kZeros, int NT, int W>
cudaError_t stream_launch(const W4Params& p, int64_t tiles, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.RB), static_cast<unsigned>(tiles));
  cfg.blockDim = dim3(32 * W);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, w4_stream_kernel<T, kG32, kZeros, NT, W>, p);
}

template <typename T, int NT, int W>
cudaError_t stream_form(const W4Params& p, int64_t tiles, cudaStream_t s) {
  if (p.group == 32)
    return p.zeros ? stream_launch<T, true, true, NT, W>(p, tiles, s)
                   : stream_launch<T, true, false, NT, W>(p, tiles, s);
  return p.zeros ? stream_launch<T, false, true, NT, W>(p, tiles, s)
                 : stream_launch<T, false, false, NT, W>(p, tiles, s);
}

template <typename T>
cudaError_t stream_any(int nt, const W4Params& p, int64_t tiles, cudaStream_t s) {
  switch (nt) {
    case 1: return stream_form<T, 1, 8>(p, tiles, s);
    case 2: return stream_form<T, 2, 8>(p, tiles, s);
    default: return stream_form<T, 4, 8>(p, tiles, s);
  }
}

int refuse(int status, const char* call, const char* why) {
  char text[160];
  std::snprintf(text, sizeof text, "%s: %s", call, why);
  return record_status(status, text);
}

bool aligned_to(const void* p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace
}  // namespace proj

using namespace proj;

struct proj_w4_ctx {
  W4Params p;       // sizes and the packed weights; x, out, offsets are each call's
  int dtype;
  uint8_t* base;    // one allocation: codes, scales, zeros, status word
};

namespace {

// Token tiles of a call: 8 rows each while a matrix meets few rows, 32 rows
// at most (the rows an expert meets on average, for a stack of experts).
int stream_nt(const proj_w4_ctx* h, int64_t m, bool experts) {
  const int64_t rows = experts ? (m + h->p.E - 1) / h->p.E : m;
  return rows <= 8 ? 1 : (rows <= 16 ? 2 : 4);
}

int run(const char* call, proj_w4_handle h, const void* x, int64_t ldx, int64_t m,
        const int32_t* offsets, bool experts, void* out, int64_t ldo, proj_stream stream) {
  if (!h) return refuse(PROJ_EINVAL, call, "NULL handle");
  if (m < 0 || ldx < h->p.K || ldo < h->p.N)
    return refuse(PROJ_EINVAL, call, "m < 0, or a row stride below K or N");
  if (!experts && h->p.E != 1)
    return refuse(PROJ_EINVAL, call, "the handle holds several experts");
  if (m > (int64_t{1} << 20) || ldx >= (int64_t{1} << 38) || ldo >= (int64_t{1} << 38))
    return refuse(PROJ_EUNSUPPORTED, call, "m > 2^20 or a row stride >= 2^38");
  if (m > 0 && (!x || !out || (experts && !offsets)))
    return refuse(PROJ_EINVAL, call, "a NULL pointer");
  if (!aligned_to(x, 16) || ldx % 8)
    return refuse(PROJ_EALIGN, call, "x is not 16-byte aligned, or ldx not a multiple of 8");
  if (!aligned_to(out, 2) || !aligned_to(offsets, 4))
    return refuse(PROJ_EALIGN, call, "out or offsets is not aligned to an element");
  if (m == 0) return PROJ_OK;
  W4Params p = h->p;
  p.x = x;
  p.ldx = ldx;
  p.m = m;
  p.out = out;
  p.ldo = ldo;
  p.offsets = experts ? offsets : nullptr;
  const int nt = stream_nt(h, m, experts);
  const int64_t per = 8 * nt;
  // tiles of the experts: at most one part-filled tile for each that has rows
  const int64_t tiles =
      experts ? std::min<int64_t>(p.E, m) + m / per : (m + per - 1) / per;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = h->dtype == PROJ_BF16 ? stream_any<__nv_bfloat16>(nt, p, tiles, s)
                                              : stream_any<__half>(nt, p, tiles, s);
  return e == cudaSuccess ? PROJ_OK : record_cuda(e, call);
}

}  // namespace

extern "C" proj_w4_handle proj_w4_prepare(const void* codes, const void* scales, const void* zeros,
                                          int64_t experts, int64_t N, int64_t K, int64_t group,
                                          int dtype, int* status) {
  const char* const call = "proj_w4_prepare";
  auto refused = [&](int st, const char* why) -> proj_w4_handle {
    refuse(st, call, why);
    if (status) *status = st;
    return nullptr;
  };
  if (!codes || !scales) return refused(PROJ_EINVAL, "codes or scales is NULL");
  if (experts < 1 || N < 1 || K < 1) return refused(PROJ_EINVAL, "experts, N or K is below 1");
  if (group != 32 && (group < 64 || group % 64))
    return refused(PROJ_EINVAL, "group is neither 32 nor a multiple of 64");
  if (dtype != PROJ_BF16 && dtype != PROJ_FP16)
    return refused(PROJ_EINVAL, "dtype is neither PROJ_BF16 nor PROJ_FP16");
  constexpr int64_t kMost = int64_t{1} << 20;
  if (experts > 1024 || N > kMost || K > kMost || group > kMost)
    return refused(PROJ_EUNSUPPORTED, "experts > 1024, or N, K or group > 2^20");
  if (!aligned_to(scales, 2)) return refused(PROJ_EALIGN, "scales is not aligned to an element");
  proj_w4_ctx* h = new (std::nothrow) proj_w4_ctx();
  if (!h) return refused(PROJ_ENOMEM, "no host memory");
  W4Params& p = h->p;
  p.E = static_cast<int>(experts);
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.group = static_cast<int>(group);
  p.RB = static_cast<int>((N + 15) / 16);
  p.KU = static_cast<int>((K + 63) / 64);
  const int64_t NG = (K + group - 1) / group;
  p.NGp = static_cast<int>(group == 32 ? 2 * p.KU : NG);  // every unit has its groups
  h->dtype = dtype;
  const int64_t blocks = experts * p.RB;
  const int64_t code_bytes = blocks * p.KU * 512;
  const int64_t scale_bytes = (blocks * p.NGp * 32 + 255) / 256 * 256;
  const int64_t zero_bytes = zeros ? (blocks * p.NGp * 16 + 255) / 256 * 256 : 0;
  cudaError_t e = cudaMalloc(reinterpret_cast<void**>(&h->base),
                             static_cast<size_t>(code_bytes + scale_bytes + zero_bytes + 256));
  if (e != cudaSuccess) {
    cudaGetLastError();
    delete h;
    record_cuda(e, call);
    refuse(PROJ_ENOMEM, call, "device memory for the packed weights");
    if (status) *status = PROJ_ENOMEM;
    return nullptr;
  }
  p.codes = reinterpret_cast<const uint4*>(h->base);
  p.scales = reinterpret_cast<const uint16_t*>(h->base + code_bytes);
  p.zeros = zeros ? h->base + code_bytes + scale_bytes : nullptr;
  p.status = reinterpret_cast<uint32_t*>(h->base + code_bytes + scale_bytes + zero_bytes);
  const int64_t lanes = blocks * p.KU * 32, cells = blocks * p.NGp * 16;
  pack_codes_kernel<<<static_cast<unsigned>((lanes + 255) / 256), 256>>>(
      static_cast<const uint8_t*>(codes), const_cast<uint4*>(p.codes), experts, N, K, p.RB, p.KU);
  pack_scales_kernel<<<static_cast<unsigned>((cells + 255) / 256), 256>>>(
      static_cast<const uint16_t*>(scales), static_cast<const uint8_t*>(zeros),
      const_cast<uint16_t*>(p.scales), const_cast<uint8_t*>(p.zeros), experts, N, NG, p.NGp, p.RB);
  e = cudaGetLastError();
  if (e == cudaSuccess) e = cudaMemsetAsync(p.status, 0, 4, nullptr);
  if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
  if (e != cudaSuccess) {
    record_cuda(e, call);
    cudaFree(h->base);
    delete h;
    if (status) *status = PROJ_ECUDA;
    return nullptr;
  }
  if (status) *status = PROJ_OK;
  return h;
}

extern "C" int proj_w4_run(proj_w4_handle h, const void* x, int64_t ldx, int64_t m, void* out,
                           int64_t ldo, proj_stream stream) {
  return run("proj_w4_run", h, x, ldx, m, nullptr, false, out, ldo, stream);
}

extern "C" int proj_w4_run_experts(proj_w4_handle h, const void* x, int64_t ldx, int64_t m,
                                   const int32_t* offsets, void* out, int64_t ldo,
                                   proj_stream stream) {
  return run("proj_w4_run_experts", h, x, ldx, m, offsets, true, out, ldo, stream);
}

extern "C" int proj_w4_describe(proj_w4_handle h, int64_t m, char* buf, size_t cap) {
  if (!h || !buf || cap == 0 || m < 0)
    return refuse(PROJ_EINVAL, "proj_w4_describe", "NULL handle or buffer, cap = 0 or m < 0");
  std::snprintf(buf, cap, "w4 stream, %d tokens a tile, exact 4-bit products",
                8 * stream_nt(h, m, h->p.E > 1));
  return PROJ_OK;
}

extern "C" int proj_w4_device_status(proj_w4_handle h, proj_stream stream, uint32_t* code) {
  const char* const call = "proj_w4_device_status";
  if (!h) return refuse(PROJ_EINVAL, call, "NULL handle");
  uint32_t word = 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemcpyAsync(&word, h->p.status, 4, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(h->p.status, 0, 4, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return record_cuda(e, call);
  if (code) *code = word;
  return word ? refuse(PROJ_EDEVICE, call, "a kernel recorded a fault") : PROJ_OK;
}

extern "C" void proj_w4_destroy(proj_w4_handle h) {
  if (!h) return;
  cudaDeviceSynchronize();
  cudaFree(h->base);
  delete h;
}
