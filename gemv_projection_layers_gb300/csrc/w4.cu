// w4.cu -- products with 4-bit weights and group scales, for one matrix or a
// stack of experts: packing, and the weight-streaming kernel.
//
//   out[i, n] = sum_g s[n, g] sum_{k in g} (q[n, k] - z[n, g]) x[i, k]
//
// The weights are read once, as 4 bits; the kernel's floor is their bytes.
// The streaming kernel stays above it for two reasons of about equal weight: the
// decode, some 200 instructions a warp for 32 rows x 64 columns (44 to make the
// operands of one block of 16 rows, the MMAs, the scales, the loads), and the
// latency of loads that go straight to registers, which the 16 warps that 128
// registers leave an SM do not hide: they issue on one cycle in two.  (4096 x
// 8192, groups of 128, 8 tokens: 10.0 us with the weights in HBM, 8.7 in L2,
// where its bf16 form takes 13.1; 8192 x 1024, 1 token: 3.4 and 3.0 us, where a
// launch alone is 2.6; 64 rows over 256 experts of 1024 x 8192: 75 us, 3.3
// TB/s.)
// Each product is one step of the warp-level MMA m16n8k16 with 16 weight rows
// on its M side and 8 tokens on its N side.  The integers q - z (at most five
// bits) are exact in bf16 and fp16, so a group's sum is the exact products'
// fp32 sum, and s multiplies that sum in fp32.
//
// Packed layout.  Rows in blocks of 16, eight blocks a tile, columns in units
// of 64.  Lane l = 4 g + t of the warp that reads unit u of block b of tile rt
// holds columns 64 u + 32 h + 16 s + 4 t + 0..3 (h, s = 0, 1) of the block's
// rows g and g + 8: 16 bytes, [h0 row g][h0 row g + 8][h1 row g][h1 row g + 8],
// at ((rt KU + u) 8 + b) 512 + 16 l.
// One load of a lane is four A fragments: the order of columns within a step
// of 16 is free as long as x follows it, and with this one a lane's B fragment
// is 8 consecutive bytes of an x row, and its A words are those that a
// 16-lane store to tensor memory takes (w4_tc.cu).  In each 32-bit word
// column 2 i stands at bit 4 i and column 2 i + 1 at bit 16 + 4 i, so one
// shift and one mask give a pair of 16-bit lanes.  Scales and zeros:
// [rt][group][b][g]{row g, row g + 8}; for groups of 32 [rt][u][b][g][h]{row
// g, row g + 8}, so that in either case one load of a lane has what a unit
// needs, and one bulk copy what the 128 rows of a unit need.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdio>
#include <cstring>
#include <new>

#include "../../include/proj.h"
#include "cluster_common.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "vec.cuh"
#include "w4.h"
#include "w4_num.cuh"

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
                                  int64_t E, int64_t N, int64_t K, int64_t RT, int64_t KU) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= E * RT * KU * 256) return;
  const int lane = static_cast<int>(i & 31), b = static_cast<int>((i >> 5) & 7);
  const int64_t u = (i >> 8) % KU;
  const int64_t rt = (i >> 8) / KU % RT;
  const int64_t e = (i >> 8) / KU / RT;
  const int g = lane >> 2, t = lane & 3;
  const int64_t bytes = (K + 1) / 2;
  uint32_t w[4];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int hi = 0; hi < 2; ++hi) {
      const int64_t n = rt * 128 + b * 16 + g + 8 * hi;
      uint32_t v = 0;
      if (n < N) {
        const uint8_t* row = codes + (e * N + n) * bytes;
        const int64_t k0 = u * 64 + 32 * h + 4 * t;
#pragma unroll
        for (int c = 0; c < 8; ++c)
          v |= code_at(row, k0 + 16 * (c >> 2) + (c & 3), K) << ((c & 1) * 16 + (c >> 1) * 4);
      }
      w[2 * h + hi] = v;
    }
  dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
}

// One thread per packed scale.  Groups beyond K and rows beyond N get 0.
// *wide becomes 1 if a finite scale s has s (q - z) above `most`, the largest
// number of its type, for a q in 0..15.
template <typename T>
__global__ void pack_scales_kernel(const uint16_t* __restrict__ scales,
                                   const uint8_t* __restrict__ zeros, uint16_t* __restrict__ ds,
                                   uint8_t* __restrict__ dz, int64_t E, int64_t N, int64_t NG,
                                   int64_t NGp, int64_t RT, bool g32, float most, uint32_t* wide) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= E * RT * NGp * 128) return;
  const int64_t j = i % (NGp * 128);  // within the tile
  const int64_t rt = i / (NGp * 128) % RT;
  const int64_t e = i / (NGp * 128) / RT;
  const int64_t grp = g32 ? 2 * (j >> 8) + ((j >> 1) & 1) : j >> 7;
  const int b = static_cast<int>(g32 ? (j >> 5) & 7 : (j >> 4) & 7);
  const int g = static_cast<int>(g32 ? (j >> 2) & 7 : (j >> 1) & 7);
  const int64_t n = rt * 128 + b * 16 + g + 8 * (j & 1);
  const bool in = n < N && grp < NG;
  const int64_t src = (e * N + n) * NG + grp;
  const uint16_t s = in ? scales[src] : 0;
  ds[i] = s;
  int z = 8;
  if (dz) {
    z = in ? zeros[src] & 15 : 0;
    dz[i] = static_cast<uint8_t>(z);
  }
  const float size = fabsf(to_f32(*reinterpret_cast<const T*>(&s)));
  if (size <= most && size * static_cast<float>(max(z, 15 - z)) > most) atomicOr(wide, 1u);
}

// ------------------------------------------------------ streaming kernel --

// Four consecutive x values of a row from column c, which K cuts: zeros from
// K on.
template <typename T>
__device__ __noinline__ uint2 load_x4_edge(const T* row, int c, int K) {
  uint2 v = make_uint2(0, 0);
  const uint16_t* r = reinterpret_cast<const uint16_t*>(row);
  if (c < K) v.x = r[c];
  if (c + 1 < K) v.x |= static_cast<uint32_t>(r[c + 1]) << 16;
  if (c + 2 < K) v.y = r[c + 2];
  if (c + 3 < K) v.y |= static_cast<uint32_t>(r[c + 3]) << 16;
  return v;
}

__device__ __forceinline__ float ld_dsmem_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

// Launch shape of the streaming kernel: NT tiles of 8 tokens, RB blocks of 16
// rows a CTA, clusters of C CTAs along K.
constexpr int kStreamWarps = 8;
struct StreamShape {
  int NT, RB, C;
  int64_t tiles;
};

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
__device__ __forceinline__ Tile find_tile(const int32_t* offsets, int E, int64_t m, int T,
                                          int index) {
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
      lo = min(max(offsets[e], 0), lim);
      hi = min(max(offsets[e + 1], lo), lim);
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

// A CTA takes RB blocks of 16 weight rows and one tile of 8 NT tokens; each
// warp of the C CTAs of a cluster has a run of the units of K; warps meet in
// shared memory, CTAs after that through distributed shared memory.  A
// warp keeps kD units of codes, scales and x in flight, all of them straight
// to registers: the x of 8 tokens is two bytes per byte of one block's codes,
// so RB = 2 blocks share it, and it comes from L2.  One matrix is short of
// warps and takes kD = 4 units; experts, whose CTAs come in several waves, do
// better with kD = 2 and three CTAs an SM (64 rows over 256 experts of 1024 x
// 8192: 77 us against 92).
template <typename T, bool kG32, bool kZeros, int NT, int RB, int kD>
__global__ void __launch_bounds__(32 * kStreamWarps, kD == 2 && NT == 1 ? 3 : 2)
    w4_stream_kernel(const W4Params p, const int C) {
  constexpr int W = kStreamWarps;
  using Scale = typename ScaleOf<kG32>::Pair;
  using Zero = typename ScaleOf<kG32>::Bytes;
  __shared__ alignas(16) float s_red[W][RB][NT][32][4];
  __shared__ float s_part[RB * 16 * NT * 8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int rank = static_cast<int>(blockIdx.x) % C;
  const int rb0 = static_cast<int>(blockIdx.x) / C * RB;

  uint4 code[kD][RB];
  Scale sc[kD][RB];
  Zero ze[kD][RB];
  uint2 xf[kD][NT][4];
  const uint4* codes[RB];
  const Scale* scales[RB];
  const Zero* zeros[RB];
  const int units = kG32 ? p.KU : p.NGp;  // lines of scales in a tile
  // the warp's run of units
  const int part = rank * W + warp;
  const int u0 = static_cast<int>(static_cast<int64_t>(part) * p.KU / (W * C));
  const int u1 = static_cast<int>(static_cast<int64_t>(part + 1) * p.KU / (W * C));
  auto open = [&](int expert) {
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const int rb = min(rb0 + r, p.RB - 1);
      const int64_t tile = static_cast<int64_t>(expert) * p.RT + (rb >> 3);
      codes[r] = p.codes + (tile * p.KU + u0) * 256 + (rb & 7) * 32 + lane;
      const int64_t at = tile * units * 64 + (rb & 7) * 8 + g;
      scales[r] = reinterpret_cast<const Scale*>(p.scales) + at;
      zeros[r] = reinterpret_cast<const Zero*>(p.zeros) + at;
    }
  };
  // unit `u` to slot d, i units behind the one that the pointers stand at
  auto fetch_w = [&](int d, int i, int u) {
    if (u >= u1) return;
    const int at = (kG32 ? u : p.group_of(u)) * 64;
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      code[d][r] = ld_stream_v4(codes[r] + i * 256);
      sc[d][r] = __ldg(scales[r] + at);
      if (kZeros) ze[d][r] = __ldg(zeros[r] + at);
    }
  };

  griddep_launch_dependents();
  const int index = static_cast<int>(blockIdx.z * gridDim.y + blockIdx.y);
  Tile tile;
  if (p.offsets) {
    griddep_wait();
    tile = find_tile<32 * W>(p.offsets, p.E, p.m, 8 * NT, index);
    if (tile.rows == 0) return;  // every CTA of the cluster
    open(tile.expert);
#pragma unroll
    for (int d = 0; d < kD; ++d) fetch_w(d, d, u0 + d);
  } else {
    tile.expert = 0;
    tile.row0 = static_cast<int64_t>(index) * 8 * NT;
    tile.rows = static_cast<int>(min(static_cast<int64_t>(8 * NT), p.m - tile.row0));
    // the weights are constant: their first loads do not wait for the kernel before
    open(0);
#pragma unroll
    for (int d = 0; d < kD; ++d) fetch_w(d, d, u0 + d);
    griddep_wait();
    if (tile.rows <= 0) return;  // behind the last tile: every CTA of the cluster
  }
  const T* x[NT];
  bool live[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    x[j] = static_cast<const T*>(p.x) + (tile.row0 + 8 * j + g) * p.ldx + u0 * 64 + 4 * t;
    live[j] = 8 * j + g < tile.rows;
#pragma unroll
    for (int d = 0; d < kD; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) xf[d][j][i] = make_uint2(0, 0);
  }
  const int whole = p.K / 64;  // units that K does not cut
  auto fetch_x = [&](int d, int b, int u) {
    if (u >= u1) return;
#pragma unroll
    for (int j = 0; j < NT; ++j)
      if (live[j]) {
        const T* at = x[j] + b * 64;
        if (u < whole) {
#pragma unroll
          for (int i = 0; i < 4; ++i) xf[d][j][i] = *reinterpret_cast<const uint2*>(at + 16 * i);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            xf[d][j][i] = load_x4_edge(at, 16 * i, p.K - u * 64 - 4 * t);
        }
      }
  };
#pragma unroll
  for (int d = 0; d < kD; ++d) fetch_x(d, d, u0 + d);

  float acc[RB][NT][4] = {};
  for (int ub = u0; ub < u1; ub += kD) {
#pragma unroll
    for (int r = 0; r < RB; ++r) codes[r] += kD * 256;
#pragma unroll
    for (int j = 0; j < NT; ++j) x[j] += kD * 64;
#pragma unroll
    for (int d = 0; d < kD; ++d) {
      const int u = ub + d;
      if (u < u1) {
#pragma unroll
        for (int r = 0; r < RB; ++r) {
          const uint32_t word[4] = {code[d][r].x, code[d][r].y, code[d][r].z, code[d][r].w};
          float part[NT][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t z = kZeros ? ScaleOf<kG32>::bytes(ze[d][r], h) : 0x0808u;
            const uint32_t zero[2] = {zero_pair<T>(z, 0), zero_pair<T>(z, 1)};
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              // rows g, g + 8 of the step's columns 4 t, + 1, then of + 2, + 3
              const uint32_t a[4] = {code_pair<T>(word[2 * h], 2 * s, zero[0]),
                                     code_pair<T>(word[2 * h + 1], 2 * s, zero[1]),
                                     code_pair<T>(word[2 * h], 2 * s + 1, zero[0]),
                                     code_pair<T>(word[2 * h + 1], 2 * s + 1, zero[1])};
#pragma unroll
              for (int j = 0; j < NT; ++j) {
                const uint2 b = xf[d][j][2 * h + s];
                if (s == 0 && (kG32 || h == 0))
                  Num<T>::mma_first(part[j], a, b.x, b.y);
                else
                  Num<T>::mma(part[j], a, b.x, b.y);
              }
            }
            if (kG32 || h == 1) {
              const uint32_t sp = ScaleOf<kG32>::pair(sc[d][r], h);
              const float s0 = to_f32(reinterpret_cast<const T*>(&sp)[0]);
              const float s1 = to_f32(reinterpret_cast<const T*>(&sp)[1]);
#pragma unroll
              for (int j = 0; j < NT; ++j) {
                acc[r][j][0] = fmaf(s0, part[j][0], acc[r][j][0]);
                acc[r][j][1] = fmaf(s0, part[j][1], acc[r][j][1]);
                acc[r][j][2] = fmaf(s1, part[j][2], acc[r][j][2]);
                acc[r][j][3] = fmaf(s1, part[j][3], acc[r][j][3]);
              }
            }
          }
        }
        fetch_w(d, d, u + kD);
        fetch_x(d, d, u + kD);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < RB; ++r)
#pragma unroll
    for (int j = 0; j < NT; ++j)
      *reinterpret_cast<float4*>(s_red[warp][r][j][lane]) =
          make_float4(acc[r][j][0], acc[r][j][1], acc[r][j][2], acc[r][j][3]);
  __syncthreads();
  // Sum the warps' partials in order.  Value i of the tile: row i % (16 RB),
  // token i / (16 RB); element c of lane l is row g + 8 (c / 2), token
  // 2 t + c % 2.
  constexpr int kRows = 16 * RB;
  T* out = static_cast<T*>(p.out) + tile.row0 * p.ldo + static_cast<int64_t>(rb0) * 16;
  const int n_left = p.N - rb0 * 16;
  for (int i = threadIdx.x; i < kRows * NT * 8; i += 32 * W) {
    const int n = i % kRows, tok = i / kRows;
    const int l = (n & 7) * 4 + ((tok & 7) >> 1);
    const int c = ((n >> 3) & 1) * 2 + (tok & 1);
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) s += s_red[w][n >> 4][tok >> 3][l][c];
    if (C > 1)
      s_part[i] = s;
    else if (tok < tile.rows && n < n_left)
      out[tok * p.ldo + n] = from_f32<T>(s);
  }
  if (C > 1) {
    cluster_sync_all();
    const uint32_t base = smem_u32(s_part);
    for (int i = rank * 32 * W + threadIdx.x; i < kRows * tile.rows; i += 32 * W * C) {
      const int n = i % kRows, tok = i / kRows;
      float s = 0.f;
      for (int r = 0; r < C; ++r)
        s += ld_dsmem_f32(map_to_rank(base + 4 * i, static_cast<uint32_t>(r)));
      if (n < n_left) out[tok * p.ldo + n] = from_f32<T>(s);
    }
    cluster_sync_all();  // no CTA leaves while another reads its partial sums
  }
}

template <typename T, bool kG32, bool kZeros, int NT, int RB, int kD>
cudaError_t stream_launch(const W4Params& p, const StreamShape& sh, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  // y has at most 65,535: 2^20 rows are more tiles
  const int64_t y = std::min<int64_t>(sh.tiles, 32768);
  cfg.gridDim = dim3(static_cast<unsigned>((p.RB + RB - 1) / RB * sh.C), static_cast<unsigned>(y),
                     static_cast<unsigned>((sh.tiles + y - 1) / y));
  cfg.blockDim = dim3(32 * kStreamWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(sh.C);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = sh.C > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, w4_stream_kernel<T, kG32, kZeros, NT, RB, kD>, p, sh.C);
}

template <typename T, int NT, int RB, int kD>
cudaError_t stream_form(const W4Params& p, const StreamShape& sh, cudaStream_t s) {
  if (p.group == 32)
    return p.zeros ? stream_launch<T, true, true, NT, RB, kD>(p, sh, s)
                   : stream_launch<T, true, false, NT, RB, kD>(p, sh, s);
  return p.zeros ? stream_launch<T, false, true, NT, RB, kD>(p, sh, s)
                 : stream_launch<T, false, false, NT, RB, kD>(p, sh, s);
}

template <typename T, int NT>
cudaError_t stream_any(const W4Params& p, const StreamShape& sh, cudaStream_t s) {
  if (sh.RB == 1) return stream_form<T, NT, 1, NT == 1 ? 4 : 2>(p, sh, s);
  if (NT == 2 || p.offsets) return stream_form<T, NT, 2, 2>(p, sh, s);
  return stream_form<T, NT, 2, NT == 1 ? 4 : 2>(p, sh, s);
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
  bool exact;       // products of the 4-bit numbers at any number of rows
  int sms;
  int clusters[9];  // [C]: clusters of C CTAs of the tensor-core kernel that run at once
};

namespace {

// What a call with m rows runs.
struct Plan {
  bool tc;
  StreamShape stream;
  int tn, C;
  int64_t grid;
};

// Rows that a matrix meets (on average, for experts) up to which the weights
// are streamed with exact 4-bit products; above, the tensor-core kernel.
// Measured: 4096 x 8192 at 16 rows 13.1 us streamed, 14.4 on the tensor cores,
// at 17 rows 17.8 and 14.4; 60 experts of 2048 x 4096, 4.3 rows each, 88 us
// and 99, at 8.5 rows 121 and 100.  Experts with fewer units of K than
// kStreamUnits keep a streaming CTA too short for what it takes to start: 104
// experts of 8192 x 512 take 204 us streamed and 76 on the tensor cores, whose
// CTAs stay; of 2048 x 4096 both take 83 us.  Unless there are few such CTAs,
// kStreamCtas an SM at most: 8 experts of 1024 x 2048, a row each (288 CTAs),
// 8.4 us streamed and 12.4 on the tensor cores, of 2048 x 768 (576) 8.3 and
// 9.6, of 5173 x 1081 (1458) 17.6 and 13.5.
// A handle that is to be exact is always streamed; every tile of 16 tokens
// then decodes the weights again.
constexpr int64_t kStreamRows = 16, kStreamRowsExperts = 6;
constexpr int kStreamUnits = 64, kStreamCtas = 4;

Plan make_plan(const proj_w4_ctx* h, int64_t m, bool experts) {
  const W4Params& p = h->p;
  Plan pl = {};
  const int64_t rows = experts ? (m + p.E - 1) / p.E : m;
  StreamShape& s = pl.stream;
  s.NT = rows <= 8 ? 1 : 2;
  const int64_t per = 8 * s.NT;
  // of the experts that have rows, each has at most one part-filled tile
  s.tiles = experts ? std::min<int64_t>(p.E, m) + m / per : (m + per - 1) / per;
  pl.tc = !h->exact &&
          (p.E > 1 ? rows > kStreamRowsExperts ||
                         (p.KU < kStreamUnits && (p.RB + 1) / 2 * s.tiles > kStreamCtas * h->sms)
                   : rows > kStreamRows);
  if (!pl.tc) {
    // Two blocks of rows share the loads of x where that leaves a CTA per SM
    // or so; K is split over a cluster while that puts at most two CTAs on an SM
    // (a row for one of 8 experts of 1000 x 8192: 6.3 us, 14.4 unsplit).
    s.RB = experts || p.RB * 3 >= h->sms * 4 ? 2 : 1;
    s.C = 1;
    const int64_t groups = (p.RB + s.RB - 1) / s.RB * s.tiles;
    while (s.C < 8 && groups * s.C <= h->sms && p.KU >= 2 * kStreamWarps * s.C)
      s.C *= 2;
  } else {
    pl.tn = rows <= 64 ? 64 : experts || m <= 128 ? 128 : 256;
    const int64_t tiles =
        experts ? std::min<int64_t>(p.E, m) + m / pl.tn : (m + pl.tn - 1) / pl.tn;
    const int64_t items = tiles * p.RT;
    // K is split while the clusters run at once and a CTA keeps two steps (146
    // rows over 8 experts of 536 x 6208: 18.5 us, 28.0 unsplit)
    pl.C = 1;
    for (int c = 2; c <= 8; ++c)
      if (items <= h->clusters[c] && p.KU >= 4 * c) pl.C = c;
    pl.grid = pl.C > 1 ? items * pl.C : std::min<int64_t>(items, h->sms);
  }
  return pl;
}

int run(const char* call, proj_w4_handle h, const void* x, int64_t ldx, int64_t m,
        const int32_t* offsets, bool experts, void* out, int64_t ldo, proj_stream stream) {
  if (!h) return refuse(PROJ_EINVAL, call, "NULL handle");
  if (m < 0 || ldx < h->p.K || ldo < h->p.N)
    return refuse(PROJ_EINVAL, call, "m < 0, or a row stride below K or N");
  if (!experts && h->p.E != 1)
    return refuse(PROJ_EINVAL, call, "the handle holds several experts");
  if (m > (int64_t{1} << 20) || ldx >= (int64_t{1} << 31) || ldo >= (int64_t{1} << 31))
    return refuse(PROJ_EUNSUPPORTED, call, "m > 2^20 or a row stride >= 2^31");
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
  const Plan pl = make_plan(h, m, experts);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool fp16 = h->dtype == PROJ_FP16;
  cudaError_t e;
  if (pl.tc)
    e = w4_tc_launch(fp16, pl.tn, p, pl.grid, pl.C, s);
  else if (pl.stream.NT == 1)
    e = fp16 ? stream_any<__half, 1>(p, pl.stream, s) : stream_any<__nv_bfloat16, 1>(p, pl.stream, s);
  else
    e = fp16 ? stream_any<__half, 2>(p, pl.stream, s) : stream_any<__nv_bfloat16, 2>(p, pl.stream, s);
  return e == cudaSuccess ? PROJ_OK : record_cuda(e, call);
}

}  // namespace

extern "C" proj_w4_handle proj_w4_prepare(const void* codes, const void* scales, const void* zeros,
                                          int64_t experts, int64_t N, int64_t K, int64_t group,
                                          int dtype, int* status) {
  return proj_w4_prepare_ex(codes, scales, zeros, experts, N, K, group, dtype, 0u, status);
}

extern "C" proj_w4_handle proj_w4_prepare_ex(const void* codes, const void* scales,
                                             const void* zeros, int64_t experts, int64_t N,
                                             int64_t K, int64_t group, int dtype, uint32_t flags,
                                             int* status) {
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
  if (flags & ~static_cast<uint32_t>(PROJ_W4_EXACT)) return refused(PROJ_EINVAL, "unknown flags");
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
  p.RT = static_cast<int>((N + 127) / 128);
  p.KU = static_cast<int>((K + 63) / 64);
  const int64_t NG = (K + group - 1) / group;
  const uint64_t upg = static_cast<uint64_t>(group) / 64;
  p.group_magic = upg ? static_cast<uint32_t>(((uint64_t{1} << 31) + upg - 1) / upg) : 0u;
  h->sms = proj_num_sms();
  for (int c = 1; c <= 8; ++c) h->clusters[c] = w4_tc_max_clusters(c);
  p.NGp = static_cast<int>(group == 32 ? 2 * p.KU : NG);  // every unit has its groups
  h->dtype = dtype;
  const int64_t row_tiles = experts * p.RT;
  const int64_t code_bytes = row_tiles * p.KU * kW4UnitBytes;
  const int64_t scale_bytes = row_tiles * p.NGp * 256;
  const int64_t zero_bytes = zeros ? (row_tiles * p.NGp * 128 + 255) / 256 * 256 : 0;
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
  const int64_t lanes = row_tiles * p.KU * 256, cells = row_tiles * p.NGp * 128;
  // the status word, and behind it the word that says whether a scale is wide
  e = cudaMemsetAsync(p.status, 0, 8, nullptr);
  pack_codes_kernel<<<static_cast<unsigned>((lanes + 255) / 256), 256>>>(
      static_cast<const uint8_t*>(codes), const_cast<uint4*>(p.codes), experts, N, K, p.RT, p.KU);
  auto* const pack_scales =
      dtype == PROJ_FP16 ? pack_scales_kernel<__half> : pack_scales_kernel<__nv_bfloat16>;
  pack_scales<<<static_cast<unsigned>((cells + 255) / 256), 256>>>(
      static_cast<const uint16_t*>(scales), static_cast<const uint8_t*>(zeros),
      const_cast<uint16_t*>(p.scales), const_cast<uint8_t*>(p.zeros), experts, N, NG, p.NGp, p.RT,
      group == 32, dtype == PROJ_FP16 ? 65504.f : 0x1.FEp127f, p.status + 1);
  if (e == cudaSuccess) e = cudaGetLastError();
  uint32_t wide = 0;
  if (e == cudaSuccess)
    e = cudaMemcpyAsync(&wide, p.status + 1, 4, cudaMemcpyDeviceToHost, nullptr);
  if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
  if (e != cudaSuccess) {
    record_cuda(e, call);
    cudaFree(h->base);
    delete h;
    if (status) *status = PROJ_ECUDA;
    return nullptr;
  }
  // Where s (q - z) leaves the range of the type, the tensor cores would be
  // given infinities: such a handle streams at any number of rows.
  h->exact = (flags & PROJ_W4_EXACT) || wide;
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
  char text[2][128];
  for (int experts = 0; experts < 2; ++experts) {
    const Plan pl = make_plan(h, m, experts);
    if (pl.tc)
      std::snprintf(text[experts], sizeof text[experts],
                    "w4 tcgen05, %d-token tiles, grid %lld, cluster %d, weights rounded to %s",
                    pl.tn, static_cast<long long>(pl.grid), pl.C,
                    h->dtype == PROJ_FP16 ? "fp16" : "bf16");
    else
      std::snprintf(text[experts], sizeof text[experts],
                    "w4 stream, %d-token tiles, %d rows, cluster %d, exact 4-bit products",
                    8 * pl.stream.NT, 16 * pl.stream.RB, pl.stream.C);
  }
  // a stack of one takes both calls
  if (h->p.E == 1 && std::strcmp(text[0], text[1]))
    std::snprintf(buf, cap, "%s; with offsets: %s", text[0], text[1]);
  else
    std::snprintf(buf, cap, "%s", text[h->p.E > 1]);
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
