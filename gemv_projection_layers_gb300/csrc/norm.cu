// norm.cu -- the norms at a block's two ends, fused with its gate and the
// residual scale, and their gradient.
//
//   n = y rp w_post,  rp = (mean y^2 + eps)^-1/2
//   u = alpha r + beta g n,  g = act(gate)
//   h = u ru w_pre,   ru = (mean u^2 + eps)^-1/2
//
// Gradient, from du' (of u) and dh, with un = u ru, yn = y rp, t = dh w_pre:
//   du = du' + ru (t - un S1),              S1 = mean(t un)
//   dr = alpha du,  c = beta g du,  b = c w_post
//   dy = rp (b - yn S2),                    S2 = mean(b yn)
//   dg = beta n du,  dw_post = sum_rows c yn,  dw_pre = sum_rows dh un
// S2 is linear in S1: with e = du' + ru t, du = e - ru un S1, so
//   S2 D = beta (A - ru S1 B),  A = sum g n e,  B = sum g n un,
// and one reduction of three sums serves the whole row.  (For a gate per
// token, dg = beta (A - ru S1 B) with g left out of A and B.)
//
// Every row is read once and stays in registers between the reductions; both
// kernels are bound by HBM.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdio>

#include "../../include/proj.h"
#include "kernels.h"
#include "ptx.cuh"
#include "vec.cuh"

namespace proj {
namespace {

constexpr int kMaxD = 16384;
constexpr int kGradCtas = 304;  // rows of the column sums' workspace, at most

__device__ __forceinline__ float act(float g, int kind) {
  return kind == PROJ_GATE_SIGMOID ? 1.f / (1.f + expf(-g)) : g;
}
// d act / d gate from the activated value.
__device__ __forceinline__ float act_slope(float g, int kind) {
  return kind == PROJ_GATE_SIGMOID ? g * (1.f - g) : 1.f;
}

// TPR threads share a row of D = up to TPR x NV x V elements; vector j of
// thread i is j TPR + i, so accesses are contiguous over the threads.
template <typename T, int V, int TPR, int NV>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR)
    norm_kernel(const __grid_constant__ proj_norm_args a) {
  constexpr int kRows = TPR < 128 ? 128 / TPR : 1;
  __shared__ float room[2 * 32];
  int turn = 0;
  const int tid = static_cast<int>(threadIdx.x) % TPR;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / TPR;
  griddep_launch_dependents();
  griddep_wait();
  if (row >= a.m) return;  // whole warps (kRows > 1 has no block barrier)
  const int D = static_cast<int>(a.D);
  const int nvec = D / V;
  const float inv_d = 1.f / static_cast<float>(D);
  const T* y = static_cast<const T*>(a.y) + row * a.ldy;
  const T* r = static_cast<const T*>(a.residual) + row * a.ldr;

  Vec<T, V> vy[NV], vr[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * TPR + tid) * V;
    if (j * TPR + tid < nvec) {
      if (a.y) vy[j] = load_vec<T, V>(y + c);
      vr[j] = load_vec<T, V>(r + c);
    }
  }
  float rp = 1.f;
  if (a.y && !a.y_plain) {
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (j * TPR + tid < nvec) {
        float v[V];
        widen(vy[j], v);
#pragma unroll
        for (int i = 0; i < V; ++i) s[0] = fmaf(v[i], v[i], s[0]);
      }
    row_sums<TPR, 1>(s, room, turn);
    rp = 1.f / sqrtf(s[0] * inv_d + a.eps);
    if (tid == 0 && a.rstd_post) a.rstd_post[row] = rp;
  }
  float g_row = 1.f;
  if (a.gate_mode == PROJ_GATE_TOKEN)
    g_row = act(to_f32(static_cast<const T*>(a.gate)[row]), a.gate_act);
  const T* gate = static_cast<const T*>(a.gate);
  if (a.gate_mode == PROJ_GATE_ELEMENT) gate += row * a.ldg;
  const bool g_vec = a.gate_mode == PROJ_GATE_CHANNEL || a.gate_mode == PROJ_GATE_ELEMENT;

  float u[NV][V];
  float s[1] = {0.f};
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * TPR + tid) * V;
    if (j * TPR + tid < nvec) {
      float rv[V];
      widen(vr[j], rv);
#pragma unroll
      for (int i = 0; i < V; ++i) u[j][i] = a.alpha * rv[i];
      if (a.y) {
        float yv[V], gv[V], wv[V];
        widen(vy[j], yv);
        if (g_vec) {
          widen(load_vec<T, V>(gate + c), gv);
        }
        if (a.w_post) widen(load_vec<T, V>(static_cast<const T*>(a.w_post) + c), wv);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float n = yv[i] * rp;
          if (a.w_post) n *= wv[i];
          const float g = g_vec ? act(gv[i], a.gate_act) : g_row;
          u[j][i] = fmaf(a.beta * g, n, u[j][i]);
        }
      }
      if (a.out) store_vec<T, V>(static_cast<T*>(a.out) + row * a.ldo + c, u[j]);
#pragma unroll
      for (int i = 0; i < V; ++i) s[0] = fmaf(u[j][i], u[j][i], s[0]);
    }
  }
  if (!a.normed && !a.rstd_pre) return;
  row_sums<TPR, 1>(s, room, turn);
  const float ru = 1.f / sqrtf(s[0] * inv_d + a.eps);
  if (tid == 0 && a.rstd_pre) a.rstd_pre[row] = ru;
  if (!a.normed) return;
  T* h = static_cast<T*>(a.normed) + row * a.ldn;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * TPR + tid) * V;
    if (j * TPR + tid < nvec) {
      float wv[V], o[V];
      if (a.w_pre) widen(load_vec<T, V>(static_cast<const T*>(a.w_pre) + c), wv);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        o[i] = u[j][i] * ru;
        if (a.w_pre) o[i] *= wv[i];
      }
      store_vec<T, V>(h + c, o);
    }
  }
}

// Column sums: part[cta][which][D] (which: 0 dw_post, 1 dw_pre, 2 dgate).
template <typename T, int V, int TPR, int NV>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR)
    norm_grad_kernel(const __grid_constant__ proj_norm_grad_args a) {
  constexpr int kRows = TPR < 128 ? 128 / TPR : 1;
  __shared__ float room[2 * 3 * 32];
  int turn = 0;
  const int tid = static_cast<int>(threadIdx.x) % TPR;
  const int part_row = static_cast<int>(blockIdx.x) * kRows + threadIdx.x / TPR;
  griddep_launch_dependents();
  griddep_wait();
  const int D = static_cast<int>(a.D);
  const int nvec = D / V;
  const float inv_d = 1.f / static_cast<float>(D);
  const bool normed = a.y && !a.y_plain;
  const bool g_vec = a.gate_mode == PROJ_GATE_CHANNEL || a.gate_mode == PROJ_GATE_ELEMENT;
  const bool g_token = a.gate_mode == PROJ_GATE_TOKEN;
  const bool col_gate = a.gate_mode == PROJ_GATE_CHANNEL && a.dgate;

  float acc_post[NV][V] = {}, acc_pre[NV][V] = {}, acc_gate[NV][V] = {};

  for (int64_t row = part_row; row < a.m; row += static_cast<int64_t>(gridDim.x) * kRows) {
    const T* gate = static_cast<const T*>(a.gate);
    if (a.gate_mode == PROJ_GATE_ELEMENT) gate += row * a.ldg;
    const float rp = normed ? a.rstd_post[row] : 1.f;
    const float ru = a.dnormed ? a.rstd_pre[row] : 1.f;
    const float g_row = g_token ? act(to_f32(gate[row]), a.gate_act) : 1.f;
    // per element: yn, g (activated), un, e
    Vec<T, V> vy[NV], vr[NV], vg[NV], vo[NV], vh[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + tid) * V;
      if (j * TPR + tid < nvec) {
        if (a.y) vy[j] = load_vec<T, V>(static_cast<const T*>(a.y) + row * a.ldy + c);
        vr[j] = load_vec<T, V>(static_cast<const T*>(a.residual) + row * a.ldr + c);
        if (g_vec) vg[j] = load_vec<T, V>(gate + c);
        if (a.dout) vo[j] = load_vec<T, V>(static_cast<const T*>(a.dout) + row * a.lddo + c);
        if (a.dnormed)
          vh[j] = load_vec<T, V>(static_cast<const T*>(a.dnormed) + row * a.lddn + c);
      }
    }
    auto element = [&](int j, int i, float wpo, float wpr, float& yn, float& n, float& g,
                       float& un, float& dh, float& e) {
      yn = a.y ? to_f32(vy[j].e[i]) * rp : 0.f;
      n = yn * wpo;
      g = g_vec ? act(to_f32(vg[j].e[i]), a.gate_act) : g_row;
      const float u = fmaf(a.beta * g, n, a.alpha * to_f32(vr[j].e[i]));
      un = u * ru;
      dh = a.dnormed ? to_f32(vh[j].e[i]) : 0.f;
      e = fmaf(ru, dh * wpr, a.dout ? to_f32(vo[j].e[i]) : 0.f);
    };
    float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + tid) * V;
      if (j * TPR + tid < nvec) {
        float wpo[V], wpr[V];
        if (a.w_post) widen(load_vec<T, V>(static_cast<const T*>(a.w_post) + c), wpo);
        if (a.w_pre) widen(load_vec<T, V>(static_cast<const T*>(a.w_pre) + c), wpr);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float wo = a.w_post ? wpo[i] : 1.f, wr = a.w_pre ? wpr[i] : 1.f;
          float yn, n, g, un, dh, e;
          element(j, i, wo, wr, yn, n, g, un, dh, e);
          s[0] = fmaf(dh * wr, un, s[0]);
          const float gn = g_token ? n : g * n;
          s[1] = fmaf(gn, e, s[1]);
          s[2] = fmaf(gn, un, s[2]);
        }
      }
    }
    row_sums<TPR, 3>(s, room, turn);
    const float s1 = a.dnormed ? s[0] * inv_d : 0.f;
    const float ab = a.beta * (s[1] - ru * s1 * s[2]);  // sum of beta [g] n du
    const float s2 = normed ? (g_token ? g_row * ab : ab) * inv_d : 0.f;
    if (g_token && a.dgate && tid == 0)
      static_cast<T*>(a.dgate)[row] = from_f32<T>(ab * act_slope(g_row, a.gate_act));
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + tid) * V;
      if (j * TPR + tid < nvec) {
        float wpo[V], wpr[V], dy[V], dr[V], dg[V];
        if (a.w_post) widen(load_vec<T, V>(static_cast<const T*>(a.w_post) + c), wpo);
        if (a.w_pre) widen(load_vec<T, V>(static_cast<const T*>(a.w_pre) + c), wpr);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float wo = a.w_post ? wpo[i] : 1.f, wr = a.w_pre ? wpr[i] : 1.f;
          float yn, n, g, un, dh, e;
          element(j, i, wo, wr, yn, n, g, un, dh, e);
          const float du = e - ru * un * s1;
          const float cc = a.beta * g * du;
          dr[i] = a.alpha * du;
          dy[i] = normed ? rp * (cc * wo - yn * s2) : cc;
          dg[i] = a.beta * n * du * act_slope(g, a.gate_act);
          acc_post[j][i] = fmaf(cc, yn, acc_post[j][i]);
          acc_pre[j][i] = fmaf(dh, un, acc_pre[j][i]);
          acc_gate[j][i] += dg[i];
        }
        if (a.dy) store_vec<T, V>(static_cast<T*>(a.dy) + row * a.lddy + c, dy);
        if (a.dresidual) store_vec<T, V>(static_cast<T*>(a.dresidual) + row * a.lddr + c, dr);
        if (a.gate_mode == PROJ_GATE_ELEMENT && a.dgate)
          store_vec<T, V>(static_cast<T*>(a.dgate) + row * a.lddg + c, dg);
      }
    }
  }
  if (!a.dw_post && !a.dw_pre && !col_gate) return;
  float* part = static_cast<float*>(a.workspace) + static_cast<size_t>(part_row) * 3 * D;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * TPR + tid) * V;
    if (j * TPR + tid < nvec) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (a.dw_post) part[c + i] = acc_post[j][i];
        if (a.dw_pre) part[D + c + i] = acc_pre[j][i];
        if (col_gate) part[2 * D + c + i] = acc_gate[j][i];
      }
    }
  }
}

// Sums the partial rows of each column in order: warps of a CTA take every
// kSumWarps-th row of 32 columns, then meet in shared memory.
constexpr int kSumWarps = 8;
__global__ void __launch_bounds__(32 * kSumWarps)
    norm_grad_sum_kernel(const float* __restrict__ part, int rows, int D, float* d0, float* d1,
                         float* d2) {
  __shared__ float room[kSumWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int which = blockIdx.y;
  float* dst = which == 0 ? d0 : (which == 1 ? d1 : d2);
  const int c = blockIdx.x * 32 + lane;
  griddep_launch_dependents();
  griddep_wait();
  if (!dst) return;
  float s = 0.f;
  if (c < D) {
#pragma unroll 8
    for (int r = warp; r < rows; r += kSumWarps)
      s += part[(static_cast<size_t>(r) * 3 + which) * D + c];
  }
  room[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < D) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < kSumWarps; ++w) t += room[w][lane];
    dst[c] = t;
  }
}

cudaLaunchConfig_t config(unsigned grid_x, unsigned grid_y, unsigned threads, cudaStream_t s,
                          cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid_x, grid_y);
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <typename T, int V, int TPR, int NV>
cudaError_t forward(const proj_norm_args& a, cudaStream_t s) {
  constexpr int kRows = TPR < 128 ? 128 / TPR : 1;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg =
      config(static_cast<unsigned>((a.m + kRows - 1) / kRows), 1, TPR < 128 ? 128 : TPR, s, attr);
  return cudaLaunchKernelEx(&cfg, norm_kernel<T, V, TPR, NV>, a);
}

int grad_parts(int64_t m) { return static_cast<int>(std::min<int64_t>(m, kGradCtas)); }

template <typename T, int V, int TPR, int NV>
cudaError_t backward(const proj_norm_grad_args& a, cudaStream_t s) {
  constexpr int kRows = TPR < 128 ? 128 / TPR : 1;
  const int grid = (grad_parts(a.m) + kRows - 1) / kRows;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg =
      config(static_cast<unsigned>(grid), 1, TPR < 128 ? 128 : TPR, s, attr);
  cudaError_t e = cudaLaunchKernelEx(&cfg, norm_grad_kernel<T, V, TPR, NV>, a);
  if (e != cudaSuccess) return e;
  float* dgate = a.gate_mode == PROJ_GATE_CHANNEL ? static_cast<float*>(a.dgate) : nullptr;
  if (!a.dw_post && !a.dw_pre && !dgate) return cudaSuccess;
  cfg = config(static_cast<unsigned>((a.D + 31) / 32), 3, 32 * kSumWarps, s, attr);
  return cudaLaunchKernelEx(&cfg, norm_grad_sum_kernel,
                            static_cast<const float*>(static_cast<float*>(a.workspace)),
                            grid * kRows, static_cast<int>(a.D), a.dw_post, a.dw_pre, dgate);
}

// Threads per row and vectors per thread by the row's vectors: the smallest
// block that holds the row with two vectors a thread (four for the longest
// rows of fp32, eight or sixteen single elements where rows do not start on
// 16 bytes).
#define PROJ_NORM_PICK(FN, T, a, s)                                          \
  if (vec) {                                                                 \
    constexpr int V = kFullVec<T>;                                           \
    const int64_t n = (a).D / V;                                             \
    if (n <= 64) return FN<T, V, 32, 2>(a, s);                               \
    if (n <= 256) return FN<T, V, 128, 2>(a, s);                             \
    if (n <= 512) return FN<T, V, 256, 2>(a, s);                             \
    if (n <= 1024) return FN<T, V, 512, 2>(a, s);                            \
    if (V == 4 && n > 2048) return FN<T, V, 1024, 4>(a, s);                  \
    return FN<T, V, 1024, 2>(a, s);                                          \
  } else {                                                                   \
    if ((a).D <= 256) return FN<T, 1, 32, 8>(a, s);                          \
    if ((a).D <= 2048) return FN<T, 1, 256, 8>(a, s);                        \
    if ((a).D <= 8192) return FN<T, 1, 1024, 8>(a, s);                       \
    return FN<T, 1, 1024, 16>(a, s);                                         \
  }

template <typename T>
cudaError_t forward_any(const proj_norm_args& a, bool vec, cudaStream_t s) {
  PROJ_NORM_PICK(forward, T, a, s)
}

template <typename T>
cudaError_t backward_any(const proj_norm_grad_args& a, bool vec, cudaStream_t s) {
  PROJ_NORM_PICK(backward, T, a, s)
}

int element_size(int dtype) { return dtype == PROJ_FP32 ? 4 : 2; }

bool aligned_to(const void* p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// What both calls ask of their common fields; nullptr if they are fine.
template <typename A>
const char* refuse_common(const A& a, int* status) {
  *status = PROJ_EINVAL;
  if (a.m < 0 || a.D < 1) return "m < 0 or D < 1";
  if (a.dtype != PROJ_BF16 && a.dtype != PROJ_FP16 && a.dtype != PROJ_FP32) return "unknown dtype";
  if (a.gate_mode < PROJ_GATE_NONE || a.gate_mode > PROJ_GATE_TOKEN) return "unknown gate_mode";
  if (a.gate_act != PROJ_GATE_LINEAR && a.gate_act != PROJ_GATE_SIGMOID) return "unknown gate_act";
  if (a.y_plain != 0 && a.y_plain != 1) return "y_plain is neither 0 nor 1";
  if (!(a.eps >= 0.f)) return "eps is negative or NaN";
  if (a.m > 0 && !a.residual) return "residual is NULL";
  if (a.m > 0 && (a.gate_mode == PROJ_GATE_NONE) != (a.gate == nullptr))
    return "gate and gate_mode do not agree";
  if (a.m > 0 && !a.y && (a.w_post || a.rstd_post || a.gate || a.y_plain))
    return "y is NULL, but w_post, rstd_post, gate or y_plain is set";
  if (a.y_plain && (a.w_post || a.rstd_post)) return "y_plain with w_post or rstd_post";
  if ((a.y && a.ldy < a.D) || a.ldr < a.D || (a.gate_mode == PROJ_GATE_ELEMENT && a.ldg < a.D))
    return "a row stride is below D";
  *status = PROJ_EUNSUPPORTED;
  if (a.D > kMaxD) return "D > 16384";
  if (a.m >= (int64_t{1} << 31)) return "m >= 2^31";
  const int el = element_size(a.dtype);
  *status = PROJ_EALIGN;
  if (!aligned_to(a.y, el) || !aligned_to(a.residual, el) || !aligned_to(a.gate, el) ||
      !aligned_to(a.w_post, el) || !aligned_to(a.w_pre, el))
    return "a pointer is not aligned to an element";
  if (!aligned_to(a.rstd_post, 4) || !aligned_to(a.rstd_pre, 4))
    return "a statistics pointer is not aligned to 4 bytes";
  *status = PROJ_OK;
  return nullptr;
}

// Whether rows of the tensor all start on 16 bytes (a NULL one does).
bool rows16(const void* p, int64_t ld, int el) {
  return !p || (aligned_to(p, 16) && (ld * el) % 16 == 0);
}

template <typename A>
bool common_rows16(const A& a, int el) {
  const bool gate_ok = a.gate_mode == PROJ_GATE_ELEMENT   ? rows16(a.gate, a.ldg, el)
                       : a.gate_mode == PROJ_GATE_CHANNEL ? rows16(a.gate, 0, el)
                                                          : true;
  return (a.D * el) % 16 == 0 && rows16(a.y, a.ldy, el) && rows16(a.residual, a.ldr, el) &&
         gate_ok && rows16(a.w_post, 0, el) && rows16(a.w_pre, 0, el);
}

int refuse(int status, const char* call, const char* why) {
  char text[160];
  std::snprintf(text, sizeof text, "%s: %s", call, why);
  return record_status(status, text);
}

}  // namespace
}  // namespace proj

using namespace proj;

extern "C" int proj_norm(const proj_norm_args* args, proj_stream stream) {
  if (!args) return refuse(PROJ_EINVAL, "proj_norm", "args is NULL");
  const proj_norm_args a = *args;
  int status = PROJ_OK;
  if (const char* why = refuse_common(a, &status)) return refuse(status, "proj_norm", why);
  if (a.m > 0 && !a.out && !a.normed) return refuse(PROJ_EINVAL, "proj_norm", "out and normed are both NULL");
  if ((a.out && a.ldo < a.D) || (a.normed && a.ldn < a.D))
    return refuse(PROJ_EINVAL, "proj_norm", "a row stride is below D");
  const int el = element_size(a.dtype);
  if (!aligned_to(a.out, el) || !aligned_to(a.normed, el))
    return refuse(PROJ_EALIGN, "proj_norm", "a pointer is not aligned to an element");
  if (a.m == 0) return PROJ_OK;
  const bool vec = common_rows16(a, el) && rows16(a.out, a.ldo, el) && rows16(a.normed, a.ldn, el);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = a.dtype == PROJ_BF16   ? forward_any<__nv_bfloat16>(a, vec, s)
                        : a.dtype == PROJ_FP16 ? forward_any<__half>(a, vec, s)
                                               : forward_any<float>(a, vec, s);
  return e == cudaSuccess ? PROJ_OK : record_cuda(e, "proj_norm: kernel launch");
}

extern "C" int64_t proj_norm_workspace(int64_t m, int64_t D) {
  if (m < 0 || D < 1 || D > kMaxD) {
    refuse(PROJ_EINVAL, "proj_norm_workspace", "m < 0 or D outside 1 .. 16384");
    return -1;
  }
  // rows are rounded up to the four that a block of warps holds
  return static_cast<int64_t>((grad_parts(m) + 3) / 4 * 4) * 3 * D * 4;
}

extern "C" int proj_norm_backward(const proj_norm_grad_args* args, proj_stream stream) {
  const char* const call = "proj_norm_backward";
  if (!args) return refuse(PROJ_EINVAL, call, "args is NULL");
  const proj_norm_grad_args a = *args;
  int status = PROJ_OK;
  if (const char* why = refuse_common(a, &status)) return refuse(status, call, why);
  if (a.m > 0 && !a.dout && !a.dnormed) return refuse(PROJ_EINVAL, call, "dout and dnormed are both NULL");
  if (a.m > 0 && a.y && !a.y_plain && !a.rstd_post) return refuse(PROJ_EINVAL, call, "rstd_post is NULL");
  if (a.m > 0 && a.dnormed && !a.rstd_pre) return refuse(PROJ_EINVAL, call, "rstd_pre is NULL");
  if (a.m > 0 && !a.y && (a.dy || a.dw_post || a.dgate))
    return refuse(PROJ_EINVAL, call, "y is NULL, but dy, dw_post or dgate is wanted");
  if (a.y_plain && a.dw_post) return refuse(PROJ_EINVAL, call, "y_plain has no dw_post");
  if (a.m > 0 && !a.gate && a.dgate) return refuse(PROJ_EINVAL, call, "dgate without a gate");
  if ((a.dout && a.lddo < a.D) || (a.dnormed && a.lddn < a.D) || (a.dy && a.lddy < a.D) ||
      (a.dresidual && a.lddr < a.D) ||
      (a.dgate && a.gate_mode == PROJ_GATE_ELEMENT && a.lddg < a.D))
    return refuse(PROJ_EINVAL, call, "a row stride is below D");
  const bool col_gate = a.dgate && a.gate_mode == PROJ_GATE_CHANNEL;
  const bool columns = a.dw_post || a.dw_pre || col_gate;
  if (a.m > 0 && columns && (!a.workspace || a.workspace_bytes < proj_norm_workspace(a.m, a.D)))
    return refuse(PROJ_EINVAL, call, "workspace is NULL or too small");
  const int el = element_size(a.dtype);
  if (!aligned_to(a.dout, el) || !aligned_to(a.dnormed, el) || !aligned_to(a.dy, el) ||
      !aligned_to(a.dresidual, el))
    return refuse(PROJ_EALIGN, call, "a pointer is not aligned to an element");
  if (!aligned_to(a.dgate, col_gate ? 4 : el) || !aligned_to(a.dw_post, 4) ||
      !aligned_to(a.dw_pre, 4))
    return refuse(PROJ_EALIGN, call, "a gradient is not aligned to an element");
  if (columns && !aligned_to(a.workspace, 16))
    return refuse(PROJ_EALIGN, call, "workspace is not 16-byte aligned");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (a.m == 0) {  // sums over no rows
    const size_t n = static_cast<size_t>(a.D) * 4;
    if (a.dw_post) e = cudaMemsetAsync(a.dw_post, 0, n, s);
    if (a.dw_pre && e == cudaSuccess) e = cudaMemsetAsync(a.dw_pre, 0, n, s);
    if (col_gate && e == cudaSuccess) e = cudaMemsetAsync(a.dgate, 0, n, s);
    return e == cudaSuccess ? PROJ_OK : record_cuda(e, "proj_norm_backward: clearing sums");
  }
  const bool gate_ok = a.gate_mode != PROJ_GATE_ELEMENT || rows16(a.dgate, a.lddg, el);
  const bool vec = common_rows16(a, el) && gate_ok && rows16(a.dout, a.lddo, el) &&
                   rows16(a.dnormed, a.lddn, el) && rows16(a.dy, a.lddy, el) &&
                   rows16(a.dresidual, a.lddr, el);
  e = a.dtype == PROJ_BF16   ? backward_any<__nv_bfloat16>(a, vec, s)
      : a.dtype == PROJ_FP16 ? backward_any<__half>(a, vec, s)
                             : backward_any<float>(a, vec, s);
  return e == cudaSuccess ? PROJ_OK : record_cuda(e, "proj_norm_backward: kernel launch");
}
