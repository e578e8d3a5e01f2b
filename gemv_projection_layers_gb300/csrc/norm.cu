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
// Both kernels are bound by HBM: a row of D = 8192 in 16 bits moves 64 KB
// forward and 128 KB backward.  A CTA takes rows in turn and has the next rows'
// tensors on their way to shared memory (16-byte asynchronous copies) while it
// works on one, so the two reductions of a row hide behind the loads of
// others, and both passes over a row read shared memory.  The gradient's
// column sums stay in registers over all of a CTA's rows and meet in a second
// kernel, in a fixed order.  The forward kernel comes to 0.8 of the measured
// copy rate (8192 x 8192 bf16, a gate per element: 125 us, 5.4 TB/s).  The
// gradient, with its column sums in registers, has 16 warps an SM -- of long
// rows, one row at a time: 55 % of the cycles issue one of its some 100
// instructions an element, in the others its warps wait for their operands or
// at the barrier between the passes, and there is no other row to turn to.  (8192 rows bf16, a sigmoid gate per element: 8192 columns 320 us,
// 3.4 TB/s; 1024, where four warps work on a row, 71 us, 1.9 TB/s; 512, a warp a
// row, 30 us.)
//
// Rows that do not start on 16 bytes (an odd D, say) keep their misalignment
// in shared memory, where the 16-byte words that hold them go, and the threads
// read and write single elements, neighbours side by side.
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

// The sigmoid's exponential and reciprocal: the 16-bit types' outputs are
// rounded to 2^-8 or 2^-11, so the hardware's approximations (2^-21 or so, of
// the value and of the slope) do; fp32 takes expf and a true quotient.
template <typename T>
__device__ __forceinline__ float sigmoid(float g) {
  if constexpr (sizeof(T) == 2) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
  } else {
    return 1.f / (1.f + expf(-g));
  }
}
template <typename T>
__device__ __forceinline__ float act(float g, int kind) {
  return kind == PROJ_GATE_SIGMOID ? sigmoid<T>(g) : g;
}
template <typename T, int E>
__device__ __forceinline__ void act_all(float (&g)[E], int kind) {
  if (kind != PROJ_GATE_SIGMOID) return;
#pragma unroll
  for (int i = 0; i < E; ++i) g[i] = sigmoid<T>(g[i]);
}
// d act / d gate, from the gate x and its value g: 1, or the sigmoid's
// sigmoid(x) sigmoid(-x).  1 - g cancels where the gate is open (in fp32 a
// relative error of 1e-4 at x = 8, and nothing is left from x = 17), so there
// sigmoid(-x) = exp(-x) g.
template <typename T>
__device__ __forceinline__ float act_slope(float x, float g, int kind) {
  if (kind != PROJ_GATE_SIGMOID) return 1.f;
  float e;
  if constexpr (sizeof(T) == 2)
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
  else
    e = expf(-x);
  return g * (x > 0.f ? e * g : 1.f - g);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
__device__ __forceinline__ void cp_async_wait_all_but(int pending) {
  if (pending <= 0)
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  else if (pending == 1)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 2;" ::: "memory");
}

// How TPR threads share a row.  kVec: group j of a thread is the 16 bytes at
// element (j TPR + tid) E; else E elements TPR apart, from j E TPR + tid.
template <typename T, bool kVec_, int TPR_, int NV_, bool kRing_ = (TPR_ >= 128 && TPR_ <= 512)>
struct Shape {
  using Type = T;
  static constexpr bool kVec = kVec_;
  static constexpr int TPR = TPR_, NV = NV_;
  static constexpr int E = kVec ? kFullVec<T> : 4;
  static constexpr int kRows = TPR < 128 ? 128 / TPR : 1;  // rows of a CTA at a time
  static constexpr int kThreads = TPR < 128 ? 128 : TPR;
  static constexpr bool kRing = kRing_;  // rows come through shared memory
  // threads of an SM in the forward kernel, by its registers
  static constexpr int kResident = kVec && NV == 1 ? 1536 : 1024;
};

// Whether the row reaches group j of a thread (kVec: with all of it, or not at
// all).  The groups that it does not reach are skipped by the callers of what
// follows; of the others, elements beyond D are 0.
template <typename S>
__device__ __forceinline__ bool reaches(int j, int tid, int D) {
  return S::kVec ? (j * S::TPR + tid) * S::E < D : j * S::E * S::TPR + tid < D;
}

// Group j of a row in global memory.
template <typename S>
__device__ __forceinline__ void load_global(const typename S::Type* row, int j, int tid, int D,
                                            float (&v)[S::E]) {
  using T = typename S::Type;
  if constexpr (S::kVec) {
    widen(load_vec<T, S::E>(row + (j * S::TPR + tid) * S::E), v);
  } else {
    const int c0 = j * S::E * S::TPR + tid;
    if ((j + 1) * S::E * S::TPR <= D) {
#pragma unroll
      for (int i = 0; i < S::E; ++i) v[i] = to_f32(row[c0 + i * S::TPR]);
    } else {
#pragma unroll
      for (int i = 0; i < S::E; ++i)
        v[i] = c0 + i * S::TPR < D ? to_f32(row[c0 + i * S::TPR]) : 0.f;
    }
  }
}

// The same of a row in shared memory, by its 32-bit address (generic loads
// are slower).
template <typename T>
__device__ __forceinline__ float load_shared_one(uint32_t addr) {
  if constexpr (sizeof(T) == 4) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
  } else {
    uint16_t b;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(b) : "r"(addr));
    return to_f32(*reinterpret_cast<const T*>(&b));
  }
}
template <typename S>
__device__ __forceinline__ void load_shared(uint32_t row, int j, int tid, int D,
                                            float (&v)[S::E]) {
  using T = typename S::Type;
  constexpr int el = sizeof(T);
  if constexpr (S::kVec) {
    const uint4 b = ld_shared_u4(row + (j * S::TPR + tid) * S::E * el);
    widen(*reinterpret_cast<const Vec<T, S::E>*>(&b), v);
  } else {
    const int c0 = j * S::E * S::TPR + tid;
    if ((j + 1) * S::E * S::TPR <= D) {
#pragma unroll
      for (int i = 0; i < S::E; ++i) v[i] = load_shared_one<T>(row + (c0 + i * S::TPR) * el);
    } else {
#pragma unroll
      for (int i = 0; i < S::E; ++i)
        v[i] = c0 + i * S::TPR < D ? load_shared_one<T>(row + (c0 + i * S::TPR) * el) : 0.f;
    }
  }
}

template <typename S>
__device__ __forceinline__ void store_global(typename S::Type* row, int j, int tid, int D,
                                             const float (&v)[S::E]) {
  using T = typename S::Type;
  if constexpr (S::kVec) {
    store_vec<T, S::E>(row + (j * S::TPR + tid) * S::E, v);
  } else {
    const int c0 = j * S::E * S::TPR + tid;
    if ((j + 1) * S::E * S::TPR <= D) {
#pragma unroll
      for (int i = 0; i < S::E; ++i) row[c0 + i * S::TPR] = from_f32<T>(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < S::E; ++i)
        if (c0 + i * S::TPR < D) row[c0 + i * S::TPR] = from_f32<T>(v[i]);
    }
  }
}

// Up to five row tensors and their ring in shared memory.
template <typename S, int NT>
struct Rows {
  using T = typename S::Type;
  const T* base[NT];  // null: not there
  int64_t ld[NT];
  uint8_t* smem;
  int64_t m;
  int D, slot, stages;  // bytes of a row's place, stages of NT places

  __device__ __forceinline__ static int skew(const T* p) {
    return S::kVec ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15);
  }
  __device__ __forceinline__ uint8_t* place(int stage, int k) const {
    return smem + (stage * NT + k) * slot;
  }
  // The threads of the CTA start the copies of one row.
  __device__ __forceinline__ void fetch(int64_t row, int stage, int tid) const {
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      if (!base[k]) continue;
      const T* src = base[k] + row * ld[k];
      uint8_t* dst = place(stage, k);
      if constexpr (S::kVec) {
        const uint32_t to = smem_u32(dst);
        // a thread copies the groups that it reads
#pragma unroll
        for (int j = 0; j < S::NV; ++j) {
          const int c = (j * S::TPR + tid) * S::E;
          if (c < D) cp_async16(to + c * static_cast<int>(sizeof(T)), src + c);
        }
      } else {
        // The 16-byte words that hold the row.  Those at its ends may hold
        // elements of other rows, or between them, which nobody uses; words
        // that reach out of the tensor go element by element.
        constexpr int el = sizeof(T);
        const char* const begin = reinterpret_cast<const char*>(base[k]);
        const char* const end = reinterpret_cast<const char*>(base[k] + (m - 1) * ld[k] + D);
        const char* const row_begin = reinterpret_cast<const char*>(src);
        const char* const row_end = row_begin + D * el;
        const int off = skew(src);
        const uint32_t to = smem_u32(dst);
        const int words = (off + D * el + 15) / 16;
        for (int i = tid; i < words; i += S::TPR) {
          const char* const w = row_begin - off + 16 * i;
          if (w >= begin && w + 16 <= end) {
            cp_async16(to + 16 * i, w);
          } else {
            for (int e = 0; e < 16; e += el)
              if (w + e >= row_begin && w + e < row_end)
                *reinterpret_cast<T*>(dst + 16 * i + e) = *reinterpret_cast<const T*>(w + e);
          }
        }
      }
    }
  }
};

// The tensors of the row at hand: where they stand.
template <typename S, int NT>
struct Row {
  using T = typename S::Type;
  const T* global[NT];
  uint32_t shared[NT];
  int D, tid;

  __device__ __forceinline__ Row(const Rows<S, NT>& rows, int64_t row, int stage, int tid_)
      : D(rows.D), tid(tid_) {
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      global[k] = rows.base[k] + row * rows.ld[k];
      shared[k] = smem_u32(rows.place(stage, k)) + Rows<S, NT>::skew(global[k]);
    }
  }
  // Group j of tensor k.
  __device__ __forceinline__ void load(int k, int j, float (&v)[S::E]) const {
    if constexpr (!S::kRing)
      load_global<S>(global[k], j, tid, D, v);
    else
      load_shared<S>(shared[k], j, tid, D, v);
  }
};

// The threads of a row have come here: a warp, or the CTA.
template <typename S>
__device__ __forceinline__ void row_sync() {
  if constexpr (S::TPR == 32)
    __syncwarp();
  else
    __syncthreads();
}

// The loop over a CTA's rows: work(row, stage) for rows first, first + step, ...
// with the next rows' copies under way.  Work has a block barrier between its
// two passes or none; without shared columns between threads (kVec) a thread
// waits for its own copies only.
template <typename S, typename R, typename F>
__device__ __forceinline__ void over_rows(const R& rows, int64_t m, int64_t first, int64_t step,
                                          int tid, F work) {
  if constexpr (!S::kRing) {
    for (int64_t row = first; row < m; row += step) work(row, 0);
  } else {
    const int ahead = rows.stages - 1;
    for (int i = 0; i < ahead; ++i) {
      if (first + i * step < m) rows.fetch(first + i * step, i, tid);
      cp_async_commit();
    }
    int stage = 0;
    for (int64_t row = first; row < m; row += step) {
      if (ahead == 0) {
        if (!S::kVec) row_sync<S>();  // the row before has been read
        rows.fetch(row, 0, tid);
        cp_async_commit();
      }
      cp_async_wait_all_but(ahead - 1);
      if (!S::kVec) row_sync<S>();
      if (ahead) {
        const int into = stage == 0 ? ahead : stage - 1;  // the stage of the row before
        if (row + ahead * step < m) rows.fetch(row + ahead * step, into, tid);
        cp_async_commit();
      }
      work(row, stage);
      if (++stage == rows.stages) stage = 0;
    }
  }
}

template <typename S>
__global__ void __launch_bounds__(S::kThreads, S::kResident / S::kThreads)
    norm_kernel(const __grid_constant__ proj_norm_args a, const int slot, const int stages) {
  using T = typename S::Type;
  constexpr int NV = S::NV, E = S::E, TPR = S::TPR;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float room[2 * 32];
  int turn = 0;
  const int tid = static_cast<int>(threadIdx.x) % TPR;
  griddep_launch_dependents();
  griddep_wait();
  const int D = static_cast<int>(a.D);
  const float inv_d = 1.f / static_cast<float>(D);
  const bool g_vec = a.gate_mode == PROJ_GATE_CHANNEL || a.gate_mode == PROJ_GATE_ELEMENT;
  Rows<S, 3> rows;
  rows.base[0] = static_cast<const T*>(a.residual);
  rows.ld[0] = a.ldr;
  rows.base[1] = static_cast<const T*>(a.y);
  rows.ld[1] = a.ldy;
  rows.base[2] = a.gate_mode == PROJ_GATE_ELEMENT ? static_cast<const T*>(a.gate) : nullptr;
  rows.ld[2] = a.ldg;
  rows.smem = smem + threadIdx.x / TPR * (stages * 3) * slot;
  rows.m = a.m;
  rows.D = D;
  rows.slot = slot;
  rows.stages = stages;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * S::kRows + threadIdx.x / TPR;

  over_rows<S>(rows, a.m, first, static_cast<int64_t>(gridDim.x) * S::kRows, tid,
               [&](int64_t row, int stage) {
    const Row<S, 3> at(rows, row, stage, tid);
    float rp = 1.f;
    if (a.y && !a.y_plain) {
      float s[1] = {0.f};
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!reaches<S>(j, tid, D)) break;
        float v[E];
        at.load(1, j, v);
#pragma unroll
        for (int i = 0; i < E; ++i) s[0] = fmaf(v[i], v[i], s[0]);
      }
      row_sums<TPR, 1>(s, room, turn);
      rp = 1.f / sqrtf(s[0] * inv_d + a.eps);
      if (tid == 0 && a.rstd_post) a.rstd_post[row] = rp;
    }
    float g_row = 1.f;
    if (a.gate_mode == PROJ_GATE_TOKEN)
      g_row = act<T>(to_f32(static_cast<const T*>(a.gate)[row]), a.gate_act);
    float u[NV][E];
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!reaches<S>(j, tid, D)) break;
      at.load(0, j, u[j]);
#pragma unroll
      for (int i = 0; i < E; ++i) u[j][i] *= a.alpha;
      if (a.y) {
        float n[E], w[E];
        at.load(1, j, n);
#pragma unroll
        for (int i = 0; i < E; ++i) n[i] *= rp;
        if (a.w_post) {
          load_global<S>(static_cast<const T*>(a.w_post), j, tid, D, w);
#pragma unroll
          for (int i = 0; i < E; ++i) n[i] *= w[i];
        }
        if (g_vec) {
          if (a.gate_mode == PROJ_GATE_ELEMENT)
            at.load(2, j, w);
          else
            load_global<S>(static_cast<const T*>(a.gate), j, tid, D, w);
          act_all<T>(w, a.gate_act);
        } else {
#pragma unroll
          for (int i = 0; i < E; ++i) w[i] = g_row;
        }
#pragma unroll
        for (int i = 0; i < E; ++i) u[j][i] = fmaf(a.beta * w[i], n[i], u[j][i]);
      }
      if (a.out) store_global<S>(static_cast<T*>(a.out) + row * a.ldo, j, tid, D, u[j]);
#pragma unroll
      for (int i = 0; i < E; ++i) s[0] = fmaf(u[j][i], u[j][i], s[0]);
    }
    if (!a.normed && !a.rstd_pre) return;
    row_sums<TPR, 1>(s, room, turn);
    const float ru = 1.f / sqrtf(s[0] * inv_d + a.eps);
    if (tid == 0 && a.rstd_pre) a.rstd_pre[row] = ru;
    if (!a.normed) return;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!reaches<S>(j, tid, D)) break;
      if (a.w_pre) {
        float w[E];
        load_global<S>(static_cast<const T*>(a.w_pre), j, tid, D, w);
#pragma unroll
        for (int i = 0; i < E; ++i) u[j][i] *= ru * w[i];
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) u[j][i] *= ru;
      }
      store_global<S>(static_cast<T*>(a.normed) + row * a.ldn, j, tid, D, u[j]);
    }
  });
}

// Column sums: part[CTA row][which][D] (which: 0 dw_post, 1 dw_pre, 2 dgate).
template <typename S>
__global__ void __launch_bounds__(S::kThreads, S::kThreads < 512 ? 512 / S::kThreads : 1)
    norm_grad_kernel(const __grid_constant__ proj_norm_grad_args a, const int slot,
                     const int stages) {
  using T = typename S::Type;
  constexpr int NV = S::NV, E = S::E, TPR = S::TPR;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float room[2 * 3 * 32];
  int turn = 0;
  const int tid = static_cast<int>(threadIdx.x) % TPR;
  const int first = static_cast<int>(blockIdx.x) * S::kRows + threadIdx.x / TPR;
  griddep_launch_dependents();
  griddep_wait();
  const int D = static_cast<int>(a.D);
  const float inv_d = 1.f / static_cast<float>(D);
  const bool normed = a.y && !a.y_plain;
  const bool g_vec = a.gate_mode == PROJ_GATE_CHANNEL || a.gate_mode == PROJ_GATE_ELEMENT;
  const bool g_token = a.gate_mode == PROJ_GATE_TOKEN;
  const bool g_channel = a.gate_mode == PROJ_GATE_CHANNEL;
  Rows<S, 5> rows;
  rows.base[0] = static_cast<const T*>(a.residual);
  rows.ld[0] = a.ldr;
  rows.base[1] = static_cast<const T*>(a.y);
  rows.ld[1] = a.ldy;
  rows.base[2] = a.gate_mode == PROJ_GATE_ELEMENT ? static_cast<const T*>(a.gate) : nullptr;
  rows.ld[2] = a.ldg;
  rows.base[3] = static_cast<const T*>(a.dout);
  rows.ld[3] = a.lddo;
  rows.base[4] = static_cast<const T*>(a.dnormed);
  rows.ld[4] = a.lddn;
  rows.smem = smem + threadIdx.x / TPR * (stages * 5) * slot;
  rows.m = a.m;
  rows.D = D;
  rows.slot = slot;
  rows.stages = stages;

  constexpr int H = E / 2;  // the arithmetic runs on pairs of elements
  // Eight elements a thread stay in registers between the passes; of sixteen the
  // second pass makes them anew.
  constexpr bool kKeep = NV * E <= 8 && TPR <= 512;
  constexpr int kKept = kKeep ? NV : 1;
  const F2 zero = f2(0.f), one = f2(1.f);
  const F2 alpha = f2(a.alpha), beta = f2(a.beta);
  // dw_post and dw_pre; for a gate per channel the first holds sum_rows beta du yn,
  // of which dw_post is g times and the gate's gradient n / yn act' times
  F2 acc_post[NV][H], acc_pre[NV][H];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < H; ++i) acc_post[j][i] = acc_pre[j][i] = zero;

  float rp_next = 1.f, ru_next = 1.f;  // the next row's factors, read a row ahead
  auto factors = [&](int64_t row) {
    if (row >= a.m) return;
    if (normed) rp_next = a.rstd_post[row];
    if (a.dnormed) ru_next = a.rstd_pre[row];
  };
  factors(first);

  over_rows<S>(rows, a.m, first, static_cast<int64_t>(gridDim.x) * S::kRows, tid,
               [&](int64_t row, int stage) {
    const Row<S, 5> at(rows, row, stage, tid);
    const F2 rp = f2(rp_next);
    const float ru_row = ru_next;
    const F2 ru = f2(ru_row);
    factors(row + static_cast<int64_t>(gridDim.x) * S::kRows);
    const float raw_row = g_token ? to_f32(static_cast<const T*>(a.gate)[row]) : 1.f;
    const float g_row = g_token ? act<T>(raw_row, a.gate_act) : 1.f;
    // group j's yn, n, un, dh, t = dh w_pre and e = du' + ru t, and w_post, with the
    // activated gate in g
    F2 yn_[kKept][H], n_[kKept][H], un_[kKept][H], dh_[kKept][H], t_[kKept][H], e_[kKept][H],
        wpo_[kKept][H];
    auto group = [&](int j, const F2 (&g)[H]) {
      const int at_j = kKeep ? j : 0;
      F2(&yn)[H] = yn_[at_j], (&n)[H] = n_[at_j], (&un)[H] = un_[at_j], (&dh)[H] = dh_[at_j];
      F2(&t)[H] = t_[at_j], (&e)[H] = e_[at_j], (&wpo)[H] = wpo_[at_j];
      float v[E];
      at.load(0, j, v);
      pairs<E>(v, un);
#pragma unroll
      for (int i = 0; i < H; ++i) un[i] = mul2(un[i], alpha);
      if (a.w_post) {
        load_global<S>(static_cast<const T*>(a.w_post), j, tid, D, v);
        pairs<E>(v, wpo);
      } else {
#pragma unroll
        for (int i = 0; i < H; ++i) wpo[i] = one;
      }
      if (a.y) {
        at.load(1, j, v);
        pairs<E>(v, yn);
#pragma unroll
        for (int i = 0; i < H; ++i) {
          yn[i] = mul2(yn[i], rp);
          n[i] = mul2(yn[i], wpo[i]);
          un[i] = fma2(mul2(beta, g[i]), n[i], un[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < H; ++i) yn[i] = n[i] = zero;
      }
      if (a.dout) {
        at.load(3, j, v);
        pairs<E>(v, e);
      } else {
#pragma unroll
        for (int i = 0; i < H; ++i) e[i] = zero;
      }
      if (a.dnormed) {
        at.load(4, j, v);
        pairs<E>(v, dh);
        if (a.w_pre) {
          load_global<S>(static_cast<const T*>(a.w_pre), j, tid, D, v);
          pairs<E>(v, t);
#pragma unroll
          for (int i = 0; i < H; ++i) t[i] = mul2(dh[i], t[i]);
        } else {
#pragma unroll
          for (int i = 0; i < H; ++i) t[i] = dh[i];
        }
#pragma unroll
        for (int i = 0; i < H; ++i) {
          un[i] = mul2(un[i], ru);
          e[i] = fma2(ru, t[i], e[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < H; ++i) dh[i] = t[i] = zero;
      }
    };
    F2 g[NV][H];
    F2 s2x[3] = {zero, zero, zero};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!reaches<S>(j, tid, D)) break;
      if (g_vec) {
        float v[E];
        if (a.gate_mode == PROJ_GATE_ELEMENT)
          at.load(2, j, v);
        else
          load_global<S>(static_cast<const T*>(a.gate), j, tid, D, v);
        act_all<T>(v, a.gate_act);
        pairs<E>(v, g[j]);
      } else {
#pragma unroll
        for (int i = 0; i < H; ++i) g[j][i] = f2(g_row);
      }
      group(j, g[j]);
      const int at_j = kKeep ? j : 0;
      F2(&n)[H] = n_[at_j], (&un)[H] = un_[at_j], (&t)[H] = t_[at_j], (&e)[H] = e_[at_j];
#pragma unroll
      for (int i = 0; i < H; ++i) {
        s2x[0] = fma2(t[i], un[i], s2x[0]);
        const F2 gn = g_token ? n[i] : mul2(g[j][i], n[i]);
        s2x[1] = fma2(gn, e[i], s2x[1]);
        s2x[2] = fma2(gn, un[i], s2x[2]);
      }
    }
    float s[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      float x, y;
      parts(s2x[i], x, y);
      s[i] = x + y;
    }
    row_sums<TPR, 3>(s, room, turn);
    if constexpr (TPR == 32) __syncwarp();  // keeps the passes apart: fewer registers
    const float s1 = a.dnormed ? ru_row * s[0] * inv_d : 0.f;
    const float ab = a.beta * (s[1] - s1 * s[2]);  // sum of beta [g] n du
    const F2 s2 = f2(normed ? -(g_token ? g_row * ab : ab) * inv_d : 0.f);
    const F2 minus_s1 = f2(-s1);
    if (g_token && a.dgate && tid == 0)
      static_cast<T*>(a.dgate)[row] = from_f32<T>(ab * act_slope<T>(raw_row, g_row, a.gate_act));
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!reaches<S>(j, tid, D)) break;
      if constexpr (!kKeep) group(j, g[j]);
      const int at_j = kKeep ? j : 0;
      F2(&yn)[H] = yn_[at_j], (&n)[H] = n_[at_j], (&un)[H] = un_[at_j], (&dh)[H] = dh_[at_j];
      F2(&e)[H] = e_[at_j], (&wpo)[H] = wpo_[at_j];
      F2 o[H];
      float out[E];
#pragma unroll
      for (int i = 0; i < H; ++i) {
        if (a.dnormed) e[i] = fma2(un[i], minus_s1, e[i]);  // du
        o[i] = mul2(alpha, e[i]);
      }
      if (a.dresidual) {
        unpair<E>(o, out);
        store_global<S>(static_cast<T*>(a.dresidual) + row * a.lddr, j, tid, D, out);
      }
      if (a.dw_pre) {
#pragma unroll
        for (int i = 0; i < H; ++i) acc_pre[j][i] = fma2(dh[i], un[i], acc_pre[j][i]);
      }
      if (!a.y) continue;
#pragma unroll
      for (int i = 0; i < H; ++i) {
        e[i] = mul2(e[i], beta);
        const F2 c = mul2(g[j][i], e[i]);
        acc_post[j][i] = fma2(g_channel ? e[i] : c, yn[i], acc_post[j][i]);
        o[i] = normed ? mul2(rp, fma2(c, wpo[i], mul2(yn[i], s2))) : c;
      }
      if (a.dy) {
        unpair<E>(o, out);
        store_global<S>(static_cast<T*>(a.dy) + row * a.lddy, j, tid, D, out);
      }
      if (a.gate_mode == PROJ_GATE_ELEMENT && a.dgate) {
#pragma unroll
        for (int i = 0; i < H; ++i) o[i] = mul2(n[i], e[i]);
        unpair<E>(o, out);
        if (a.gate_act == PROJ_GATE_SIGMOID) {
          float v[E], gv[E];
          at.load(2, j, v);
          unpair<E>(g[j], gv);
#pragma unroll
          for (int i = 0; i < E; ++i) out[i] *= act_slope<T>(v[i], gv[i], PROJ_GATE_SIGMOID);
        }
        store_global<S>(static_cast<T*>(a.dgate) + row * a.lddg, j, tid, D, out);
      }
    }
  });
  const bool col_gate = g_channel && a.dgate;
  if (!a.dw_post && !a.dw_pre && !col_gate) return;
  float* const part = static_cast<float*>(a.workspace) + static_cast<size_t>(blockIdx.x) * 3 * D;
  // rows of one CTA meet in shared memory, where no copies are under way now
  float* const to =
      S::kRows > 1 ? reinterpret_cast<float*>(smem) + threadIdx.x / TPR * 3 * D : part;
  if (S::kRows > 1) __syncthreads();
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (!reaches<S>(j, tid, D)) break;
    float post[E], pre[E], gate[E];
    unpair<E>(acc_post[j], post);
    unpair<E>(acc_pre[j], pre);
#pragma unroll
    for (int i = 0; i < E; ++i) gate[i] = 0.f;
    if (g_channel) {
      float w[E];
      load_global<S>(static_cast<const T*>(a.gate), j, tid, D, gate);
      if (a.w_post) {
        load_global<S>(static_cast<const T*>(a.w_post), j, tid, D, w);
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) w[i] = 1.f;
      }
#pragma unroll
      for (int i = 0; i < E; ++i) {
        // fp32 outputs, once a column: the exact exponential whatever T is
        const float q = post[i], g = act<float>(gate[i], a.gate_act);
        post[i] = g * q;
        gate[i] = w[i] * act_slope<float>(gate[i], g, a.gate_act) * q;
      }
    }
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int c = S::kVec ? (j * TPR + tid) * E + i : (j * E + i) * TPR + tid;
      if (c < D) {
        to[c] = post[i];
        to[D + c] = pre[i];
        to[2 * D + c] = gate[i];
      }
    }
  }
  if constexpr (S::kRows > 1) {
    __syncthreads();
    const float* const all = reinterpret_cast<const float*>(smem);
    for (int c = threadIdx.x; c < 3 * D; c += S::kThreads) {
      float t = 0.f;
#pragma unroll
      for (int k = 0; k < S::kRows; ++k) t += all[k * 3 * D + c];
      part[c] = t;
    }
  }
}

// Sums the partial rows of each column in order: warps of a CTA take every
// kSumWarps-th row of 32 columns, then meet in shared memory.
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(32 * kSumWarps)
    norm_grad_sum_kernel(const float* part, int rows, int D, float* d0, float* d1, float* d2) {
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

cudaLaunchConfig_t config(unsigned grid_x, unsigned grid_y, unsigned threads, size_t smem,
                          cudaStream_t s, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid_x, grid_y);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// CTAs of the gradient, and with it rows of the column sums' workspace, at
// most: longer rows have more threads and fewer CTAs fit an SM.
constexpr int kGradSms = 152;
int grad_ctas(int64_t D) { return kGradSms * (D > 4096 ? 1 : D > 1024 ? 2 : 4); }

constexpr int kSmemMost = 220 * 1024;

// A row's place in shared memory (with room for its misalignment) and the
// stages of `tensors` places that fit `budget` (0 to `most`).
template <typename S>
void ring_shape(int64_t D, int tensors, int budget, int most, int* slot, int* stages) {
  *slot = static_cast<int>((D * sizeof(typename S::Type) + 15) / 16 * 16 + 16);
  *stages = S::kRing ? std::max(1, std::min(most, budget / (S::kRows * tensors * *slot))) : 0;
}

template <typename S>
cudaError_t forward(const proj_norm_args& a, cudaStream_t s) {
  // As many CTAs an SM as its registers hold, fewer where two stages of the
  // rows do not fit their part of its shared memory.
  int slot, stages;
  int ctas = S::kResident / S::kThreads;
  ring_shape<S>(a.D, 3, kSmemMost / ctas, 3, &slot, &stages);
  while (S::kRing && stages < 2 && ctas > 1)
    ring_shape<S>(a.D, 3, kSmemMost / --ctas, 3, &slot, &stages);
  const size_t smem = static_cast<size_t>(S::kRows) * 3 * slot * stages;
  if (smem > 48 * 1024) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e =
        allow_smem(reinterpret_cast<const void*>(norm_kernel<S>), kSmemMost, done);
    if (e != cudaSuccess) return e;
  }
  int64_t grid = (a.m + S::kRows - 1) / S::kRows;
  if (S::kRing) {
    const int per_sm =
        std::max(1, std::min(static_cast<int>(kSmemMost / smem), S::kResident / S::kThreads));
    grid = std::min<int64_t>(grid, static_cast<int64_t>(per_sm) * std::max(1, proj_num_sms()));
  }
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = config(static_cast<unsigned>(grid), 1, S::kThreads, smem, s, attr);
  return cudaLaunchKernelEx(&cfg, norm_kernel<S>, a, slot, stages);
}

template <typename S>
cudaError_t backward(const proj_norm_grad_args& a, cudaStream_t s) {
  // as many CTAs an SM as have 128 registers a thread (never more than grad_ctas)
  constexpr int per_sm = S::kThreads < 512 ? 512 / S::kThreads : 1;
  const int grid = static_cast<int>(
      std::min<int64_t>((a.m + S::kRows - 1) / S::kRows, kGradSms * per_sm));
  int slot, stages;
  ring_shape<S>(a.D, 5, kSmemMost / per_sm, 3, &slot, &stages);
  const size_t ring = static_cast<size_t>(S::kRows) * 5 * slot * stages;
  const size_t joined = S::kRows > 1 ? static_cast<size_t>(S::kRows) * 3 * a.D * 4 : 0;
  const size_t smem = std::max(ring, joined);
  if (smem > 48 * 1024) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e =
        allow_smem(reinterpret_cast<const void*>(norm_grad_kernel<S>), kSmemMost, done);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = config(static_cast<unsigned>(grid), 1, S::kThreads, smem, s, attr);
  cudaError_t e = cudaLaunchKernelEx(&cfg, norm_grad_kernel<S>, a, slot, stages);
  if (e != cudaSuccess) return e;
  float* dgate = a.gate_mode == PROJ_GATE_CHANNEL ? static_cast<float*>(a.dgate) : nullptr;
  if (!a.dw_post && !a.dw_pre && !dgate) return cudaSuccess;
  cfg = config(static_cast<unsigned>((a.D + 31) / 32), 3, 32 * kSumWarps, 0, s, attr);
  return cudaLaunchKernelEx(&cfg, norm_grad_sum_kernel,
                            static_cast<const float*>(static_cast<float*>(a.workspace)),
                            grid, static_cast<int>(a.D), a.dw_post, a.dw_pre, dgate);
}

// Threads per row by its length: 16 elements of 16 bits a thread (8 or 16 of
// fp32), a warp for the shortest rows, which has no ring forward (a ring: 7.6 us
// for 8192 x 128 bf16 against 6.9).  Eight elements are better for up to 1024
// columns forward (8192 x 520: 17.8 us against 20.6; 1024 the same) and up to
// 2048 in the gradient, whose second pass then finds them in registers (8192 x
// 2048: 90 us against 117; at 4096, with one row an SM at a time, 179 against
// 160).  Beyond 8192 columns there is no ring, and both passes read global
// memory.
template <typename T>
cudaError_t forward_any(const proj_norm_args& a, bool vec, cudaStream_t s) {
  if (vec) {
    const int64_t n = a.D / kFullVec<T>;
    if (n <= 64) return forward<Shape<T, true, 32, 2>>(a, s);
    if (a.D <= 1024) return forward<Shape<T, true, 128, 8 / kFullVec<T>>>(a, s);
    if (n <= 256) return forward<Shape<T, true, 128, 2>>(a, s);
    if (n <= 512) return forward<Shape<T, true, 256, 2>>(a, s);
    if (n <= 1024) return forward<Shape<T, true, 512, 2>>(a, s);
    if constexpr (kFullVec<T> == 4) {
      if (n <= 2048) return forward<Shape<T, true, 512, 4>>(a, s);
      return forward<Shape<T, true, 1024, 4>>(a, s);
    } else {
      return forward<Shape<T, true, 1024, 2>>(a, s);
    }
  }
  if (a.D <= 512) return forward<Shape<T, false, 32, 4>>(a, s);
  if (a.D <= 2048) return forward<Shape<T, false, 128, 4>>(a, s);
  if (a.D <= 4096) return forward<Shape<T, false, 256, 4>>(a, s);
  if (a.D <= 8192) return forward<Shape<T, false, 512, 4>>(a, s);
  return forward<Shape<T, false, 1024, 4>>(a, s);
}

template <typename T>
cudaError_t backward_any(const proj_norm_grad_args& a, bool vec, cudaStream_t s) {
  constexpr int kEight = 8 / kFullVec<T>;  // groups of eight elements
  if (vec) {
    const int64_t n = a.D / kFullVec<T>;
    if (n <= 64) return backward<Shape<T, true, 32, 2, true>>(a, s);
    if (a.D <= 1024) return backward<Shape<T, true, 128, kEight>>(a, s);
    if (a.D <= 2048) return backward<Shape<T, true, 256, kEight>>(a, s);
    if constexpr (kFullVec<T> == 8)
      if (a.D <= 4096) return backward<Shape<T, true, 256, 2>>(a, s);
    if (n <= 1024) return backward<Shape<T, true, 512, 2>>(a, s);
    if constexpr (kFullVec<T> == 4) {
      if (n <= 2048) return backward<Shape<T, true, 512, 4>>(a, s);
      return backward<Shape<T, true, 1024, 4>>(a, s);
    } else {
      return backward<Shape<T, true, 1024, 2>>(a, s);
    }
  }
  if (a.D <= 512) return backward<Shape<T, false, 32, 4, true>>(a, s);
  if (a.D <= 1024) return backward<Shape<T, false, 128, 2>>(a, s);
  if (a.D <= 2048) return backward<Shape<T, false, 256, 2>>(a, s);
  if (a.D <= 4096) return backward<Shape<T, false, 256, 4>>(a, s);
  if (a.D <= 8192) return backward<Shape<T, false, 512, 4>>(a, s);
  return backward<Shape<T, false, 1024, 4>>(a, s);
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
  return std::min<int64_t>(m, grad_ctas(D)) * 3 * D * 4;
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
