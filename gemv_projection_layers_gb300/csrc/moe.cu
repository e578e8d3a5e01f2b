// moe.cu -- tokens to their experts and back: choice of the k largest router
// logits, stable counting sort by expert, gather, weighted combine, and the
// gradients.
//
// The sort.  Entries (t, j) in flat order are cut into blocks, one per CTA,
// and a block into chunks of 32, one per warp.  In a chunk a lane's rank among
// equal experts comes from a match over the warp; per expert, chunk counts are
// summed over the chunks before it, block counts (the workspace table, [block]
// [expert]) over the blocks before it, and totals over the experts before it.
// All of it is whole-number arithmetic, stable and the same on every call (the
// shared atomic additions are of whole numbers, whose order does not matter).
// One block: one launch does everything.  More: a first launch chooses and
// counts, a second places.  (4096 tokens, 8 of 256 experts: 11 and 13 us; the
// choice is bound by its instructions, some 970 a token and warp.)  Of few
// blocks each sums the counts of all; of more than kScanBlocks a launch
// between the two does so once, or the time would grow with the tokens' square.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdio>

#include "../../include/proj.h"
#include "kernels.h"
#include "ptx.cuh"
#include "vec.cuh"

namespace proj {
namespace {

constexpr int kMaxExperts = 1024;
constexpr int kMaxK = 32;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kTableBytes = 96 * 1024;  // shared chunk table: [chunks][E] of 16 bits, at most

// ------------------------------------------------------------------ choice --

// A key that orders like the float, equal for +0 and -0; 0 for what is never
// chosen (NaN and -infinity).
__device__ __forceinline__ uint32_t order_key(float v) {
  if (!(v > -INFINITY)) return 0u;
  const uint32_t u = __float_as_uint(v + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
// exp(v - top) with the limit 1 at v == top, also where both are infinite.
__device__ __forceinline__ float exp_below(float v, float top) {
  return v == top ? 1.f : expf(v - top);
}

// One warp chooses for one token; EPL = experts a lane holds (expert
// i 32 + lane).  Lane j < k returns choice j (-1: none left) and its weight.
template <int EPL>
__device__ __forceinline__ void choose(const float* logits, int E, int k, int mode, int lane,
                                       int& expert, float& weight) {
  uint32_t key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = i * 32 + lane;
    key[i] = e < E ? order_key(logits[e]) : 0u;
  }
  float all = 0.f;
  uint32_t top = 0u;
  if (mode == PROJ_ROUTE_ALL) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) top = max(top, key[i]);
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    const float tv = key_value(top);
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (key[i]) all += exp_below(key_value(key[i]), tv);
    all = warp_sum(all);
  }
  expert = -1;
  uint32_t mine = 0u;
  for (int j = 0; j < k; ++j) {
    uint32_t best = 0u;
    int at = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (key[i] > best) {  // the first of equal ones: the lowest index of this lane
        best = key[i];
        at = i;
      }
    const uint32_t win = __reduce_max_sync(0xFFFFFFFFu, best);
    if (!win) break;  // nothing left to choose
    if (j == 0) top = win;
    const uint32_t idx = __reduce_min_sync(
        0xFFFFFFFFu, best == win ? static_cast<uint32_t>(at * 32 + lane) : 0xFFFFFFFFu);
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (static_cast<uint32_t>(i * 32 + lane) == idx) key[i] = 0u;
    if (lane == j) {
      expert = static_cast<int>(idx);
      mine = win;
    }
  }
  const float part = expert >= 0 ? exp_below(key_value(mine), key_value(top)) : 0.f;
  const float total = mode == PROJ_ROUTE_ALL ? all : warp_sum(part);
  weight = expert >= 0 ? part / total : 0.f;
}

// ------------------------------------------------------------------- sort --

struct SortParams {
  const float* logits;  // null: expert is an input
  int64_t ldl;
  int32_t* expert;
  float* weight;
  int32_t* offsets;  // null: choose only
  int32_t* order;
  int32_t* slot;
  int32_t* table;  // [blocks][E]
  int64_t m;
  int E, k, mode;
  int tokens;  // per block
  int blocks;
  bool scanned;  // the table holds sums over the blocks before, and behind them the totals
};

// Counts of each expert in the chunks of this block, from its entries'
// experts: table[chunk][e], and each entry's rank in its chunk left to the
// caller (recomputed from the same match).
__device__ __forceinline__ int chunk_rank(int e, bool real, int lane, int& count, bool& last) {
  const uint32_t same = __match_any_sync(0xFFFFFFFFu, real ? e : -1);
  count = __popc(same);
  const uint32_t below = same & ((1u << lane) - 1u);
  last = (same >> lane) == 1u;  // the highest lane of its expert writes the count
  return __popc(below);
}

// Exclusive sums over the E totals in s_total (E <= 1024), by the whole block;
// s_total becomes the exclusive sums, the grand total is returned.
__device__ __forceinline__ int scan_experts(int* s_total, int* s_warp, int E) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int v = tid < E ? s_total[tid] : 0;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += t;
  }
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  int w = s_warp[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xFFFFFFFFu, w, o);
    if (lane >= o) w += t;
  }
  const int before = warp ? __shfl_sync(0xFFFFFFFFu, w, warp - 1) : 0;
  const int total = __shfl_sync(0xFFFFFFFFu, w, 31);
  if (tid < E) s_total[tid] = before + inc - v;
  __syncthreads();
  return total;
}

__device__ __forceinline__ bool is_expert(int e, int E) { return e >= 0 && e < E; }

// Chooses (with logits) and counts; with one block also places.
template <int EPL>
__global__ void __launch_bounds__(kSortThreads) choose_count_kernel(const SortParams p) {
  extern __shared__ __align__(16) uint16_t s_table[];  // [chunks][E]
  __shared__ int s_total[kMaxExperts];
  __shared__ int s_warp[kSortWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_launch_dependents();
  griddep_wait();
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.tokens;
  const int nt = static_cast<int>(min(static_cast<int64_t>(p.tokens), p.m - t0));
  if (p.logits) {
    for (int t = warp; t < nt; t += kSortWarps) {
      int e;
      float w;
      choose<EPL>(p.logits + (t0 + t) * p.ldl, p.E, p.k, p.mode, lane, e, w);
      if (lane < p.k) {
        p.expert[(t0 + t) * p.k + lane] = e;
        p.weight[(t0 + t) * p.k + lane] = w;
      }
    }
  }
  if (!p.offsets) return;
  const int n = nt * p.k;
  const int chunks = (n + 31) / 32;
  for (int i = tid; i < (chunks * p.E + 1) / 2; i += kSortThreads)
    reinterpret_cast<uint32_t*>(s_table)[i] = 0u;
  __syncthreads();  // also publishes this block's choices to the block
  const int32_t* expert = p.expert + t0 * p.k;
  for (int c = warp; c < chunks; c += kSortWarps) {
    const int i = c * 32 + lane;
    const int e = i < n ? expert[i] : -1;
    const bool real = is_expert(e, p.E);
    int count;
    bool last;
    chunk_rank(e, real, lane, count, last);
    if (real && last) s_table[c * p.E + e] = static_cast<uint16_t>(count);
  }
  __syncthreads();
  // per expert: counts -> exclusive sums over the chunks
  int total = 0;
  if (tid < p.E) {
    for (int c = 0; c < chunks; ++c) {
      const int v = s_table[c * p.E + tid];
      s_table[c * p.E + tid] = static_cast<uint16_t>(total);
      total += v;
    }
    if (p.blocks > 1) p.table[static_cast<int64_t>(blockIdx.x) * p.E + tid] = total;
  }
  if (p.blocks > 1) return;
  if (tid < p.E) s_total[tid] = total;
  __syncthreads();
  const int kept = scan_experts(s_total, s_warp, p.E);
  if (tid < p.E) p.offsets[tid] = s_total[tid];
  if (tid == 0) p.offsets[p.E] = kept;
  for (int c = warp; c < chunks; c += kSortWarps) {
    const int i = c * 32 + lane;
    const int e = i < n ? expert[i] : -1;
    const bool real = is_expert(e, p.E);
    int count;
    bool last;
    const int rank = chunk_rank(e, real, lane, count, last);
    if (i < n) {
      const int at = real ? s_total[e] + s_table[c * p.E + e] + rank : -1;
      p.slot[i] = at;
      if (real) p.order[at] = i;
    }
  }
  for (int i = kept + tid; i < n; i += kSortThreads) p.order[i] = -1;
}

// Turns the blocks' counts of 32 experts into the sums over the blocks before,
// and writes the totals behind them: a lane an expert, a warp a run of blocks,
// twice over the table.
__global__ void __launch_bounds__(kSortThreads) scan_blocks_kernel(int32_t* table, int blocks,
                                                                   int E) {
  __shared__ int s_sum[kSortWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e = static_cast<int>(blockIdx.x) * 32 + lane;
  const int b0 = static_cast<int>(static_cast<int64_t>(warp) * blocks / kSortWarps);
  const int b1 = static_cast<int>(static_cast<int64_t>(warp + 1) * blocks / kSortWarps);
  griddep_launch_dependents();
  griddep_wait();
  int sum = 0;
  if (e < E) {
#pragma unroll 8
    for (int b = b0; b < b1; ++b) sum += table[static_cast<int64_t>(b) * E + e];
  }
  s_sum[warp][lane] = sum;
  __syncthreads();
  if (e >= E) return;
  int run = 0;
  for (int w = 0; w < warp; ++w) run += s_sum[w][lane];
#pragma unroll 8
  for (int b = b0; b < b1; ++b) {
    int32_t* const at = table + static_cast<int64_t>(b) * E + e;
    const int v = *at;
    *at = run;
    run += v;
  }
  if (warp == kSortWarps - 1) table[static_cast<int64_t>(blocks) * E + e] = run;
}

// Places the entries of one block, from every block's counts.
__global__ void __launch_bounds__(kSortThreads) place_kernel(const SortParams p) {
  extern __shared__ __align__(16) uint16_t s_table[];
  __shared__ int s_total[kMaxExperts];
  __shared__ int s_base[kMaxExperts];
  __shared__ int s_warp[kSortWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_launch_dependents();
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.tokens;
  const int nt = static_cast<int>(min(static_cast<int64_t>(p.tokens), p.m - t0));
  const int n = nt * p.k;
  const int chunks = (n + 31) / 32;
  for (int i = tid; i < (chunks * p.E + 1) / 2; i += kSortThreads)
    reinterpret_cast<uint32_t*>(s_table)[i] = 0u;
  if (tid < p.E) s_total[tid] = s_base[tid] = 0;
  __syncthreads();
  griddep_wait();
  const int32_t* expert = p.expert + t0 * p.k;
  for (int c = warp; c < chunks; c += kSortWarps) {
    const int i = c * 32 + lane;
    const int e = i < n ? expert[i] : -1;
    const bool real = is_expert(e, p.E);
    int count;
    bool last;
    chunk_rank(e, real, lane, count, last);
    if (real && last) s_table[c * p.E + e] = static_cast<uint16_t>(count);
  }
  // Every block's counts, by as many threads per expert as there are (sums of
  // whole numbers: their order does not matter), where nobody has summed them.
  const int parts = kSortThreads / p.E;
  if (p.scanned) {
    if (tid < p.E) {
      s_base[tid] = p.table[static_cast<int64_t>(blockIdx.x) * p.E + tid];
      s_total[tid] = p.table[static_cast<int64_t>(p.blocks) * p.E + tid];
    }
  } else if (tid < parts * p.E) {
    const int e = tid % p.E;
    int before = 0, total = 0;
#pragma unroll 8
    for (int b = tid / p.E; b < p.blocks; b += parts) {
      const int v = p.table[static_cast<int64_t>(b) * p.E + e];
      if (b < static_cast<int>(blockIdx.x)) before += v;
      total += v;
    }
    atomicAdd(s_total + e, total);
    atomicAdd(s_base + e, before);
  }
  __syncthreads();
  if (tid < p.E) {
    int run = 0;
    for (int c = 0; c < chunks; ++c) {
      const int v = s_table[c * p.E + tid];
      s_table[c * p.E + tid] = static_cast<uint16_t>(run);
      run += v;
    }
  }
  const int kept = scan_experts(s_total, s_warp, p.E);
  if (tid < p.E) s_base[tid] += s_total[tid];
  if (blockIdx.x == 0) {
    if (tid < p.E) p.offsets[tid] = s_total[tid];
    if (tid == 0) p.offsets[p.E] = kept;
  }
  __syncthreads();
  for (int c = warp; c < chunks; c += kSortWarps) {
    const int i = c * 32 + lane;
    const int e = i < n ? expert[i] : -1;
    const bool real = is_expert(e, p.E);
    int count;
    bool last;
    const int rank = chunk_rank(e, real, lane, count, last);
    if (i < n) {
      const int at = real ? s_base[e] + s_table[c * p.E + e] + rank : -1;
      p.slot[t0 * p.k + i] = at;
      if (real) p.order[at] = static_cast<int32_t>(t0 * p.k + i);
    }
  }
  const int64_t all = p.m * p.k;
  for (int64_t i = kept + static_cast<int64_t>(blockIdx.x) * kSortThreads + tid; i < all;
       i += static_cast<int64_t>(gridDim.x) * kSortThreads)
    p.order[i] = -1;
}

// ------------------------------------------------------- gather, combine --

struct RowsParams {
  const void* a;  // gather: x; combine: ys; backward: dout
  int64_t lda;
  const void* b;  // backward: ys
  int64_t ldb;
  const int32_t* slot;
  const float* weight;
  void* out;  // gather: xs; combine: out; backward: dys
  int64_t ldo;
  float* dweight;
  int64_t m;
  int64_t D;
  int k;
};

constexpr int kRowThreads = 256;

__device__ __forceinline__ bool is_slot(int s, int64_t rows) { return s >= 0 && s < rows; }

// The slots and weights of eight entries of a token from j0 on (-1: no row).
// Kernels before this one on the stream may have made them, so they are read
// by ordinary loads, as everything but a handle's weights is.
struct Eight {
  int s[8];
  float w[8];
  __device__ __forceinline__ void slots(const RowsParams& p, int64_t t, int j0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = j0 + j < p.k ? p.slot[t * p.k + j0 + j] : -1;
  }
  __device__ __forceinline__ void weights(const RowsParams& p, int64_t t, int j0) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      w[j] = p.weight && j0 + j < p.k ? p.weight[t * p.k + j0 + j] : 1.f;
  }
};

// Rows are read and written V elements at a time, as wide as every row's
// alignment allows (16, 8 or 4 bytes, or single elements for an odd width);
// a thread has U of them under way, so that narrow accesses keep about as
// many bytes in flight as wide ones.  Rows on 16 bytes are bound by HBM (gather
// of 4096 x 8 rows of 8192 bf16: 92 us, 6.6 TB/s), others by the number of
// accesses (of 2000 x 6 rows of 5001: 32 us, 4.4 TB/s).  (Gradient of the
// combine, the same tensors: 174 us, 6.6 TB/s, and 67 us, 3.9 TB/s; 1000 tokens
// x 6 of 4100 fp16: 23 us, 4.6 TB/s, where the third trip of a row of 1025
// words has one thread at work.)
template <typename T, int V>
constexpr int kAhead = 16 / (V * static_cast<int>(sizeof(T))) < 8
                           ? 16 / (V * static_cast<int>(sizeof(T)))
                           : 8;

template <typename T, int V>
__global__ void __launch_bounds__(kRowThreads) gather_kernel(const RowsParams p) {
  constexpr int U = kAhead<T, V>;
  griddep_launch_dependents();
  griddep_wait();
  const int64_t t = blockIdx.x;
  const int64_t nvec = p.D / V, rows = p.m * p.k;
  const T* x = static_cast<const T*>(p.a) + t * p.lda;
  T* xs = static_cast<T*>(p.out);
  for (int64_t v0 = static_cast<int64_t>(blockIdx.y) * kRowThreads * U + threadIdx.x; v0 < nvec;
       v0 += static_cast<int64_t>(gridDim.y) * kRowThreads * U) {
    Vec<T, V> val[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (v0 + u * kRowThreads < nvec) val[u] = load_vec<T, V>(x + (v0 + u * kRowThreads) * V);
    for (int j0 = 0; j0 < p.k; j0 += 8) {
      Eight to;
      to.slots(p, t, j0);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (!is_slot(to.s[j], rows)) continue;
        T* at = xs + to.s[j] * p.ldo + v0 * V;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (v0 + u * kRowThreads < nvec)
            *reinterpret_cast<Vec<T, V>*>(at + u * kRowThreads * V) = val[u];
      }
    }
  }
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// The combine is bound by the loads of k rows per token from anywhere.  A CTA
// takes pieces (token, 4 KB of columns, eight entries) in turn and has the rows
// of the next kDeep - 1 on their way to shared memory: no registers are held by
// loads in flight, and the slots of a piece are read one piece before its copies
// start.  (4096 tokens x 8 rows of 8192 bf16: 119 us, 289 with the rows loaded
// to registers.)  Rows that start on 16 bytes, and end so (kUnit = 16): a
// thread reads back what it copied itself, without barriers.  Any others keep
// their misalignment in shared memory, where the 16-byte words that hold them
// go -- with elements of neighbouring rows, which nobody uses, at the ends --
// and threads read kUnit bytes, 4 or an element as the rows' alignment allows,
// side by side and behind a barrier.  Words that reach out of ys go element by
// element.  (2000 tokens x 6 rows of 5001 bf16: 68 us, 107 through registers.)
constexpr int kDeep = 3;
constexpr int kPieceBytes = kRowThreads * 16;
constexpr int kPlace = kPieceBytes + 32;  // of a row's piece in shared memory
constexpr int kDeepBytes = kDeep * 8 * kPlace;

template <typename T, int kUnit>
__global__ void __launch_bounds__(kRowThreads, 2)
    combine_kernel(const RowsParams p, const int columns, const int width) {
  constexpr int V = 16 / static_cast<int>(sizeof(T));
  constexpr int el = sizeof(T);
  constexpr bool kWhole = kUnit == 16;
  constexpr int UE = kUnit / el, NU = V / UE;  // elements of a unit, units of a thread
  extern __shared__ __align__(16) uint8_t s_rows[];  // [kDeep][8] of kPlace
  griddep_launch_dependents();
  griddep_wait();
  const int D = static_cast<int>(p.D), tid = threadIdx.x;
  const int64_t rows = p.m * p.k;
  const T* ys = static_cast<const T*>(p.a);
  const char* const begin = reinterpret_cast<const char*>(ys);
  const char* const end = reinterpret_cast<const char*>(ys + (rows - 1) * p.lda + p.D);
  const int jgroups = (p.k + 7) / 8;  // a token's entries, eight at a time, are the fastest
  const int64_t total = p.m * columns;

  struct At {
    int64_t t;
    int c0, j0;
  };
  auto where = [&](int64_t n) {  // this CTA's n-th piece
    const int64_t i = blockIdx.x + n / jgroups * gridDim.x;
    At at;
    at.t = i < total ? i / columns : -1;
    at.c0 = static_cast<int>(i % columns) * width;
    at.j0 = static_cast<int>(n % jgroups) * 8;
    return at;
  };
  auto start = [&](const At& at, const int (&s)[8], int stage) {
    if (at.t < 0) return;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (is_slot(s[j], rows)) {
        const T* from = ys + s[j] * p.lda + at.c0;
        uint8_t* const place = s_rows + (stage * 8 + j) * kPlace;
        if constexpr (kWhole) {
          if (tid * V < min(width, D - at.c0))
            cp_async16(smem_u32(place) + tid * 16, from + tid * V);
        } else {
          const char* const first = reinterpret_cast<const char*>(from);
          const int off = static_cast<int>(reinterpret_cast<uintptr_t>(first) & 15);
          const int bytes = min(width, D - at.c0) * el;
          const int words = (off + bytes + 15) / 16;
          for (int i = tid; i < words; i += kRowThreads) {
            const char* const w = first - off + 16 * i;
            if (w >= begin && w + 16 <= end) {
              cp_async16(smem_u32(place) + 16 * i, w);
            } else {
              for (int e = 0; e < 16; e += el)
                if (w + e >= first && w + e < first + bytes)
                  *reinterpret_cast<T*>(place + 16 * i + e) = *reinterpret_cast<const T*>(w + e);
            }
          }
        }
      }
  };

  Eight ahead, cur;
  for (int d = 0; d < kDeep - 1; ++d) {
    const At at = where(d);
    if (at.t >= 0) ahead.slots(p, at.t, at.j0);
    start(at, ahead.s, d);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  At next = where(kDeep - 1);
  if (next.t >= 0) ahead.slots(p, next.t, next.j0);
  At at = where(0);
  if (at.t >= 0) {
    cur.slots(p, at.t, at.j0);
    cur.weights(p, at.t, at.j0);
  }
  float acc[V] = {};
  int stage = 0;
  for (int64_t n = 0; at.t >= 0; ++n) {
    const int wide = min(width, D - at.c0);
    asm volatile("cp.async.wait_group %0;" ::"n"(kDeep - 2) : "memory");
    if (!kWhole) __syncthreads();  // the piece is there, and the one before has been read
    // start the piece kDeep - 1 ahead in the stage that the last one left
    start(next, ahead.s, stage == 0 ? kDeep - 1 : stage - 1);
    asm volatile("cp.async.commit_group;" ::: "memory");
    next = where(n + kDeep);
    if (next.t >= 0) ahead.slots(p, next.t, next.j0);
    const At after = where(n + 1);
    Eight then;
    if (after.t >= 0) {
      then.slots(p, after.t, after.j0);
      then.weights(p, after.t, after.j0);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (is_slot(cur.s[j], rows)) {
        const uint8_t* const place = s_rows + (stage * 8 + j) * kPlace;
        if constexpr (kWhole) {
          if (tid * V < wide) {
            float f[V];
            widen(*reinterpret_cast<const Vec<T, V>*>(place + tid * 16), f);
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = fmaf(cur.w[j], f[i], acc[i]);
          }
        } else {
          const T* const first = ys + cur.s[j] * p.lda + at.c0;
          const uint8_t* const e = place + (reinterpret_cast<uintptr_t>(first) & 15);
#pragma unroll
          for (int i = 0; i < NU; ++i) {
            const int u = i * kRowThreads + tid;
            if (u * UE < wide) {
              float f[UE];
              widen(*reinterpret_cast<const Vec<T, UE>*>(e + u * kUnit), f);
#pragma unroll
              for (int l = 0; l < UE; ++l)
                acc[i * UE + l] = fmaf(cur.w[j], f[l], acc[i * UE + l]);
            }
          }
        }
      }
    if (at.j0 + 8 >= p.k) {
      T* out = static_cast<T*>(p.out) + at.t * p.ldo + at.c0;
      if constexpr (kWhole) {
        if (tid * V < wide) store_vec<T, V>(out + tid * V, acc);
      } else {
#pragma unroll
        for (int i = 0; i < NU; ++i) {
          const int u = i * kRowThreads + tid;
          if (u * UE < wide) {
            float f[UE];
#pragma unroll
            for (int l = 0; l < UE; ++l) f[l] = acc[i * UE + l];
            store_vec<T, UE>(out + u * UE, f);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = 0.f;
    }
    at = after;
    cur = then;
    if (++stage == kDeep) stage = 0;
  }
}

// One token per CTA: the k dot products run over the whole row, KJ entries at
// a time.
template <typename T, int V>
__global__ void __launch_bounds__(kRowThreads) combine_grad_kernel(const RowsParams p) {
  constexpr int U = kAhead<T, V>, KJ = 8;
  __shared__ float room[2 * KJ * 32];
  int turn = 0;
  griddep_launch_dependents();
  griddep_wait();
  const int64_t t = blockIdx.x;
  const int64_t nvec = p.D / V, rows = p.m * p.k;
  const T* dout = static_cast<const T*>(p.a) + t * p.lda;
  const T* ys = static_cast<const T*>(p.b);
  const int32_t* slot = p.slot + t * p.k;
  T* dys = static_cast<T*>(p.out);
  for (int j0 = 0; j0 < p.k; j0 += KJ) {
    int s[KJ];
    float w[KJ], dot[KJ];
#pragma unroll
    for (int j = 0; j < KJ; ++j) {
      s[j] = j0 + j < p.k ? slot[j0 + j] : -1;
      if (!is_slot(s[j], rows)) s[j] = -1;
      w[j] = s[j] >= 0 && p.out ? (p.weight ? p.weight[t * p.k + j0 + j] : 1.f) : 0.f;
      dot[j] = 0.f;
    }
    for (int64_t v0 = threadIdx.x; v0 < nvec; v0 += kRowThreads * U) {
      Vec<T, V> dv[U], val[KJ][U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (v0 + u * kRowThreads < nvec) dv[u] = load_vec<T, V>(dout + (v0 + u * kRowThreads) * V);
      if (p.dweight) {
#pragma unroll
        for (int j = 0; j < KJ; ++j)
          if (s[j] >= 0) {
            const T* from = ys + s[j] * p.ldb + v0 * V;
#pragma unroll
            for (int u = 0; u < U; ++u)
              if (v0 + u * kRowThreads < nvec)
                val[j][u] = load_vec<T, V>(from + u * kRowThreads * V);
          }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (v0 + u * kRowThreads >= nvec) continue;
        float d[V];
        widen(dv[u], d);
#pragma unroll
        for (int j = 0; j < KJ; ++j)
          if (s[j] >= 0) {
            if (p.dweight) {
              float f[V];
              widen(val[j][u], f);
#pragma unroll
              for (int i = 0; i < V; ++i) dot[j] = fmaf(d[i], f[i], dot[j]);
            }
            if (p.out) {
              float o[V];
#pragma unroll
              for (int i = 0; i < V; ++i) o[i] = w[j] * d[i];
              store_vec<T, V>(dys + s[j] * p.ldo + (v0 + u * kRowThreads) * V, o);
            }
          }
      }
    }
    if (p.dweight) {
      row_sums<kRowThreads, KJ>(dot, room, turn);
#pragma unroll
      for (int j = 0; j < KJ; ++j)
        if (threadIdx.x == j && j0 + j < p.k) p.dweight[t * p.k + j0 + j] = dot[j];
    }
  }
}

// ------------------------------------------------------- route, backward --

struct RouteGradParams {
  const float* logits;
  int64_t ldl;
  const int32_t* expert;
  const float* weight;
  const float* dweight;
  float* dlogits;
  int64_t lddl;
  int64_t m;
  int E, k, mode;
};

constexpr int kGradWarps = 8;

// One warp per token.  Lane j holds choice j; the choices are handed to the
// lane that holds their expert by a pass over the k of them.
template <int EPL>
__global__ void __launch_bounds__(32 * kGradWarps) route_grad_kernel(const RouteGradParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kGradWarps + (threadIdx.x >> 5);
  if (t >= p.m) return;
  int e = -1;
  float w = 0.f, dw = 0.f;
  if (lane < p.k) {
    e = p.expert[t * p.k + lane];
    if (is_expert(e, p.E)) {
      w = p.weight[t * p.k + lane];
      dw = p.dweight[t * p.k + lane];
    } else {
      e = -1;
    }
  }
  const float inner = warp_sum(w * dw);
  float g[EPL];
  if (p.mode == PROJ_ROUTE_ALL) {
    uint32_t key[EPL], top = 0u;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int x = i * 32 + lane;
      key[i] = x < p.E ? order_key(p.logits[t * p.ldl + x]) : 0u;
      top = max(top, key[i]);
    }
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    const float tv = key_value(top);
    float all = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      g[i] = key[i] ? exp_below(key_value(key[i]), tv) : 0.f;
      all += g[i];
    }
    all = warp_sum(all);
    const float scale = all > 0.f ? 1.f / all : 0.f;
    float take[EPL] = {};
    for (int j = 0; j < p.k; ++j) {
      const int ej = __shfl_sync(0xFFFFFFFFu, e, j);
      const float dj = __shfl_sync(0xFFFFFFFFu, dw, j);
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (ej == i * 32 + lane) take[i] += dj;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) g[i] = g[i] * scale * (take[i] - inner);
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) g[i] = 0.f;
    const float own = w * (dw - inner);
    for (int j = 0; j < p.k; ++j) {
      const int ej = __shfl_sync(0xFFFFFFFFu, e, j);
      const float oj = __shfl_sync(0xFFFFFFFFu, own, j);
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (ej == i * 32 + lane) g[i] += oj;
    }
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int x = i * 32 + lane;
    if (x < p.E) p.dlogits[t * p.lddl + x] = g[i];
  }
}

// --------------------------------------------------------------- launches --

cudaLaunchConfig_t config(int64_t grid_x, int64_t grid_y, unsigned threads, size_t smem,
                          cudaStream_t s, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid_x), static_cast<unsigned>(grid_y));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// Tokens per block of the sort: one block, and with it one launch, up to 64
// tokens (two a warp); more tokens are spread over as many blocks as there are
// SMs, a warp choosing for at least one token each, as far as the chunk table
// fits shared memory.
int sort_tokens(int64_t m, int E, int k) {
  const int64_t tokens = m <= 64 ? 64 : std::max<int64_t>(kSortWarps, (m + 151) / 152);
  // chunk table in shared memory, counts in 16 bits
  const int64_t most = std::min<int64_t>(kTableBytes / (2 * E) * 32, 32768) / k;
  return static_cast<int>(std::max<int64_t>(1, std::min(tokens, most)));
}
int64_t sort_blocks(int64_t m, int E, int k) {
  const int tokens = sort_tokens(m, E, k);
  return (m + tokens - 1) / tokens;
}
// Blocks beyond which their counts are summed by a launch of its own.  (Sort of
// 8 of 256 experts, every block for itself and by one launch: 196 blocks 52.0
// and 52.8 us, 261 blocks 54.0 and 51.4, 1366 blocks 363 and 212; 8 of 1024,
// 2^20 tokens in 5462 blocks: 12,036 and 397.)
constexpr int64_t kScanBlocks = 256;
// Rows of the table in the workspace.
int64_t table_rows(int64_t blocks) { return blocks > kScanBlocks ? blocks + 1 : blocks; }
size_t sort_smem(int tokens, int E, int k) {
  const int chunks = (tokens * k + 31) / 32;
  return (static_cast<size_t>(chunks) * E * 2 + 15) & ~static_cast<size_t>(15);
}

template <int EPL>
cudaError_t choose_count(const SortParams& p, size_t smem, cudaStream_t s) {
  if (smem > 48 * 1024) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(choose_count_kernel<EPL>),
                                     kTableBytes + 16, done);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = config(p.blocks, 1, kSortThreads, smem, s, attr);
  return cudaLaunchKernelEx(&cfg, choose_count_kernel<EPL>, p);
}

cudaError_t sort_launch(const SortParams& p, cudaStream_t s) {
  const size_t smem = p.offsets ? sort_smem(p.tokens, p.E, p.k) : 0;
  cudaError_t e;
  if (!p.logits || p.E <= 64)
    e = choose_count<2>(p, smem, s);
  else if (p.E <= 256)
    e = choose_count<8>(p, smem, s);
  else
    e = choose_count<32>(p, smem, s);
  if (e != cudaSuccess || !p.offsets || p.blocks <= 1) return e;
  if (smem > 48 * 1024) {
    static std::atomic<uint64_t> done{0};
    e = allow_smem(reinterpret_cast<const void*>(place_kernel), kTableBytes + 16, done);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr[1];
  if (p.scanned) {
    const cudaLaunchConfig_t cfg = config((p.E + 31) / 32, 1, kSortThreads, 0, s, attr);
    e = cudaLaunchKernelEx(&cfg, scan_blocks_kernel, p.table, p.blocks, p.E);
    if (e != cudaSuccess) return e;
  }
  const cudaLaunchConfig_t cfg = config(p.blocks, 1, kSortThreads, smem, s, attr);
  return cudaLaunchKernelEx(&cfg, place_kernel, p);
}

int refuse(int status, const char* call, const char* why) {
  char text[160];
  std::snprintf(text, sizeof text, "%s: %s", call, why);
  return record_status(status, text);
}

bool aligned_to(const void* p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Sizes that every call shares; nullptr if they are fine.
const char* refuse_sizes(int64_t m, int64_t E, int64_t k, int* status) {
  *status = PROJ_EINVAL;
  if (m < 0 || E < 1 || k < 1 || k > E) return "m < 0, E < 1, or k outside 1 .. E";
  *status = PROJ_EUNSUPPORTED;
  if (E > kMaxExperts) return "more than 1024 experts";
  if (k > kMaxK) return "k > 32";
  if (m >= (int64_t{1} << 31) / k) return "m * k >= 2^31";
  *status = PROJ_OK;
  return nullptr;
}

int sort_call(const char* call, SortParams p, void* workspace, int64_t workspace_bytes,
              cudaStream_t s) {
  if (p.m == 0) {
    if (!p.offsets) return PROJ_OK;
    const cudaError_t e = cudaMemsetAsync(p.offsets, 0, sizeof(int32_t) * (p.E + 1), s);
    return e == cudaSuccess ? PROJ_OK : record_cuda(e, call);
  }
  p.tokens = sort_tokens(p.m, p.E, p.k);
  p.blocks = static_cast<int>(sort_blocks(p.m, p.E, p.k));
  if (p.offsets && p.blocks > 1) {
    const int64_t want = table_rows(p.blocks) * p.E * 4;
    if (!workspace || workspace_bytes < want)
      return refuse(PROJ_EINVAL, call, "workspace is NULL or too small");
    if (!aligned_to(workspace, 16))
      return refuse(PROJ_EALIGN, call, "workspace is not 16-byte aligned");
    p.table = static_cast<int32_t*>(workspace);
    p.scanned = p.blocks > kScanBlocks;
  }
  const cudaError_t e = sort_launch(p, s);
  return e == cudaSuccess ? PROJ_OK : record_cuda(e, call);
}

// Common to gather and combine; nullptr if fine.
const char* refuse_rows(const RowsParams& p, int64_t k, int dtype, int* status) {
  *status = PROJ_EINVAL;
  if (p.m < 0 || p.D < 1 || k < 1) return "m < 0, D < 1 or k < 1";
  if (dtype != PROJ_BF16 && dtype != PROJ_FP16 && dtype != PROJ_FP32) return "unknown dtype";
  if (p.m > 0 && (!p.a || !p.slot)) return "a NULL pointer";
  if (p.lda < p.D || (p.b && p.ldb < p.D) || (p.out && p.ldo < p.D)) return "a row stride is below D";
  *status = PROJ_EUNSUPPORTED;
  if (k > kMaxK) return "k > 32";
  if (p.m >= (int64_t{1} << 31) / k) return "m * k >= 2^31";
  if (p.D > (int64_t{1} << 30)) return "D > 2^30";
  const int el = dtype == PROJ_FP32 ? 4 : 2;
  *status = PROJ_EALIGN;
  if (!aligned_to(p.a, el) || !aligned_to(p.b, el) || !aligned_to(p.out, el) ||
      !aligned_to(p.slot, 4) || !aligned_to(p.weight, 4) || !aligned_to(p.dweight, 4))
    return "a pointer is not aligned to an element";
  *status = PROJ_OK;
  return nullptr;
}

enum class Op { kGather, kCombine, kGrad };

template <typename T, int V>
cudaError_t rows_launch(Op op, const RowsParams& p, cudaStream_t s) {
  const int64_t nvec = p.D / V;
  const int64_t per = kRowThreads * kAhead<T, V>;
  const int64_t ny = op == Op::kGrad ? 1 : std::min<int64_t>(64, (nvec + per - 1) / per);
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = config(p.m, ny, kRowThreads, 0, s, attr);
  return op == Op::kGather ? cudaLaunchKernelEx(&cfg, gather_kernel<T, V>, p)
                           : cudaLaunchKernelEx(&cfg, combine_grad_kernel<T, V>, p);
}

template <typename T, int kUnit>
cudaError_t combine_launch(const RowsParams& p, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e =
      allow_smem(reinterpret_cast<const void*>(combine_kernel<T, kUnit>), kDeepBytes, done);
  if (e != cudaSuccess) return e;
  constexpr int kCols = kPieceBytes / static_cast<int>(sizeof(T));
  // pieces of about equal width, in 16 bytes
  const int64_t columns = (p.D + kCols - 1) / kCols;
  constexpr int kStep = 16 / static_cast<int>(sizeof(T));
  const int64_t width = ((p.D + columns - 1) / columns + kStep - 1) / kStep * kStep;
  const int64_t grid = std::min<int64_t>(p.m * columns, 2 * std::max(1, proj_num_sms()));
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = config(grid, 1, kRowThreads, kDeepBytes, s, attr);
  return cudaLaunchKernelEx(&cfg, combine_kernel<T, kUnit>, p, static_cast<int>(columns),
                            static_cast<int>(width));
}

// Whether every row of every tensor starts on a multiple of `bytes`, and so
// does its end.
bool rows_on(const RowsParams& p, int el, int bytes) {
  auto fits = [&](const void* q, int64_t ld) {
    return !q || (aligned_to(q, bytes) && (ld * el) % bytes == 0);
  };
  return (p.D * el) % bytes == 0 && fits(p.a, p.lda) && fits(p.b, p.ldb) && fits(p.out, p.ldo);
}

template <typename T>
cudaError_t rows_any(Op op, const RowsParams& p, cudaStream_t s) {
  constexpr int el = sizeof(T);
  if (op == Op::kCombine)
    return rows_on(p, el, 16)  ? combine_launch<T, 16>(p, s)
           : rows_on(p, el, 4) ? combine_launch<T, 4>(p, s)
                               : combine_launch<T, el>(p, s);
  if (rows_on(p, el, 16)) return rows_launch<T, 16 / el>(op, p, s);
  if (rows_on(p, el, 8)) return rows_launch<T, 8 / el>(op, p, s);
  if constexpr (el == 2)
    if (rows_on(p, el, 4)) return rows_launch<T, 2>(op, p, s);
  return rows_launch<T, 1>(op, p, s);
}

int rows_call(const char* call, Op op, const RowsParams& p, int dtype, proj_stream stream) {
  if (p.m == 0) return PROJ_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == PROJ_BF16   ? rows_any<__nv_bfloat16>(op, p, s)
                        : dtype == PROJ_FP16 ? rows_any<__half>(op, p, s)
                                             : rows_any<float>(op, p, s);
  return e == cudaSuccess ? PROJ_OK : record_cuda(e, call);
}

}  // namespace
}  // namespace proj

using namespace proj;

extern "C" int64_t proj_moe_workspace(int64_t m, int64_t experts, int64_t k) {
  int status = PROJ_OK;
  if (const char* why = refuse_sizes(m, experts, k, &status)) {
    refuse(status, "proj_moe_workspace", why);
    return -1;
  }
  const int64_t blocks = sort_blocks(m, static_cast<int>(experts), static_cast<int>(k));
  return blocks > 1 ? table_rows(blocks) * experts * 4 : 0;
}

extern "C" int proj_moe_route(const float* logits, int64_t ldl, int64_t m, int64_t experts,
                              int64_t k, int mode, int32_t* expert, float* weight,
                              int32_t* offsets, int32_t* order, int32_t* slot, void* workspace,
                              int64_t workspace_bytes, proj_stream stream) {
  const char* const call = "proj_moe_route";
  int status = PROJ_OK;
  if (const char* why = refuse_sizes(m, experts, k, &status)) return refuse(status, call, why);
  if (mode != PROJ_ROUTE_CHOSEN && mode != PROJ_ROUTE_ALL)
    return refuse(PROJ_EINVAL, call, "unknown mode");
  if (m > 0 && (!logits || !expert || !weight))
    return refuse(PROJ_EINVAL, call, "logits, expert or weight is NULL");
  if (ldl < experts) return refuse(PROJ_EINVAL, call, "ldl is below the number of experts");
  if ((offsets != nullptr) != (order != nullptr) || (offsets != nullptr) != (slot != nullptr))
    return refuse(PROJ_EINVAL, call, "offsets, order and slot are not all given or all NULL");
  if (!aligned_to(logits, 4) || !aligned_to(expert, 4) || !aligned_to(weight, 4) ||
      !aligned_to(offsets, 4) || !aligned_to(order, 4) || !aligned_to(slot, 4))
    return refuse(PROJ_EALIGN, call, "a pointer is not aligned to 4 bytes");
  SortParams p = {};
  p.logits = logits;
  p.ldl = ldl;
  p.expert = expert;
  p.weight = weight;
  p.offsets = offsets;
  p.order = order;
  p.slot = slot;
  p.m = m;
  p.E = static_cast<int>(experts);
  p.k = static_cast<int>(k);
  p.mode = mode;
  return sort_call(call, p, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int proj_moe_sort(const int32_t* expert, int64_t m, int64_t experts, int64_t k,
                             int32_t* offsets, int32_t* order, int32_t* slot, void* workspace,
                             int64_t workspace_bytes, proj_stream stream) {
  const char* const call = "proj_moe_sort";
  int status = PROJ_OK;
  if (const char* why = refuse_sizes(m, experts, k, &status)) return refuse(status, call, why);
  if (!offsets || (m > 0 && (!expert || !order || !slot)))
    return refuse(PROJ_EINVAL, call, "a NULL pointer");
  if (!aligned_to(expert, 4) || !aligned_to(offsets, 4) || !aligned_to(order, 4) ||
      !aligned_to(slot, 4))
    return refuse(PROJ_EALIGN, call, "a pointer is not aligned to 4 bytes");
  SortParams p = {};
  p.expert = const_cast<int32_t*>(expert);  // read only: there are no logits
  p.offsets = offsets;
  p.order = order;
  p.slot = slot;
  p.m = m;
  p.E = static_cast<int>(experts);
  p.k = static_cast<int>(k);
  return sort_call(call, p, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int proj_moe_gather(const void* x, int64_t ldx, const int32_t* slot, int64_t m,
                               int64_t D, int64_t k, int dtype, void* xs, int64_t ldxs,
                               proj_stream stream) {
  RowsParams p = {};
  p.a = x;
  p.lda = ldx;
  p.slot = slot;
  p.out = xs;
  p.ldo = ldxs;
  p.m = m;
  p.D = D;
  p.k = static_cast<int>(k);
  int status = PROJ_OK;
  if (const char* why = refuse_rows(p, k, dtype, &status))
    return refuse(status, "proj_moe_gather", why);
  if (m > 0 && !xs) return refuse(PROJ_EINVAL, "proj_moe_gather", "xs is NULL");
  return rows_call("proj_moe_gather", Op::kGather, p, dtype, stream);
}

extern "C" int proj_moe_combine(const void* ys, int64_t ldys, const int32_t* slot,
                                const float* weight, int64_t m, int64_t D, int64_t k, int dtype,
                                void* out, int64_t ldo, proj_stream stream) {
  RowsParams p = {};
  p.a = ys;
  p.lda = ldys;
  p.slot = slot;
  p.weight = weight;
  p.out = out;
  p.ldo = ldo;
  p.m = m;
  p.D = D;
  p.k = static_cast<int>(k);
  int status = PROJ_OK;
  if (const char* why = refuse_rows(p, k, dtype, &status))
    return refuse(status, "proj_moe_combine", why);
  if (m > 0 && !out) return refuse(PROJ_EINVAL, "proj_moe_combine", "out is NULL");
  return rows_call("proj_moe_combine", Op::kCombine, p, dtype, stream);
}

extern "C" int proj_moe_combine_backward(const void* dout, int64_t lddo, const void* ys,
                                         int64_t ldys, const int32_t* slot, const float* weight,
                                         int64_t m, int64_t D, int64_t k, int dtype, void* dys,
                                         int64_t lddys, float* dweight, proj_stream stream) {
  const char* const call = "proj_moe_combine_backward";
  RowsParams p = {};
  p.a = dout;
  p.lda = lddo;
  p.b = dweight ? ys : nullptr;
  p.ldb = ldys;
  p.slot = slot;
  p.weight = weight;
  p.out = dys;
  p.ldo = lddys;
  p.dweight = dweight;
  p.m = m;
  p.D = D;
  p.k = static_cast<int>(k);
  int status = PROJ_OK;
  if (const char* why = refuse_rows(p, k, dtype, &status)) return refuse(status, call, why);
  if (m > 0 && !dys && !dweight) return refuse(PROJ_EINVAL, call, "dys and dweight are both NULL");
  if (m > 0 && dweight && !ys) return refuse(PROJ_EINVAL, call, "dweight is wanted, but ys is NULL");
  return rows_call(call, Op::kGrad, p, dtype, stream);
}

extern "C" int proj_moe_route_backward(const float* logits, int64_t ldl, int64_t m,
                                       int64_t experts, int64_t k, int mode,
                                       const int32_t* expert, const float* weight,
                                       const float* dweight, float* dlogits, int64_t lddl,
                                       proj_stream stream) {
  const char* const call = "proj_moe_route_backward";
  int status = PROJ_OK;
  if (const char* why = refuse_sizes(m, experts, k, &status)) return refuse(status, call, why);
  if (mode != PROJ_ROUTE_CHOSEN && mode != PROJ_ROUTE_ALL)
    return refuse(PROJ_EINVAL, call, "unknown mode");
  if (m > 0 && (!expert || !weight || !dweight || !dlogits || (mode == PROJ_ROUTE_ALL && !logits)))
    return refuse(PROJ_EINVAL, call, "a NULL pointer");
  if ((mode == PROJ_ROUTE_ALL && ldl < experts) || lddl < experts)
    return refuse(PROJ_EINVAL, call, "a row stride is below the number of experts");
  if (!aligned_to(logits, 4) || !aligned_to(expert, 4) || !aligned_to(weight, 4) ||
      !aligned_to(dweight, 4) || !aligned_to(dlogits, 4))
    return refuse(PROJ_EALIGN, call, "a pointer is not aligned to 4 bytes");
  if (m == 0) return PROJ_OK;
  RouteGradParams p = {logits, ldl, expert, weight, dweight, dlogits, lddl, m,
                       static_cast<int>(experts), static_cast<int>(k), mode};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg =
      config((m + kGradWarps - 1) / kGradWarps, 1, 32 * kGradWarps, 0, s, attr);
  const cudaError_t e = experts <= 64    ? cudaLaunchKernelEx(&cfg, route_grad_kernel<2>, p)
                        : experts <= 256 ? cudaLaunchKernelEx(&cfg, route_grad_kernel<8>, p)
                                         : cudaLaunchKernelEx(&cfg, route_grad_kernel<32>, p);
  return e == cudaSuccess ? PROJ_OK : record_cuda(e, call);
}
