// attn.h -- attention of drafted tokens over the cache: what its kernels share
// (attn.cu: calls, streaming kernel, join; attn_tc.cu: tcgen05 kernel).
//
// Work is cut on the device, by the lengths that the call has: an item is a
// sequence, a head of keys and values, and `tile_rows` of its rows (a row is a
// drafted token and a query head of the group; row r is token r / group, head
// r % group); it has ceil(keys / unit) units.  The items' units stand in one line
// of W, and CTA c takes `each` of them from c `each` on: as many as spread the line
// over all CTAs, but 2^min_shift at least, unless there are items for more CTAs.  So
// every SM has the same share whatever the lengths, a CTA leaves at most two items
// unfinished (one it did not begin, one it does not end), and the partial results
// need room for two items a CTA and nothing that grows with the batch.  A second
// kernel joins them in the order of their CTAs.  (In batches of many items the
// streaming kernel gives shares to warps: "CTA" is a warp then.)
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv.h"
#include "ptx.cuh"
#include "vec.cuh"

namespace proj {

struct AttnParams {
  KvCache c;
  const uint8_t* q;
  int64_t ldq;  // bytes, as ldg and ldo
  const int32_t* offsets;
  const int32_t* start;
  const uint32_t* mask;
  int64_t ldm;
  int words;
  float scale_log2;  // scale * log2(e)
  const uint8_t* gate;
  int64_t ldg;
  int sigmoid;
  uint8_t* out;
  int64_t ldo;
  float* lse;
  int m, heads, D;
  Divisor group;
  int tile_rows, unit, ctas, spread, solo;
  int tile_shift, unit_shift, min_shift;  // logarithms; min_shift: of a share's least units
  struct Split* splits;  // [ctas]
  float* part_o;   // [2 ctas][tile_rows][D]: sums relative to 2^m
  float* part_ml;  // [2 ctas][tile_rows][2]: m, sum
  uint32_t* status;
};

// A sequence's part in the call.
struct Sequence {
  int lo, rows;     // first row of the call, drafted tokens
  int start, len;   // positions before the drafts, positions in all
  int tiles, units;
};

__device__ __forceinline__ Sequence sequence_at(const AttnParams& p, int b) {
  Sequence s;
  int hi;
  rows_of(p.offsets, b, p.m, s.lo, hi);
  s.rows = hi - s.lo;
  s.start = min(max(p.start[b], 0), p.c.capacity);
  s.len = min(s.start + s.rows, p.c.capacity);
  const int64_t rows = static_cast<int64_t>(s.rows) * static_cast<int>(p.group.d);
  s.tiles = static_cast<int>((rows + p.tile_rows - 1) >> p.tile_shift);
  // an item without keys has one unit all the same: its rows are written
  s.units = max(1, (s.len + p.unit - 1) >> p.unit_shift);
  return s;
}

// Units of a sequence; no more than 2^46 (years of work) are counted, so that sums
// and products below stay within 64 bits whatever stands in offsets and start.
__device__ __forceinline__ int64_t units_of(const AttnParams& p, const Sequence& s) {
  const int64_t all = static_cast<int64_t>(s.tiles) * s.units;
  return min(all < (int64_t{1} << 45) ? all * p.c.heads : all, int64_t{1} << 46);
}

// What a CTA leaves to be joined: the item in which its share begins, if that
// began before and this is its second CTA (rows 0: nothing).  The list stands at the
// workspace's start, which is aligned to 16 bytes and no more.
struct alignas(16) Split {
  int rows, lo, row0, head, first, last;  // first, last: the item's CTAs
  int pad[2];
};
static_assert(sizeof(Split) == 32 && alignof(Split) == 16, "an entry of the workspace");

// This CTA's share.
struct Share {
  int64_t each, first, end;  // units of a CTA, and this one's range
  int b;           // the sequence that holds `first`
  int64_t before;  // units of the sequences before b
};

// a / b of numbers that are not negative: mostly both have 32 bits, and the long
// division stands out of the way.
static __device__ __noinline__ int64_t divide_long(int64_t a, int64_t b) { return a / b; }
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  if (__builtin_expect(((a | b) >> 32) == 0, 1)) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return divide_long(a, b);
}

// The same where the quotient is often 0.
__device__ __forceinline__ int64_t item_of(int64_t a, int64_t b) { return a < b ? 0 : divide(a, b); }

// Reads the parameters of a launch: before the dependency wait, so that what they
// cost to come to the SM's constant cache passes beside the kernel before.
__device__ __forceinline__ void touch(const AttnParams& p) {
  asm volatile("" ::"l"(p.c.k), "l"(p.c.table), "r"(p.c.page.mul), "l"(p.q), "l"(p.start), "r"(p.words),
               "l"(p.out), "r"(p.m), "r"(p.ctas), "l"(p.splits), "l"(p.part_ml));
}
// The share's ends, once the units and items of all sequences are known.
__device__ __forceinline__ bool share_ends(const AttnParams& p, int cta, int64_t W, int items, Share& s) {
  const int64_t ctas = min(static_cast<int64_t>(p.ctas), max(W >> p.min_shift, static_cast<int64_t>(items)));
  if (W == 0) return false;
  s.each = divide(W + ctas - 1, ctas);
  s.first = s.each * cta;
  s.end = min(W, s.first + s.each);
  return s.first < W;
}
// Items are counted up to what CTAs there can be.
__device__ __forceinline__ int add_items(const AttnParams& p, int items, const Sequence& seq) {
  return static_cast<int>(min(items + static_cast<int64_t>(seq.tiles) * p.c.heads, int64_t{1} << 16));
}

// Few sequences: every warp finds the share by itself, without a barrier.
constexpr int kWarpSequences = 64;
__device__ __forceinline__ bool find_share_warp(const AttnParams& p, int cta, Share& s) {
  const int lane = threadIdx.x & 31, n = p.c.sequences;
  int64_t u[kWarpSequences / 32], sum = 0;
  int items = 0;
#pragma unroll
  for (int i = 0; i < kWarpSequences / 32; ++i) {
    const int b = lane * (kWarpSequences / 32) + i;
    u[i] = 0;
    if (b < n) {
      const Sequence seq = sequence_at(p, b);
      u[i] = units_of(p, seq);
      items = add_items(p, items, seq);
    }
    sum += u[i];
  }
  int64_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += v;
  }
  items = __reduce_add_sync(0xFFFFFFFFu, items);
  if (!share_ends(p, cta, __shfl_sync(0xFFFFFFFFu, inc, 31), items, s)) return false;
  int64_t before = inc - sum;
  const uint32_t here = __ballot_sync(0xFFFFFFFFu, s.first >= before && s.first < inc);
  int b = lane * (kWarpSequences / 32);
#pragma unroll
  for (int i = 0; i < kWarpSequences / 32 - 1; ++i)
    if (s.first >= before + u[i]) {
      before += u[i];
      ++b;
    }
  const int from = __ffs(here) - 1;
  s.b = __shfl_sync(0xFFFFFFFFu, b, from & 31);
  s.before = __shfl_sync(0xFFFFFFFFu, before, from & 31);
  return here != 0;
}

// The same for one warp and any number of sequences: a run of them a lane.
__device__ __forceinline__ bool find_share_walk(const AttnParams& p, int cta, Share& s) {
  if (p.c.sequences <= kWarpSequences) return find_share_warp(p, cta, s);
  const int lane = threadIdx.x & 31;
  const int per = (p.c.sequences + 31) / 32;
  const int b0 = min(lane * per, p.c.sequences), b1 = min(b0 + per, p.c.sequences);
  int64_t sum = 0;
  int items = 0;
  for (int b = b0; b < b1; ++b) {
    const Sequence seq = sequence_at(p, b);
    sum += units_of(p, seq);
    items = add_items(p, items, seq);
  }
  int64_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += v;
  }
  items = __reduce_add_sync(0xFFFFFFFFu, min(items, 1 << 16));
  if (!share_ends(p, cta, __shfl_sync(0xFFFFFFFFu, inc, 31), items, s)) return false;
  int64_t before = inc - sum;
  const bool here = s.first >= before && s.first < inc;
  int b = b0;
  if (here) {
    for (; b < b1 - 1; ++b) {
      const int64_t u = units_of(p, sequence_at(p, b));
      if (s.first < before + u) break;
      before += u;
    }
  }
  const uint32_t who = __ballot_sync(0xFFFFFFFFu, here);
  s.b = __shfl_sync(0xFFFFFFFFu, b, (__ffs(who) - 1) & 31);
  s.before = __shfl_sync(0xFFFFFFFFu, before, (__ffs(who) - 1) & 31);
  return who != 0;
}

// All threads of the CTA; kThreads of them.  `cta`: whose share (kSolo: the first
// warp's; each has its own).  False: none.
template <int kThreads, bool kSolo>
__device__ __forceinline__ bool find_share(const AttnParams& p, int cta, Share& s) {
  constexpr int kShares = kSolo ? kThreads / 32 : 1;
  const int mine = kSolo ? threadIdx.x >> 5 : 0;
  if (p.c.sequences <= kWarpSequences) return find_share_warp(p, cta + mine, s);
  __shared__ int64_t warp_sum[kThreads / 32];
  __shared__ int warp_items[kThreads / 32];
  __shared__ int found_b[kShares];
  __shared__ int64_t found_before[kShares];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.c.sequences + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, p.c.sequences), b1 = min(b0 + per, p.c.sequences);
  int64_t sum = 0;
  int items = 0;
  for (int b = b0; b < b1; ++b) {
    const Sequence seq = sequence_at(p, b);
    sum += units_of(p, seq);
    items = add_items(p, items, seq);
  }
  int64_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += v;
  }
  items = __reduce_add_sync(0xFFFFFFFFu, items);
  if (lane == 31) {
    warp_sum[warp] = inc;
    warp_items[warp] = items;
  }
  if (tid < kShares) found_b[tid] = -1;
  __syncthreads();
  int64_t before = inc - sum, W = 0;
  items = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    W += warp_sum[w];
    items += warp_items[w];
  }
  if (W == 0) return false;
  const bool some = share_ends(p, cta + mine, W, items, s);
  const int64_t end = before + sum;
  int64_t at = s.each * cta;
  int i = 0;
  for (; i < kShares && at < before; ++i) at += s.each;
  // the shares that begin in this thread's sequences
  for (int b = b0; i < kShares && at < end;) {
    const int64_t u = units_of(p, sequence_at(p, b));
    for (; i < kShares && at < before + u; ++i) {
      found_b[i] = b;
      found_before[i] = before;
      at += s.each;
    }
    before += u;
    ++b;
  }
  __syncthreads();
  s.b = found_b[mine];
  s.before = found_before[mine];
  return some && s.b >= 0;
}

__device__ __forceinline__ Split split_of(const AttnParams& p, const Share& s, int cta) {
  Split r = {};
  const Sequence seq = sequence_at(p, s.b);
  const int64_t item = item_of(s.first - s.before, seq.units);
  const int64_t begin = s.before + item * seq.units;
  if (begin == s.first) return r;
  r.first = static_cast<int>(divide(begin, s.each));
  if (cta != r.first + 1) return r;
  r.last = static_cast<int>(divide(begin + seq.units - 1, s.each));
  r.lo = seq.lo;
  r.head = static_cast<int>(item_of(item, seq.tiles));
  r.row0 = static_cast<int>(item - static_cast<int64_t>(r.head) * seq.tiles) * p.tile_rows;
  r.rows = min(p.tile_rows, seq.rows * static_cast<int>(p.group.d) - r.row0);
  return r;
}

// exp2 by the special-function unit: relative error 2^-22; -inf gives 0.
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// A row's reference moves when a score is more than 2^kSlack above it, and is
// 2^kLift as a probability: at most 2^14, twice that with V's scale, and 2^-28 of
// the reference is where fp16 ends (65504 and 2^-24).
constexpr float kSlack = 10.f, kLift = 4.f;

// V's scales come relative to a reference that all rows of an item share, a power
// of two near the largest one met, and p times that is rounded to fp16.  Before the
// drafts every row sees every key, and what is lost is 2^-29 of the largest value
// seen, for each key.  A draft's scale is met by rows that do not see it too.  So
// where keys are masked, a raise of the shared reference lowers the rows' own (what
// is summed of V stays as it is, p grows), while a row's sum stays below 2^kSumBits;
// and a row's own reference is then the largest score plus the logarithm of V's
// scale, down to 2^-kRoom, of what it sees.  So p times the scale is 2^kLift there,
// whatever stands in other drafts, and p alone at most 2^(kRoom + kSlack + kLift),
// far from where its sums leave fp32.
constexpr float kRoom = 64.f;
constexpr int kSumBits = 96;
__device__ __forceinline__ int exponent_of(float x) { return static_cast<int>(__float_as_uint(x) >> 23 & 255u) - 127; }
__device__ __forceinline__ float power_of_two(int n) { return __uint_as_float(static_cast<uint32_t>(n + 127) << 23); }
// By how many powers of two a row's reference goes down, of `rise`: 0 .. 120.
__device__ __forceinline__ int lowered(float sum, int rise) {
  return max(0, min(min(rise, 120), kSumBits - exponent_of(sum)));
}

// The reference of a row that has seen nothing yet.
constexpr float kNoScore = -3e38f;

// N neighbouring entries of a finished row: sum / l, gated, rounded.  The gate
// has been read already: it may be `out` itself.
template <typename T, int N, int V>
__device__ __forceinline__ void write_out(const AttnParams& p, int64_t row, int column,
                                          const float (&sum)[N], float l,
                                          const Vec<T, V> (&gate)[N / V]) {
  const float inv = l == 0.f ? 0.f : __frcp_rn(l);  // nothing seen: 0
#pragma unroll
  for (int i = 0; i < N / V; ++i) {
    float o[V];
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = l == 0.f ? 0.f : sum[i * V + j] * inv;
    if (p.gate) {
      float x[V];
      widen(gate[i], x);
#pragma unroll
      for (int j = 0; j < V; ++j) o[j] *= p.sigmoid ? __fdividef(1.f, 1.f + __expf(-x[j])) : x[j];
    }
    store_vec<T, V>(reinterpret_cast<T*>(p.out + row * p.ldo) + column + i * V, o);
  }
}
__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// tcgen05 kernel (attn_tc.cu).
constexpr int kAttnTcRows = 128;  // rows of an item there
constexpr int kAttnTcUnit = 64;
cudaError_t attn_tc_launch(const AttnParams& p, int dtype, int format, cudaStream_t s);

}  // namespace proj
