// kv.cu -- rows of keys and values to the cache, back from it, and accepted
// drafts to their places.
//
// Writing quantises: a row's largest magnitude, the scale and its reciprocal
// (rounded to nearest each), a multiplication and a rounding an entry.  Reading multiplies code by scale and rounds.  Moving
// copies bytes.  All three are bound by the bytes they move, and by one chain
// of dependent loads (offsets, start, table, entry) where there are few rows
// (2.2 us).  139000 rows of 8 heads of 128 back from e4m3: 178 us (5.8 TB/s); 8192
// rows of 8 heads to int8: 12.9 us (3.9 TB/s; the chain is a third of it); 256 paths
// of 32 rows of 8 heads, 16-bit: 11.7 us (3.6 TB/s).
//
// A warp takes a row of the call: it finds the row's sequence once (a search
// in `offsets` that halves the range five times a step: 32 lanes look at 32
// places), then goes over the heads of keys and values, D / 8 or D / 16 lanes
// to a head's row and 16 bytes a lane.  Where there are fewer rows than warps
// that run at a time, the heads of a row are spread over several warps.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdio>

#include "kernels.h"
#include "kv.h"
#include "kv_num.cuh"
#include "ptx.cuh"
#include "vec.cuh"

namespace proj {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct RowsParams {
  KvCache c;
  const int32_t* offsets;
  const int32_t* start;
  int m;
  int split;        // warps to a row
  uint8_t* k;       // rows of the call
  uint8_t* v;
  int64_t ldk, ldv;  // bytes
};

// The sequence of a row: how many of offsets[1 .. n] are not above it (all of
// a warp's lanes together); n where it is none's.
__device__ __forceinline__ int sequence_of(const int32_t* offsets, int n, int row, int lane) {
  int lo = 0, left = n;
  while (left > 0) {
    const int step = (left + 31) / 32;
    const int at = lo + (lane + 1) * step - 1;
    const bool below = at < lo + left && offsets[at + 1] <= row;
    const int passed = __popc(__ballot_sync(0xFFFFFFFFu, below)) * step;
    lo += passed;
    left = min(step - 1, left - passed);
  }
  return lo;
}

// The position that a row of the call stands for; false where it is no
// sequence's.
__device__ __forceinline__ bool position_of(const RowsParams& p, int row, int lane, int& sequence,
                                            int& position) {
  sequence = sequence_of(p.offsets, p.c.sequences, row, lane);
  if (sequence >= p.c.sequences) return false;
  const int lo = max(p.offsets[sequence], 0);
  if (row < lo) return false;
  const int64_t at = static_cast<int64_t>(p.start[sequence]) + (row - lo);
  position = at < 0 || at >= p.c.capacity ? -1 : static_cast<int>(at);
  return true;
}

// kFormat: enum proj_kv_format.  A lane has 16 entries of a head's row: what a row
// costs beside its entries (scale, addresses) weighs half as much as with eight.
template <typename T, int kFormat, int D>
__global__ void __launch_bounds__(kThreads, 8) kv_write_kernel(const RowsParams p) {
  constexpr int L = D / 16;  // lanes of a row
  const int lane = threadIdx.x & 31;
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  griddep_launch_dependents();
  griddep_wait();
  const int64_t row = warp / p.split;
  if (row >= p.m) return;
  int sequence, position, id = 0, spot = 0;
  if (!position_of(p, static_cast<int>(row), lane, sequence, position)) return;
  if (!page_of(p.c, sequence, position, id, spot)) return;
  const int items = 2 * p.c.heads, passes = (items * L + 31) / 32;
  const int part = static_cast<int>(warp - row * p.split);
  const Entry first = entry_at(p.c, id, spot, 0);
  const uint8_t* const k_row = p.k + row * p.ldk;
  const uint8_t* const v_row = p.v + row * p.ldv;
#pragma unroll 1
  for (int pass = part; pass < passes; pass += p.split) {
    const int item = pass * (32 / L) + lane / L;
    const bool real = item < items;
    const bool is_v = item >= p.c.heads;
    const int head = real ? item - (is_v ? p.c.heads : 0) : 0;
    const uint8_t* from = (is_v ? v_row : k_row) + (head * D + (lane % L) * 16) * 2;
    const uint4 x = *reinterpret_cast<const uint4*>(from), y = *reinterpret_cast<const uint4*>(from + 16);
    uint8_t* to = (is_v ? p.c.v : p.c.k) + first.at + head * p.c.head_stride;
    if constexpr (kFormat == PROJ_KV_ROWS) {
      if (real) {
        *reinterpret_cast<uint4*>(to + (lane % L) * 32) = x;
        *reinterpret_cast<uint4*>(to + (lane % L) * 32 + 16) = y;
      }
    } else {
      // Magnitudes order as their bits, with infinities and NaN above the rest.
      const uint32_t m = 0x7FFF7FFFu;
      uint32_t top = __vmaxu2(__vmaxu2(__vmaxu2(x.x & m, x.y & m), __vmaxu2(x.z & m, x.w & m)),
                              __vmaxu2(__vmaxu2(y.x & m, y.y & m), __vmaxu2(y.z & m, y.w & m)));
#pragma unroll
      for (int o = L / 2; o; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
      float amax, other;
      top = max(top & 0xFFFFu, top >> 16);
      widen2(top, amax, other, T());
      const bool finite = amax < INFINITY;
      constexpr float kTop = kFormat == PROJ_KV_E4M3 ? 448.f : 127.f;
      const float scale = fmaxf(__fdiv_rn(amax, kTop), 1.17549435e-38f);
      const F2 inv = f2(finite ? __frcp_rn(scale) : 0.f);
      const uint32_t word[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
      uint32_t code[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float f[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          widen2(finite ? word[2 * i + j] : 0u, f[2 * j], f[2 * j + 1], T());
          parts(mul2(f2(f[2 * j], f[2 * j + 1]), inv), f[2 * j], f[2 * j + 1]);
        }
        code[i] = encode4<kFormat>(f[0], f[1], f[2], f[3]);
      }
      if (real) {
        *reinterpret_cast<uint4*>(to + (lane % L) * 16) = make_uint4(code[0], code[1], code[2], code[3]);
        if (lane % L == 0)
          (is_v ? p.c.v_scale : p.c.k_scale)[first.scale + static_cast<int64_t>(head) * p.c.page.d] =
              finite ? scale : __uint_as_float(0x7FC00000u);
      }
    }
  }
}

// A lane has 16 bytes of entries.
template <typename T, int kFormat, int D>
__global__ void __launch_bounds__(kThreads, 8) kv_read_kernel(const RowsParams p) {
  constexpr int E = kFormat == PROJ_KV_ROWS ? 8 : 16;
  constexpr int L = D / E;
  const int lane = threadIdx.x & 31;
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  griddep_launch_dependents();
  griddep_wait();
  const int64_t row = warp / p.split;
  if (row >= p.m) return;
  int sequence, position, id = 0, spot = 0;
  if (!position_of(p, static_cast<int>(row), lane, sequence, position)) return;
  const bool here = page_of(p.c, sequence, position, id, spot);
  if (!here) id = spot = 0;
  const int items = 2 * p.c.heads, passes = (items * L + 31) / 32;
  const int part = static_cast<int>(warp - row * p.split);
#pragma unroll 1
  for (int pass = part; pass < passes; pass += p.split) {
    const int item = pass * (32 / L) + lane / L;
    const bool is_v = item >= p.c.heads;
    const int head = item < items ? item - (is_v ? p.c.heads : 0) : 0;
    const bool real = item < items && (is_v ? p.v : p.k) != nullptr;
    const Entry e = entry_at(p.c, id, spot, head);
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    float scale = 0.f;
    if (here && real) {
      w = *reinterpret_cast<const uint4*>((is_v ? p.c.v : p.c.k) + e.at + (lane % L) * 16);
      if constexpr (kFormat != PROJ_KV_ROWS) scale = (is_v ? p.c.v_scale : p.c.k_scale)[e.scale];
    }
    if (!real) continue;
    uint8_t* to = (is_v ? p.v + row * p.ldv : p.k + row * p.ldk) +
                  (static_cast<int64_t>(head) * D + (lane % L) * E) * 2;
    if constexpr (kFormat == PROJ_KV_ROWS) {
      *reinterpret_cast<uint4*>(to) = w;
    } else {
      const uint32_t word[4] = {w.x, w.y, w.z, w.w};
      float f[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        widen2(decode_pair<kFormat>(word[i], 0), f[4 * i], f[4 * i + 1], __half());
        widen2(decode_pair<kFormat>(word[i], 1), f[4 * i + 2], f[4 * i + 3], __half());
      }
      float a[8], b[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] = f[i] * scale;
        b[i] = f[i + 8] * scale;
      }
      store_vec<T, 8>(reinterpret_cast<T*>(to), a);
      store_vec<T, 8>(reinterpret_cast<T*>(to) + 8, b);
    }
  }
}

struct MoveParams {
  KvCache c;
  const int32_t* start;
  const int32_t* path;
  int64_t ldp;
  int depth, words, word_shift, scales;  // 16-byte words of an entry and their logarithm; 1: a scale as well
  int32_t* next;
};

// A CTA has 32 of the 16-byte words of a sequence's entries (scales behind them),
// one a lane, and goes through the path in runs of 32: lanes check that it
// ascends and find the places of an entry each, and the warps take the entries in
// turn.  All loads of a run come before its first store: a target can be another
// entry's source, of the same run or an earlier one, but not of a later one, whose
// sources lie behind.  (Runs of 64 hold twice as much in registers, for fewer CTAs an
// SM: 256 paths of 32 x 16 heads' rows took 19.5 us, 11.7 so, in 2.7 rounds of CTAs.)
constexpr int kRun = 32;

__global__ void __launch_bounds__(kThreads, 5) kv_move_kernel(const MoveParams p) {
  constexpr int kEach = kRun / kWarps;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.y;
  const int words = 2 * p.c.heads * p.words;
  int unit = blockIdx.x * 32 + lane;
  const bool is_scale = unit >= words;
  const bool mine = unit < words + 2 * p.c.heads * p.scales;
  if (is_scale) unit -= words;
  const int item = is_scale ? unit : unit >> p.word_shift, word = unit - (item << p.word_shift);
  const bool is_v = item >= p.c.heads;
  const int head = mine ? item - (is_v ? p.c.heads : 0) : 0;
  uint8_t* const entries = (is_v ? p.c.v : p.c.k) + head * p.c.head_stride + word * 16;
  float* const scales = (is_v ? p.c.v_scale : p.c.k_scale) + static_cast<int64_t>(head) * p.c.page.d;
  griddep_launch_dependents();
  griddep_wait();
  const int start = p.start[b];
  const int32_t* path = p.path + b * p.ldp;
  int before = -1, n = 0;
  for (bool more = true; more && n < p.depth;) {
    // Entry `lane` of the run: both of its pages are asked for together.
    const int step = n + lane < p.depth ? path[n + lane] : -1;
    const int64_t at[2] = {static_cast<int64_t>(start) + step, static_cast<int64_t>(start) + n + lane};
    // entries that stay where they are are not touched
    bool ok = at[0] != at[1] && step >= 0;
    int id[2], spot[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      ok = ok && at[x] >= 0 && at[x] < p.c.capacity;
      const int position = ok ? static_cast<int>(at[x]) : 0;
      const int slot = quotient(position, p.c.page);
      spot[x] = position - slot * static_cast<int>(p.c.page.d);
      id[x] = p.c.table[b * p.c.ldt + slot];
    }
    const int above = __shfl_up_sync(0xFFFFFFFFu, step, 1);
    const uint32_t rises = __ballot_sync(0xFFFFFFFFu, step > (lane ? above : before));
    const int length = __ffs(~rises) - 1;  // of the leading part that rises; -1: all do
    const int count = length < 0 ? 32 : length;
    more = count == 32;
    before = __shfl_sync(0xFFFFFFFFu, step, 31);
    Entry place[2];  // source, target
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      ok = ok && id[x] >= 0 && id[x] < p.c.pages;
      place[x] = entry_at(p.c, id[x], spot[x], 0);
    }
    const uint32_t good = __ballot_sync(0xFFFFFFFFu, ok && lane < count);
    uint4 w[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int e = i * kWarps + warp;
      if (!(good >> e & 1)) continue;  // the whole warp
      const int64_t source = __shfl_sync(0xFFFFFFFFu, place[0].at, e);
      if (mine && !is_scale) w[i] = *reinterpret_cast<const uint4*>(entries + source);
      if (p.scales) {
        const int64_t scale = __shfl_sync(0xFFFFFFFFu, place[0].scale, e);
        if (mine && is_scale) w[i].x = __float_as_uint(scales[scale]);
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int e = i * kWarps + warp;
      if (!(good >> e & 1)) continue;
      const int64_t target = __shfl_sync(0xFFFFFFFFu, place[1].at, e);
      if (mine && !is_scale) *reinterpret_cast<uint4*>(entries + target) = w[i];
      if (p.scales) {
        const int64_t scale = __shfl_sync(0xFFFFFFFFu, place[1].scale, e);
        if (mine && is_scale) scales[scale] = __uint_as_float(w[i].x);
      }
    }
    n += count;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.next) p.next[b] = start + n;
}

cudaLaunchConfig_t config(int64_t grid_x, int64_t grid_y, cudaStream_t s,
                          cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid_x), static_cast<unsigned>(grid_y));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

using RowsKernel = void (*)(RowsParams);

template <typename T, int D>
RowsKernel pick(int format, bool write) {
  switch (format) {
    case PROJ_KV_ROWS:
      return write ? kv_write_kernel<T, PROJ_KV_ROWS, D> : kv_read_kernel<T, PROJ_KV_ROWS, D>;
    case PROJ_KV_E4M3:
      return write ? kv_write_kernel<T, PROJ_KV_E4M3, D> : kv_read_kernel<T, PROJ_KV_E4M3, D>;
    default:
      return write ? kv_write_kernel<T, PROJ_KV_INT8, D> : kv_read_kernel<T, PROJ_KV_INT8, D>;
  }
}

int rows_call(const char* call, bool write, const proj_kv_cache* cache, const int32_t* offsets,
              const int32_t* start, int64_t m, const void* k, int64_t ldk, const void* v,
              int64_t ldv, proj_stream stream) {
  int status = PROJ_OK;
  if (const char* why = refuse_cache(cache, &status)) return kv_refuse(status, call, why);
  const proj_kv_cache& c = *cache;
  if (m < 0) return kv_refuse(PROJ_EINVAL, call, "m < 0");
  if (m >= (int64_t{1} << 30)) return kv_refuse(PROJ_EUNSUPPORTED, call, "m >= 2^30");
  if (m > 0 && c.sequences > 0 && (!offsets || !start))
    return kv_refuse(PROJ_EINVAL, call, "offsets or start is NULL");
  if (m > 0 && (write ? !k || !v : !k && !v)) return kv_refuse(PROJ_EINVAL, call, "k or v is NULL");
  const int64_t width = c.heads * c.D;
  if ((k && ldk < width) || (v && ldv < width))
    return kv_refuse(PROJ_EINVAL, call, "a row stride is below heads D");
  if (ldk >= (int64_t{1} << 31) || ldv >= (int64_t{1} << 31))
    return kv_refuse(PROJ_EUNSUPPORTED, call, "a row stride of 2^31 or more");
  if (!kv_aligned(k, 16) || !kv_aligned(v, 16) || (k && ldk % 8) || (v && ldv % 8))
    return kv_refuse(PROJ_EALIGN, call, "rows of k or v do not start on 16 bytes");
  if (!kv_aligned(offsets, 4) || !kv_aligned(start, 4))
    return kv_refuse(PROJ_EALIGN, call, "offsets or start is not aligned to 4 bytes");
  if (m == 0 || c.sequences == 0) return PROJ_OK;
  RowsParams p = {};
  p.c = device_cache(c);
  p.offsets = offsets;
  p.start = start;
  p.m = static_cast<int>(m);
  p.k = static_cast<uint8_t*>(const_cast<void*>(k));
  p.v = static_cast<uint8_t*>(const_cast<void*>(v));
  p.ldk = ldk * 2;
  p.ldv = ldv * 2;
  const int lanes = static_cast<int>(c.D) / (!write && c.format == PROJ_KV_ROWS ? 8 : 16);
  const int64_t passes = (2 * c.heads * lanes + 31) / 32;
  // 4096 warps: some 27 an SM, enough to have the bytes in flight that HBM wants
  p.split = static_cast<int>(std::max<int64_t>(1, std::min(passes, 4096 / m)));
  RowsKernel kernel;
  if (c.dtype == PROJ_BF16)
    kernel = c.D == 64 ? pick<__nv_bfloat16, 64>(c.format, write) : pick<__nv_bfloat16, 128>(c.format, write);
  else
    kernel = c.D == 64 ? pick<__half, 64>(c.format, write) : pick<__half, 128>(c.format, write);
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg =
      config((m * p.split + kWarps - 1) / kWarps, 1, reinterpret_cast<cudaStream_t>(stream), attr);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e == cudaSuccess ? PROJ_OK : record_cuda(e, call);
}

}  // namespace

int kv_refuse(int status, const char* call, const char* why) {
  char text[160];
  std::snprintf(text, sizeof text, "%s: %s", call, why);
  return record_status(status, text);
}

const char* refuse_cache(const proj_kv_cache* cache, int* status) {
  *status = PROJ_EINVAL;
  if (!cache) return "cache is NULL";
  const proj_kv_cache& c = *cache;
  if (c.format < PROJ_KV_ROWS || c.format > PROJ_KV_INT8) return "unknown format";
  if (c.dtype != PROJ_BF16 && c.dtype != PROJ_FP16) return "dtype is neither PROJ_BF16 nor PROJ_FP16";
  if (c.pages < 1 || c.page < 1 || c.heads < 1 || c.width < 1 || c.sequences < 0)
    return "pages, page, heads or width < 1, or sequences < 0";
  if (c.ldt < c.width) return "ldt is below width";
  if (!c.k || !c.v || (c.sequences > 0 && !c.table)) return "k, v or table is NULL";
  const bool scaled = c.format != PROJ_KV_ROWS;
  if (scaled != (c.k_scale != nullptr) || scaled != (c.v_scale != nullptr))
    return "scales and format do not agree";
  if (c.page_stride < c.D || c.head_stride < c.D || c.token_stride < c.D)
    return "a stride of the cache is below D";
  *status = PROJ_EUNSUPPORTED;
  if (c.D != 64 && c.D != 128) return "D is neither 64 nor 128";
  if (c.heads > 1024) return "more than 1024 heads";
  if (c.page > 65536) return "pages of more than 65536 tokens";
  if (c.pages >= (int64_t{1} << 31)) return "2^31 pages or more";
  if (c.sequences > 65536) return "more than 65536 sequences";
  if (c.width >= (int64_t{1} << 30) / c.page) return "width page >= 2^30";
  if (c.ldt >= (int64_t{1} << 31)) return "ldt >= 2^31";
  const int64_t el = scaled ? 1 : 2, most = int64_t{1} << 31;
  if (c.page_stride >= most / el || c.token_stride >= most / el || c.head_stride >= (most << 16))
    return "a page or token stride of 2^31 bytes or a head stride of 2^47 or more";
  *status = PROJ_EALIGN;
  if (!kv_aligned(c.k, 16) || !kv_aligned(c.v, 16) || c.page_stride * el % 16 ||
      c.head_stride * el % 16 || c.token_stride * el % 16)
    return "entries of the cache do not start on 16 bytes";
  if (!kv_aligned(c.k_scale, 4) || !kv_aligned(c.v_scale, 4) || !kv_aligned(c.table, 4))
    return "scales or table are not aligned to 4 bytes";
  *status = PROJ_OK;
  return nullptr;
}

KvCache device_cache(const proj_kv_cache& c) {
  const int64_t el = c.format == PROJ_KV_ROWS ? 2 : 1;
  KvCache d = {};
  d.k = static_cast<uint8_t*>(c.k);
  d.v = static_cast<uint8_t*>(c.v);
  d.k_scale = c.k_scale;
  d.v_scale = c.v_scale;
  d.page_stride = c.page_stride * el;
  d.head_stride = c.head_stride * el;
  d.token_stride = c.token_stride * el;
  d.table = c.table;
  d.ldt = c.ldt;
  d.page = make_divisor(static_cast<uint32_t>(c.page));
  d.pages = static_cast<int>(c.pages);
  d.heads = static_cast<int>(c.heads);
  d.width = static_cast<int>(c.width);
  d.sequences = static_cast<int>(c.sequences);
  d.page_scales = static_cast<int>(c.heads * c.page);
  d.capacity = static_cast<int>(c.width * c.page);
  return d;
}

}  // namespace proj

using namespace proj;

extern "C" int proj_kv_write(const proj_kv_cache* cache, const int32_t* offsets,
                             const int32_t* start, int64_t m, const void* k, int64_t ldk,
                             const void* v, int64_t ldv, proj_stream stream) {
  return rows_call("proj_kv_write", true, cache, offsets, start, m, k, ldk, v, ldv, stream);
}

extern "C" int proj_kv_read(const proj_kv_cache* cache, const int32_t* offsets,
                            const int32_t* start, int64_t m, void* k, int64_t ldk, void* v,
                            int64_t ldv, proj_stream stream) {
  return rows_call("proj_kv_read", false, cache, offsets, start, m, k, ldk, v, ldv, stream);
}

extern "C" int proj_kv_move(const proj_kv_cache* cache, const int32_t* start, const int32_t* path,
                            int64_t ldp, int64_t depth, int32_t* next_start, proj_stream stream) {
  const char* const call = "proj_kv_move";
  int status = PROJ_OK;
  if (const char* why = refuse_cache(cache, &status)) return kv_refuse(status, call, why);
  const proj_kv_cache& c = *cache;
  if (depth < 0 || ldp < depth) return kv_refuse(PROJ_EINVAL, call, "depth < 0, or ldp below depth");
  if (depth >= (int64_t{1} << 30) || ldp >= (int64_t{1} << 31))
    return kv_refuse(PROJ_EUNSUPPORTED, call, "depth >= 2^30 or ldp >= 2^31");
  if (c.sequences > 0 && (!start || (depth > 0 && !path)))
    return kv_refuse(PROJ_EINVAL, call, "start or path is NULL");
  if (next_start && next_start == start)
    return kv_refuse(PROJ_EINVAL, call, "next_start is start itself");
  if (!kv_aligned(start, 4) || !kv_aligned(path, 4) || !kv_aligned(next_start, 4))
    return kv_refuse(PROJ_EALIGN, call, "a pointer is not aligned to 4 bytes");
  if (c.sequences == 0 || (depth == 0 && !next_start)) return PROJ_OK;
  MoveParams p = {};
  p.c = device_cache(c);
  p.start = start;
  p.path = path;
  p.ldp = ldp;
  p.depth = static_cast<int>(depth);
  p.scales = c.format != PROJ_KV_ROWS;
  p.words = static_cast<int>(c.D) * (p.scales ? 1 : 2) / 16;
  p.word_shift = p.words == 4 ? 2 : p.words == 8 ? 3 : 4;
  p.next = next_start;
  const int64_t units = 2 * c.heads * (p.words + p.scales);
  // grid y: sequences, of which 65535 are allowed there; the last one of 65536 goes alone
  for (int64_t at = 0; at < c.sequences; at += 65535) {
    MoveParams q = p;
    q.c.table = p.c.table + at * c.ldt;
    q.start = start + at;
    q.path = path + at * ldp;
    q.next = next_start ? next_start + at : nullptr;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg =
        config((units + 31) / 32, std::min<int64_t>(65535, c.sequences - at),
               reinterpret_cast<cudaStream_t>(stream), attr);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kv_move_kernel, q);
    if (e != cudaSuccess) return record_cuda(e, call);
  }
  return PROJ_OK;
}
