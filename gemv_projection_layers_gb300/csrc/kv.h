// kv.h -- the cache of keys and values as the kernels see it (kv.cu, attn.cu,
// attn_tc.cu), and the host checks that its calls share.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/proj.h"

namespace proj {

// Quotients by a divisor that is known at launch: the multiplication of
// Granlund and Montgomery, "Division by invariant integers using
// multiplication" (1994), fig. 4.1; exact for numerators below 2^31.
struct Divisor {
  uint32_t d, mul, shift;
};
inline Divisor make_divisor(uint32_t d) {
  uint32_t s = 0;
  while ((uint64_t{1} << s) < d) ++s;
  const uint64_t mul = ((uint64_t{1} << 32) * ((uint64_t{1} << s) - d)) / d + 1;
  return {d, static_cast<uint32_t>(mul), s};
}
__device__ __forceinline__ int quotient(int n, const Divisor& v) {
  return static_cast<int>((__umulhi(v.mul, static_cast<uint32_t>(n)) + static_cast<uint32_t>(n)) >> v.shift);
}

struct KvCache {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  int64_t page_stride, head_stride, token_stride;  // bytes; pages and tokens: below 2^31
  const int32_t* table;
  int64_t ldt;
  Divisor page;
  int pages, heads, width, sequences;
  int page_scales;  // scales of a page: heads * page
  int capacity;  // positions of a sequence: width * page, below 2^31
};

// Where a position of a sequence stands: the byte offset of a head's entry and
// the index of its scale; false where the table has no page for it.
struct Entry {
  int64_t at, scale;
};
__device__ __forceinline__ bool page_of(const KvCache& c, int sequence, int position, int& id,
                                        int& spot) {
  if (position < 0 || position >= c.capacity) return false;
  const int slot = quotient(position, c.page);
  spot = position - slot * static_cast<int>(c.page.d);
  id = c.table[sequence * c.ldt + slot];
  return id >= 0 && id < c.pages;
}
__device__ __forceinline__ Entry entry_at(const KvCache& c, int id, int spot, int head) {
  return {id * c.page_stride + head * c.head_stride + spot * c.token_stride,
          (static_cast<int64_t>(id) * c.heads + head) * c.page.d + spot};
}

// Rows lo .. hi - 1 of the call are the sequence's: offsets are moved into
// 0 .. m and taken as not decreasing.
__device__ __forceinline__ void rows_of(const int32_t* offsets, int sequence, int m, int& lo,
                                        int& hi) {
  lo = min(max(offsets[sequence], 0), m);
  hi = min(max(offsets[sequence + 1], lo), m);
}

// Host side: the cache's fields checked (nullptr and PROJ_OK if they are
// fine) and laid out for the kernels.
const char* refuse_cache(const proj_kv_cache* c, int* status);
KvCache device_cache(const proj_kv_cache& c);
int kv_refuse(int status, const char* call, const char* why);
inline bool kv_aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace proj
