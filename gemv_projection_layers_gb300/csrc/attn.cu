// attn.cu -- attention of drafted tokens over the cache: the calls, the kernel
// for few rows, and the join of partial results.
//
// The kernel for few rows (a group's heads times a sequence's drafts up to 32, and
// more of a short cache; items of 8 or 16) is a stream over the cache.  Per key and
// head it reads 2 D entries and does 4 D operations a row, so with 8 rows and 8-bit
// entries the cache's bytes at HBM's rate leave the tensor cores of the warp-level MMA
// a fifth of their time; what counts is that the bytes flow.  Each of a CTA's eight
// warps has a ring of its own in shared memory, filled by 16-byte asynchronous copies,
// and takes every eighth step of the CTA's share, 32 keys (16 of 16-bit entries and
// 128 dimensions): nothing but the end of an item is a barrier for the CTA.  Where
// there are many items, each warp has a share of its own and no barrier at all.  From
// 16384 to 65536 keys of 16 sequences a call's time grows as the bytes at HBM's
// measured rate do (e4m3 20 us a 20 us, 16-bit 38 a 39); below, it is the chain
// of a call that shows: lengths, pages, first bytes, the warps' and the CTAs' sums
// (9 us for one sequence of 8192 keys, of which the join is some 3).
//
// Keys are the M side of both products, rows the N side (eight at a time, so
// nothing is padded to 16):
//   S^T [16 keys x 8 rows] = K [16 x D] Q^T,   O^T [D x 8 rows] += V^T [D x 16] P^T.
// K and V come out of the ring as A fragments (ldmatrix, V transposed) and are
// decoded in registers, once, for all rows: 8-bit codes are exact in fp16.  A
// 16-bit unit of ldmatrix is then two codes, so the order of dimensions within
// 16 is the one it gives, for Q alike, and output rows 2 i, 2 i + 1 are
// neighbours.  P^T goes from accumulators to B fragments by transposing 8 x 8
// blocks in registers.
//
// Softmax, one pass: each warp holds for its rows a reference m and sums
// relative to 2^m, and a score well above m moves it (a vote; no shuffles
// otherwise).  Scales of V multiply p, relative to the largest one met (kRoom in
// attn.h: what that means for rows that do not see it).
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdio>
#include <type_traits>

#include "attn.h"
#include "kernels.h"
#include "kv_num.cuh"

namespace proj {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
__device__ uint32_t g_attn_status;  // what bounded waits that gave up leave

constexpr int kUnit = 32;  // keys of a unit of work

template <int kFormat, int D, int NT>
struct Stream {
  static constexpr int kRow = kFormat == PROJ_KV_ROWS ? 2 * D : D;  // bytes of an entry
  static constexpr int kStep = kRow == 256 ? 16 : 32;              // keys of a warp's step
  static constexpr int kTiles = kStep / 16;
  static constexpr int kHalf = kStep * kRow;                       // K or V of a step
  static constexpr int kStage = 2 * kHalf + 8 * kStep;             // and their scales
  static constexpr int kStages = kRow == 64 ? 5 : 3;
  static constexpr int kRing = kStages * kStage;  // of a warp
  static constexpr int kRows = 8 * NT;
  static constexpr int kPitch = D + 4;            // floats of a row in the merge
  static constexpr int kMerge = kWarps * kRows * kPitch * 4;
  static constexpr int kMl = kWarps * kRows * 8;
  static constexpr int kSmem = (kWarps * kRing > kMerge ? kWarps * kRing : kMerge) + kMl;
  static_assert(kSmem + 1024 <= 232448, "shared memory");
};

// Where 16-byte piece c of a row stands: eight rows' pieces of one column fall
// into different banks.
template <int kRow>
__device__ __forceinline__ uint32_t place(int row, int c) {
  const int turn = kRow == 64 ? (row >> 1) & 3 : row & 7;
  return row * kRow + ((c ^ turn) << 4);
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1, __half) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1, __nv_bfloat16) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ld_shared_f(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

// Whether one of a pair of 16-bit numbers is an infinity or a NaN.
__device__ __forceinline__ bool odd_pair(uint32_t w, __half) {
  return (w & 0x7C00u) == 0x7C00u || (w & 0x7C000000u) == 0x7C000000u;
}
__device__ __forceinline__ bool odd_pair(uint32_t w, __nv_bfloat16) {
  return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}

// kSolo: each warp has a share of its own, and the sums of an item's part are its
// alone; nothing in the kernel is a barrier for the CTA.
template <typename T, int kFormat, int D, int NT, bool kSolo>
__global__ void __launch_bounds__(kThreads, 1) attn_stream_kernel(const AttnParams p) {
  using F = Stream<kFormat, D, NT>;
  constexpr bool kCoded = kFormat != PROJ_KV_ROWS;
  using C = std::conditional_t<kCoded, __half, T>;  // what is multiplied
  constexpr bool kRest = !kCoded;  // P as a sum of two 16-bit numbers
  constexpr int kRow = F::kRow, S = F::kStages, KK = D / 16, kPieces = kRow / 16;
  constexpr int kTurn = 32 / kPieces;  // rows that a warp copies at a time
  constexpr int kStep = F::kStep, MT = F::kTiles, kUnitSteps = kUnit / kStep;
  constexpr uint32_t kAll = kStep == 32 ? 0xFFFFFFFFu : 0xFFFFu;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ uint32_t s_valid[kWarps][S];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c4 = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * F::kRing;
  constexpr int kTeam = kSolo ? 1 : kWarps;  // warps to a share
  const int member = kSolo ? 0 : warp, tid = kSolo ? lane : threadIdx.x;
  const int worker = kSolo ? blockIdx.x * kWarps + warp : blockIdx.x;
  const auto team_sync = [] {
    if constexpr (kSolo)
      __syncwarp();
    else
      __syncthreads();
  };
  float* const merge = reinterpret_cast<float*>(smem + (kSolo ? warp * F::kRing : 0));
  float* const s_ml = reinterpret_cast<float*>(smem + F::kSmem - F::kMl) + (kSolo ? warp * F::kRows * 2 : 0);

  touch(p);
  griddep_launch_dependents();
  griddep_wait();
  Share share;
  if (!find_share<kThreads, kSolo>(p, kSolo ? blockIdx.x * kWarps : blockIdx.x, share)) {
    if (tid == 0) p.splits[worker] = Split{};
    return;
  }

  const int G = static_cast<int>(p.group.d);
  int b = share.b;
  int64_t before = share.before;
  Sequence seq = sequence_at(p, b);
  bool told = false;
  for (int64_t at = share.first; at < share.end;) {
    while (at >= before + units_of(p, seq)) {
      before += units_of(p, seq);
      if (++b >= p.c.sequences) return;
      seq = sequence_at(p, b);
    }
    const int64_t local = at - before;
    const int64_t item = item_of(local, seq.units);
    const int u0 = static_cast<int>(local - item * seq.units);
    const int u1 = static_cast<int>(min(static_cast<int64_t>(seq.units), u0 + (share.end - at)));
    const int head = static_cast<int>(item_of(item, seq.tiles));
    const int row0 = static_cast<int>(item - static_cast<int64_t>(head) * seq.tiles) * F::kRows;
    const int all_rows = seq.rows * G;

    // --------------------------------------------------------------- ring --
    const int all_steps = (u1 - u0) * kUnitSteps;
    const int steps = all_steps > member ? (all_steps - member + kTeam - 1) / kTeam : 0;
    const auto first_key = [&](int i) { return u0 * kUnit + (member + i * kTeam) * kStep; };
    const int32_t* const table = p.c.table + b * p.c.ldt;
    const int64_t head_at = head * p.c.head_stride, head_scale = static_cast<int64_t>(head) * p.c.page.d;
    // the page of key `lane` (< kStep) of step i, or -1
    const auto page_id = [&](int i) {
      const int pos = first_key(i) + lane;
      if (i >= steps || lane >= kStep || pos >= seq.len) return -1;
      return table[quotient(pos, p.c.page)];
    };
    const auto issue = [&](int i, int id, int slot) {
      if (i < steps) {
        const int pos = first_key(i) + lane;
        const int spot = pos - quotient(pos, p.c.page) * static_cast<int>(p.c.page.d);
        const bool ok = id >= 0 && id < p.c.pages;
        const int64_t at = ok ? head_at + static_cast<int64_t>(id) * static_cast<int>(p.c.page_stride) +
                                    static_cast<int64_t>(spot) * static_cast<int>(p.c.token_stride)
                              : 0;
        const uint32_t valid = __ballot_sync(0xFFFFFFFFu, ok) & kAll;
        const uint32_t stage = ring + slot * F::kStage;
        if (lane == 0) s_valid[warp][slot] = valid;
        const uint8_t* const k_from = p.c.k + lane % kPieces * 16;
        const uint8_t* const v_from = p.c.v + lane % kPieces * 16;
#pragma unroll
        for (int j = 0; j < kStep / kTurn; ++j) {
          const int key = j * kTurn + lane / kPieces;
          const int64_t from = __shfl_sync(0xFFFFFFFFu, at, key);
          const int bytes = valid >> key & 1 ? 16 : 0;
          const uint32_t to = stage + place<kRow>(key, lane % kPieces);
          copy16(to, k_from + from, bytes);
          copy16(to + F::kHalf, v_from + from, bytes);
        }
        if constexpr (kCoded) {
          if (lane < kStep) {
            const int64_t from = ok ? head_scale + static_cast<int64_t>(id) * p.c.page_scales + spot : 0;
            copy4(stage + 2 * F::kHalf + lane * 4, p.c.k_scale + from, ok ? 4 : 0);
            copy4(stage + 2 * F::kHalf + 4 * kStep + lane * 4, p.c.v_scale + from, ok ? 4 : 0);
          }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int ids[S];
#pragma unroll
    for (int i = 0; i < S; ++i) ids[i] = page_id(i);
#pragma unroll
    for (int i = 0; i < S - 1; ++i) issue(i, ids[i], i);
    int next_id = ids[S - 1], slot = 0, in_slot = S - 1;


    // ------------------------------------------------------------ queries --
    uint32_t qf[KK][NT][2];
    float fq[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = row0 + nt * 8 + g;
      const int t = quotient(r, p.group);
      const uint8_t* from = p.q + (seq.lo + t) * p.ldq + static_cast<int64_t>(head * G + r - t * G) * D * 2;
      const bool real = r < all_rows;
      if constexpr (!kCoded) {
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
          qf[kk][nt][0] = real ? *reinterpret_cast<const uint32_t*>(from + kk * 32 + c4 * 4) : 0u;
          qf[kk][nt][1] = real ? *reinterpret_cast<const uint32_t*>(from + kk * 32 + 16 + c4 * 4) : 0u;
        }
        fq[nt][0] = fq[nt][1] = p.scale_log2;
      } else {
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
          const uint2 w = real ? *reinterpret_cast<const uint2*>(from + kk * 32 + c4 * 8) : make_uint2(0u, 0u);
          qf[kk][nt][0] = w.x;
          qf[kk][nt][1] = w.y;
        }
        float f = 1.f;
        if constexpr (std::is_same_v<T, __nv_bfloat16>) {
          // bf16 to fp16: the row's largest magnitude is brought to 2^14 .. 2^15
          uint32_t top = 0;
#pragma unroll
          for (int kk = 0; kk < KK; ++kk)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              top = max(max(top, qf[kk][nt][i] & 0x7FFFu), qf[kk][nt][i] >> 16 & 0x7FFFu);
          top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
          top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
          int e = 0;
          if (top > 0 && top < 0x7F80u) {
            const float v = __uint_as_float(top << 16);
            e = 14 - ilogbf(v);
          }
          // two factors: 2^e alone can leave fp32's range
          const float fa = scalbnf(1.f, e / 2), fb = scalbnf(1.f, e - e / 2);
#pragma unroll
          for (int kk = 0; kk < KK; ++kk)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float x, y;
              widen2(qf[kk][nt][i], x, y, __nv_bfloat16());
              qf[kk][nt][i] = pack2(x * fa * fb, y * fa * fb, __half());
            }
          f = scalbnf(1.f, -e);
        }
        fq[nt][0] = __shfl_sync(0xFFFFFFFFu, f, c4 * 8) * p.scale_log2;
        fq[nt][1] = __shfl_sync(0xFFFFFFFFu, f, c4 * 8 + 4) * p.scale_log2;
      }
    }

    float o[KK][NT][4], ref[NT][2], sum[NT][2];
    float v_ref = 0.f, v_inv = 0.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      ref[nt][0] = ref[nt][1] = kNoScore;
      sum[nt][0] = sum[nt][1] = 0.f;
#pragma unroll
      for (int kk = 0; kk < KK; ++kk)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[kk][nt][i] = 0.f;
    }

#pragma unroll 1
    for (int i = 0; i < steps; ++i) {
      asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
      __syncwarp();
      {
        const int id = next_id;
        next_id = page_id(i + S);
        issue(i + S - 1, id, in_slot);
        if (++in_slot == S) in_slot = 0;
      }
      const uint32_t stage = ring + slot * F::kStage;
      const int key0 = first_key(i);
      const uint32_t valid = *reinterpret_cast<volatile uint32_t*>(&s_valid[warp][slot]);
      if (++slot == S) slot = 0;

      // ---------------------------------------------------- S^T = K Q^T --
      float s[MT][NT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[mt][nt][j] = 0.f;
      // matrices: keys 0-7 and 8-15 of one piece, then of the next
      const int mrow = (lane & 7) + (lane & 8), mpiece = lane >> 4;
#pragma unroll
      for (int kk = 0; kk < (kCoded ? KK / 2 : KK); ++kk) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          uint32_t w[4];
          ldsm4(w, stage + mt * 16 * kRow + place<kRow>(mrow, 2 * kk + mpiece));
          if constexpr (kCoded) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t a[4] = {decode_pair<kFormat>(w[2 * h], 0), decode_pair<kFormat>(w[2 * h + 1], 0),
                                     decode_pair<kFormat>(w[2 * h], 1), decode_pair<kFormat>(w[2 * h + 1], 1)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma16816(s[mt][nt], a, qf[2 * kk + h][nt][0], qf[2 * kk + h][nt][1], C());
            }
          } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816(s[mt][nt], w, qf[kk][nt][0], qf[kk][nt][1], C());
          }
        }
      }

      // -------------------------------------------------------- softmax --
      const uint32_t scales = stage + 2 * F::kHalf + g * 4;
      float vs[MT][2];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float ks[2] = {1.f, 1.f};
        vs[mt][0] = vs[mt][1] = 1.f;
        if constexpr (kCoded) {
          ks[0] = ld_shared_f(scales + mt * 64);
          ks[1] = ld_shared_f(scales + mt * 64 + 32);
          vs[mt][0] = ld_shared_f(scales + 4 * kStep + mt * 64);
          vs[mt][1] = ld_shared_f(scales + 4 * kStep + mt * 64 + 32);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            s[mt][nt][j] = kCoded ? s[mt][nt][j] * fq[nt][j & 1] * ks[j >> 1] : s[mt][nt][j] * fq[nt][j & 1];
      }
      // Steps with keys without a page or beyond the last, or with drafts: what a
      // row does not see is taken out.  Bit 4 (NT mt + nt) + j: seen.
      const bool partial = valid != kAll || key0 + kStep > seq.start;
      uint32_t seen = 0xFFFFFFFFu;
      if (__builtin_expect(partial, 0)) {
        seen = 0;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int spot = mt * 16 + g + (j >> 1) * 8, draft = key0 + spot - seq.start;
              const int r = row0 + nt * 8 + c4 * 2 + (j & 1);
              bool sees = (valid >> spot & 1) && r < all_rows;
              if (sees && draft >= 0) {
                const int t = quotient(r, p.group);
                if (p.mask)
                  sees = (draft >> 5) < p.words && (p.mask[(seq.lo + t) * p.ldm + (draft >> 5)] >> (draft & 31) & 1);
                else
                  sees = draft <= t;
              }
              if (sees)
                seen |= 1u << (4 * (NT * mt + nt) + j);
              else
                s[mt][nt][j] = -INFINITY;
            }
      }
      if constexpr (kCoded) {
        // scales that are no finite number do not enter the reference: they make
        // p NaN for the rows that see the key, and only for those
        float top = 0.f;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!(fabsf(vs[mt][h]) < INFINITY)) vs[mt][h] = __uint_as_float(0x7FC00000u);
            top = fmaxf(top, fabsf(vs[mt][h]));  // the finite ones
          }
        if (__any_sync(0xFFFFFFFFu, top > 2.f * v_ref)) {
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
          // a power of two not above the largest one: its reciprocal is exact
          top = fmaxf(__uint_as_float(__float_as_uint(top) & 0x7F800000u), fmaxf(v_ref, 1.17549435e-38f));
          const float down = v_ref / top;
          const int rise = v_ref > 0.f ? exponent_of(top) - exponent_of(v_ref) : 0;
          v_ref = top;
          v_inv = 1.f / top;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i2 = 0; i2 < 2; ++i2) {
              float its_down = down;
              if (partial && rise > 0) {
                // not every row sees the key: the rows' references go down instead, and
                // come up again below for those that do
                float most = sum[nt][i2];
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, x));
                const int low = lowered(most, rise);
                ref[nt][i2] -= static_cast<float>(low);
                sum[nt][i2] *= power_of_two(low);
                its_down *= power_of_two(low);
              }
#pragma unroll
              for (int kk = 0; kk < KK; ++kk) {
                o[kk][nt][i2] *= its_down;
                o[kk][nt][2 + i2] *= its_down;
              }
            }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          vs[mt][0] *= v_inv;
          vs[mt][1] *= v_inv;
        }
      }
      bool beyond = false;
      float tops[NT][2];
      const auto find_tops = [&](auto by_scale) {
        float lv[MT][2];  // logarithms of V's scales
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) lv[mt][h] = by_scale ? fmaxf(__log2f(fabsf(vs[mt][h])), -kRoom) : 0.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i2 = 0; i2 < 2; ++i2) {
            tops[nt][i2] = -INFINITY;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                tops[nt][i2] = fmaxf(tops[nt][i2], by_scale ? s[mt][nt][2 * h + i2] + lv[mt][h] : s[mt][nt][2 * h + i2]);
          }
      };
      if (kCoded && __builtin_expect(partial, 0))
        find_tops(std::true_type());
      else
        find_tops(std::false_type());
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i2 = 0; i2 < 2; ++i2) beyond |= tops[nt][i2] > ref[nt][i2] + kSlack;
      if (__any_sync(0xFFFFFFFFu, beyond)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i2 = 0; i2 < 2; ++i2) {
            float top = tops[nt][i2];
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
            top = fmaxf(top, ref[nt][i2]);
            const float down = exp2_fast(ref[nt][i2] - top);
            ref[nt][i2] = top;
            sum[nt][i2] *= down;
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
              o[kk][nt][i2] *= down;
              o[kk][nt][2 + i2] *= down;
            }
          }
      }
      // 16-bit caches: what the rounding leaves is a second factor (no time: 32 tokens
      // over up to 16384 34.9 us with it, 35.2 without; the error against 64 bits is
      // the output's own rounding then).  With 8-bit caches, where decoding already
      // takes the issue slots, it would cost 32 rows 11 % (32 x 8000, 8 heads 123 us,
      // 137 with it), 16 rows 5 to 11 and 8 rows 1 to 3, and p stays one fp16 number:
      // error 0.0003 in fp16 for 0.0002, in bf16 no more than the output's rounding.
      uint32_t pb[MT][NT][2], rest[MT][NT][2];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float e[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) e[j] = exp2_fast(s[mt][nt][j] - (ref[nt][j & 1] - kLift));
          sum[nt][0] += e[0] + e[2];
          sum[nt][1] += e[1] + e[3];
          if constexpr (kCoded) {
#pragma unroll
            for (int j = 0; j < 4; ++j) e[j] *= vs[mt][j >> 1];
            if (__builtin_expect(partial, 0)) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (!(seen >> (4 * (NT * mt + nt) + j) & 1)) e[j] = 0.f;
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t w = pack2(e[2 * h], e[2 * h + 1], C());
            pb[mt][nt][h] = transpose8(w);
            if constexpr (kRest) {
              float x, y;
              widen2(w, x, y, C());
              rest[mt][nt][h] = transpose8(pack2(e[2 * h] - x, e[2 * h + 1] - y, C()));
            }
          }
        }

      // -------------------------------------------------- O^T += V^T P^T --
      const int trow = (lane & 7) + (kCoded ? lane & 8 : lane >> 4 << 3);
      const int tpiece = kCoded ? lane >> 4 : lane >> 3 & 1;
      const auto v_frag = [&](int mt, int kk, uint32_t (&a)[4], uint32_t (&a2)[4]) {
        // 8 bit: dimensions 32 kk .. + 31 as two fragments; 16 bit: 16 kk .. + 15
        uint32_t w[4];
        ldsm4t(w, stage + F::kHalf + mt * 16 * kRow + place<kRow>(trow, 2 * kk + tpiece));
        if constexpr (kCoded) {
          decode_cross<kFormat>(w[0], a[0], a[1]);
          decode_cross<kFormat>(w[1], a[2], a[3]);
          decode_cross<kFormat>(w[2], a2[0], a2[1]);
          decode_cross<kFormat>(w[3], a2[2], a2[3]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) a[j] = w[j];
        }
      };
      constexpr int kSteps = kCoded ? KK / 2 : KK;
      uint32_t odd = 0;
      if (kFormat != PROJ_KV_INT8 && __builtin_expect(partial, 0)) {
#pragma unroll 1
        for (int kk = 0; kk < kSteps; ++kk)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            uint32_t a[4], a2[4] = {0u, 0u, 0u, 0u};
            v_frag(mt, kk, a, a2);
#pragma unroll
            for (int j = 0; j < 4; ++j) odd |= odd_pair(a[j], C()) || odd_pair(a2[j], C());
          }
        odd = __any_sync(0xFFFFFFFFu, odd);
      }
      if (__builtin_expect(!odd, 1)) {
#pragma unroll
        for (int kk = 0; kk < kSteps; ++kk)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            uint32_t a[4], a2[4];
            v_frag(mt, kk, a, a2);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if constexpr (kCoded) {
                mma16816(o[2 * kk][nt], a, pb[mt][nt][0], pb[mt][nt][1], C());
                mma16816(o[2 * kk + 1][nt], a2, pb[mt][nt][0], pb[mt][nt][1], C());
              } else {
                mma16816(o[kk][nt], a, pb[mt][nt][0], pb[mt][nt][1], C());
                if constexpr (kRest) mma16816(o[kk][nt], a, rest[mt][nt][0], rest[mt][nt][1], C());
              }
            }
          }
      } else {
        // A value of V in this step is no finite number, and 0 times it is NaN:
        // key by key, added where the row sees the key.
#pragma unroll
        for (int kk = 0; kk < kSteps; ++kk)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            uint32_t a[2][4];
            v_frag(mt, kk, a[0], a[1]);
#pragma unroll 1
            for (int key = 0; key < 16; ++key) {
              const uint32_t sees = __shfl_sync(0xFFFFFFFFu, seen, (key & 7) * 4 + c4) >> (4 * NT * mt + (key & 8 ? 2 : 0));
              const bool mine = (key & 7) >> 1 == c4;
              const uint32_t half = mine ? (key & 1 ? 0xFFFF0000u : 0xFFFFu) : 0u;
              const uint32_t lo = key & 8 ? 0u : half, hi = key & 8 ? half : 0u;
#pragma unroll
              for (int h = 0; h < (kCoded ? 2 : 1); ++h) {
                const uint32_t one[4] = {a[h][0] & lo, a[h][1] & lo, a[h][2] & hi, a[h][3] & hi};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  float d[4] = {0.f, 0.f, 0.f, 0.f};
                  mma16816(d, one, pb[mt][nt][0] & lo, pb[mt][nt][1] & hi, C());
                  if constexpr (kRest) mma16816(d, one, rest[mt][nt][0] & lo, rest[mt][nt][1] & hi, C());
#pragma unroll
                  for (int j = 0; j < 4; ++j)
                    if (sees >> (4 * nt + (j & 1)) & 1) o[kCoded ? 2 * kk + h : kk][nt][j] += d[j];
                }
              }
            }
          }
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");

    // --------------------------------------------- the warps' sums joined --
    // A thread has kOuts rows, four columns of each; their gate is read meanwhile
    // (by a warp that has all rows, one at a time: other warps are at work).
    const bool whole = u0 == 0 && u1 == seq.units;
    constexpr int kTeamThreads = 32 * kTeam;
    constexpr int kOuts = F::kRows * (D / 4) / kTeamThreads > 0 ? F::kRows * (D / 4) / kTeamThreads : 1;
    const int quad = tid % (D / 4);
    const auto out_row = [&](int n) { return tid / (D / 4) + n * (kTeamThreads / (D / 4)); };
    Vec<T, 4> gate[kSolo ? 1 : kOuts][1] = {};
    const auto read_gate = [&](int n, Vec<T, 4>& to) {
      const int r = row0 + out_row(n), t = quotient(r, p.group);
      if (whole && p.gate && r < all_rows && out_row(n) < F::kRows)
        to = load_vec<T, 4>(reinterpret_cast<const T*>(p.gate + static_cast<int64_t>(seq.lo + t) * p.ldg) +
                            (head * G + r - t * G) * D + quad * 4);
    };
    if constexpr (!kSolo) {
#pragma unroll
      for (int n = 0; n < kOuts; ++n) read_gate(n, gate[n][0]);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) sum[nt][i] += __shfl_xor_sync(0xFFFFFFFFu, sum[nt][i], x);
    if (!told && tid == kTeamThreads - 1) p.splits[worker] = split_of(p, share, worker);
    told = true;
    team_sync();  // every warp is done with its ring
    const float up = kCoded ? v_ref : 1.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = nt * 8 + c4 * 2 + i;
        if (g == 0) {
          s_ml[(member * F::kRows + r) * 2] = ref[nt][i] - kLift;
          s_ml[(member * F::kRows + r) * 2 + 1] = sum[nt][i];
        }
        float* to = merge + (member * F::kRows + r) * F::kPitch;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
          if constexpr (kCoded) {
            *reinterpret_cast<float2*>(to + kk * 16 + 2 * g) =
                make_float2(o[kk][nt][i] * up, o[kk][nt][2 + i] * up);
          } else {
            to[kk * 16 + g] = o[kk][nt][i];
            to[kk * 16 + 8 + g] = o[kk][nt][2 + i];
          }
        }
      }
    }
    team_sync();
#pragma unroll(kSolo ? 1 : kOuts)
    for (int n = 0; n < kOuts; ++n) {
      const int r = out_row(n);
      if (row0 + r >= all_rows || r >= F::kRows) continue;
      Vec<T, 4>(&its_gate)[1] = gate[kSolo ? 0 : n];
      if constexpr (kSolo) read_gate(n, its_gate[0]);
      float top = s_ml[r * 2];
#pragma unroll
      for (int w = 1; w < kTeam; ++w) top = fmaxf(top, s_ml[(w * F::kRows + r) * 2]);
      float l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kTeam; ++w) {
        const float f = exp2_fast(s_ml[(w * F::kRows + r) * 2] - top);
        l += f * s_ml[(w * F::kRows + r) * 2 + 1];
        const float4 v = *reinterpret_cast<const float4*>(merge + (w * F::kRows + r) * F::kPitch + quad * 4);
        acc[0] += f * v.x;
        acc[1] += f * v.y;
        acc[2] += f * v.z;
        acc[3] += f * v.w;
      }
      if (whole) {
        const int t = quotient(row0 + r, p.group);
        const int j = head * G + row0 + r - t * G;
        write_out<T>(p, static_cast<int64_t>(seq.lo + t), j * D + quad * 4, acc, l, its_gate);
        if (p.lse && quad == 0) p.lse[static_cast<int64_t>(seq.lo + t) * p.heads + j] = lse_of(top, l);
      } else {
        const int part = 2 * worker + (u0 == 0 ? 1 : 0);
        float* to = p.part_o + (static_cast<int64_t>(part) * F::kRows + r) * D + quad * 4;
        *reinterpret_cast<float4*>(to) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        if (quad == 0)
          *reinterpret_cast<float2*>(p.part_ml + (static_cast<int64_t>(part) * F::kRows + r) * 2) =
              make_float2(top, l);
      }
    }
    team_sync();  // the ring is free again
    at += u1 - u0;
  }
}

// The join.  CTA (x, y) has the x-th item that was split, rows y, y + gridDim.y,
// ... in sets of threads that span a row.  Few rows in all (`spread`): a CTA's sets
// share a row's partial results, each relative to a running maximum, and meet in
// shared memory.  Many: each set takes a row.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) attn_join_kernel(const AttnParams p) {
  constexpr int kLanes = D / 4, kSets = kThreads / kLanes;
  __shared__ float s_o[kSets][D], s_ml[kSets][2];
  __shared__ Split s_split;
  __shared__ int s_count[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  touch(p);
  griddep_launch_dependents();
  griddep_wait();
  // the item: the x-th that a CTA left
  if (threadIdx.x == 0) s_split.rows = 0;
  int before = 0;
  for (int c = 0; c < p.ctas; c += kThreads) {
    const int at = c + static_cast<int>(threadIdx.x);
    const Split mine = at < p.ctas ? p.splits[at] : Split{};
    const uint32_t some = __ballot_sync(0xFFFFFFFFu, mine.rows > 0);
    if (lane == 0) s_count[warp] = __popc(some);
    __syncthreads();
    int rank = before + __popc(some & ((1u << lane) - 1u));
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) rank += s_count[w];
      before += s_count[w];
    }
    if (mine.rows > 0 && rank == static_cast<int>(blockIdx.x)) s_split = mine;
    __syncthreads();
  }
  const Split it = s_split;
  if (it.rows == 0) return;
  const int G = static_cast<int>(p.group.d);
  const int set = threadIdx.x / kLanes, quad = threadIdx.x % kLanes;
  const bool alone = !p.spread;  // a set has a row to itself: then no barrier below is reached
  const int y0 = alone ? blockIdx.y * kSets + set : blockIdx.y, dy = alone ? gridDim.y * kSets : gridDim.y;
  for (int r = y0; r < it.rows; r += dy) {
    float top = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    const int t = quotient(it.row0 + r, p.group);
    const int j = it.head * G + it.row0 + r - t * G;
    Vec<T, 4> gate[1] = {};
    if (p.gate) gate[0] = load_vec<T, 4>(reinterpret_cast<const T*>(p.gate + static_cast<int64_t>(it.lo + t) * p.ldg) + j * D + quad * 4);
#pragma unroll 8
    for (int c = it.first + (alone ? 0 : set); c <= it.last; c += alone ? 1 : kSets) {
      const int64_t slot = 2ll * c + (c == it.first ? 1 : 0);
      const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + (slot * p.tile_rows + r) * 2);
      const float4 v = *reinterpret_cast<const float4*>(p.part_o + (slot * p.tile_rows + r) * D + quad * 4);
      const float now = fmaxf(top, ml.x);
      const float a = exp2_fast(top - now), f = exp2_fast(ml.x - now);
      top = now;
      l = l * a + ml.y * f;
      acc[0] = acc[0] * a + v.x * f;
      acc[1] = acc[1] * a + v.y * f;
      acc[2] = acc[2] * a + v.z * f;
      acc[3] = acc[3] * a + v.w * f;
    }
    if (!alone) {
      *reinterpret_cast<float4*>(&s_o[set][quad * 4]) = make_float4(acc[0], acc[1], acc[2], acc[3]);
      if (quad == 0) {
        s_ml[set][0] = top;
        s_ml[set][1] = l;
      }
      __syncthreads();
      if (set == 0) {
        top = s_ml[0][0];
#pragma unroll
        for (int i = 1; i < kSets; ++i) top = fmaxf(top, s_ml[i][0]);
        l = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = 0.f;
#pragma unroll
        for (int i = 0; i < kSets; ++i) {
          const float f = exp2_fast(s_ml[i][0] - top);
          l += f * s_ml[i][1];
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[j] += f * s_o[i][quad * 4 + j];
        }
      }
      __syncthreads();
    }
    if (alone || set == 0) {
      write_out<T>(p, static_cast<int64_t>(it.lo + t), j * D + quad * 4, acc, l, gate);
      if (p.lse && quad == 0) p.lse[static_cast<int64_t>(it.lo + t) * p.heads + j] = lse_of(top, l);
    }
  }
}

// ------------------------------------------------------------------- host --

template <typename P>
cudaError_t launch(void (*kernel)(P), dim3 grid, size_t smem, const P& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename T, int kFormat, int D, int NT, bool kSolo>
cudaError_t stream_launch(const AttnParams& p, cudaStream_t s) {
  using F = Stream<kFormat, D, NT>;
  const auto kernel = attn_stream_kernel<T, kFormat, D, NT, kSolo>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), F::kSmem, done);
  return e == cudaSuccess ? launch(kernel, dim3(p.ctas / (kSolo ? kWarps : 1)), F::kSmem, p, s) : e;
}

template <typename T, int kFormat, int D>
cudaError_t stream_rows(const AttnParams& p, cudaStream_t s) {
  if (p.solo)
    return p.tile_rows == 8 ? stream_launch<T, kFormat, D, 1, true>(p, s) : stream_launch<T, kFormat, D, 2, true>(p, s);
  return p.tile_rows == 8 ? stream_launch<T, kFormat, D, 1, false>(p, s) : stream_launch<T, kFormat, D, 2, false>(p, s);
}

template <typename T, int D>
cudaError_t stream_format(int format, const AttnParams& p, cudaStream_t s) {
  return format == PROJ_KV_ROWS   ? stream_rows<T, PROJ_KV_ROWS, D>(p, s)
         : format == PROJ_KV_E4M3 ? stream_rows<T, PROJ_KV_E4M3, D>(p, s)
                                  : stream_rows<T, PROJ_KV_INT8, D>(p, s);
}

struct Plan {
  bool tc, solo;
  int64_t rows;  // of a sequence and a head of keys and values, on average
  int tile_rows, unit, sms, ctas, min_units;  // ctas: shares
  int64_t bytes;
};

// Which kernel, and rows of an item.  Numbers of rows and lengths are known on the
// device only: the plan goes by the rows that a sequence and a head of keys and
// values have on average, and by the table's width.
//
// Up to 16 rows are streamed, in items of 8 or 16.  Up to 32 too, in two items, of
// which the second reads the cache from L2; not so 16-bit entries of 128 dimensions
// in a cache of twice the L2 (2^19 tokens and heads).  More than 32 are streamed
// while there is little to do: an item of 16 rows costs the streaming kernel some
// 0.13 us by itself and 1 us for every 1100 units, while a tcgen05 call is not under
// 15 to 30 us (128 units a CTA, with 64 for each item, is where they meet).
// D = 128, eight query heads on each, streamed against tcgen05, us:
//                                        e4m3      16-bit
//    16 sequences x 32768 keys, 16 rows   32  54    39  45
//    32 x  2000, 8 heads,       32 rows   54  88    60  68
//    32 x  8000, 8 heads,       32 rows  121 183   200 134  (16-bit: tcgen05)
//     1 x  4096,                64 rows   15  20    13  17
//    16 x  4096,                64 rows   25  31    24  29
//    16 x 32768,                64 rows   69  60     -   -  (tcgen05)
//    32 x  4000,                64 rows   41  36    38  32  (tcgen05)
//   256 x   300,                64 rows   59  46    58  40  (tcgen05)
//     8 x  1900,               256 rows   33  34    28  30
//     1 x  1000,               512 rows   16  30    14  26
//
// More than three items to two SMs are streamed by warps with a share each: an
// item's ends (its lengths, first pages, queries, and the sums that a CTA's warps
// join) then pass beside other warps' items.  By CTAs against by warps, us:
//    16 x 2000, 8 heads,  8 rows   e4m3  24  30   16-bit  26  33  (by CTAs)
//    32 x 2000, 8 heads, 16 rows         57  40           52  46
//    64 x  300, 8 heads,  8 rows         43  28           38  29
//    64 x 4000, 8 heads,  8 rows         86  68          116 112
//    64 x 4000, 8 heads, 16 rows        121  80          129 122
//   256 x 1000, 8 heads,  8 rows        132  98          136 130
//   256 x  300, 1 head,  16 rows         37  45           30  41  (warps all the same)
//   256 x 2000, 1 head,  16 rows         50  40           48  46
// So of many short sequences with one head the rule takes the slower form.  (Both
// tables are of before V's scales had a reference by row where keys are masked: over
// 8-bit caches the streaming kernel takes 1 to 3 % more since, tcgen05 0 to 1.)
// A share has at least 256 keys of a CTA: a step for each of the streaming kernel's
// warps (one sequence of 8192 keys: 9.0 us; with 128 keys 9.4, with 512 9.2), four
// tiles of the tcgen05 kernel (2: the same or 0.3 us slower, 8: 1-3); and 128 of a
// warp.
const char* make_plan(const proj_kv_cache* cache, int64_t m, int64_t heads, Plan* plan,
                      int* status) {
  if (const char* why = refuse_cache(cache, status)) return why;
  *status = PROJ_EINVAL;
  if (m < 0) return "m < 0";
  if (heads < 1 || heads % cache->heads) return "heads is no multiple of the cache's";
  *status = PROJ_EUNSUPPORTED;
  if (heads > 1024) return "more than 1024 heads";
  if (m > (int64_t{1} << 20)) return "m > 2^20";
  *status = PROJ_OK;
  const int64_t rows = cache->sequences
                           ? (m + cache->sequences - 1) / cache->sequences * (heads / cache->heads)
                           : 1;
  int sms = 0, dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
    sms = 152;
  // the streaming kernel's items and, at most, their units
  const int64_t items = (rows + 15) / 16 * cache->sequences * cache->heads;
  const int64_t capacity = cache->width * cache->page;
  const int64_t units = items * ((capacity + kUnit - 1) / kUnit);
  const bool wide = cache->format == PROJ_KV_ROWS && cache->D == 128;
  plan->rows = rows;
  if (rows > 32)
    plan->tc = units + 64 * items > 128 * static_cast<int64_t>(sms);
  else
    plan->tc = rows > 16 && wide && cache->sequences * cache->heads * capacity > (int64_t{1} << 19);
  plan->unit = plan->tc ? kAttnTcUnit : kUnit;
  plan->tile_rows = plan->tc ? kAttnTcRows : rows <= 8 ? 8 : 16;
  const int64_t parts = (rows + plan->tile_rows - 1) / plan->tile_rows * cache->sequences * cache->heads;
  plan->solo = !plan->tc && 2 * parts > 3 * static_cast<int64_t>(sms);
  plan->min_units = plan->tc || plan->solo ? 4 : kWarps;
  plan->sms = sms;
  plan->ctas = plan->solo ? kWarps * sms : sms;
  // never less for more rows: the most shares there are, whatever the kernel
  plan->bytes = int64_t{2} * plan->ctas * plan->tile_rows * (cache->D + 2) * 4 +
                int64_t{kWarps} * sms * static_cast<int64_t>(sizeof(Split));
  return nullptr;
}

}  // namespace
}  // namespace proj

using namespace proj;

extern "C" int64_t proj_attn_workspace(const proj_kv_cache* cache, int64_t m, int64_t heads) {
  Plan plan;
  int status = PROJ_OK;
  if (const char* why = make_plan(cache, m, heads, &plan, &status)) {
    kv_refuse(status, "proj_attn_workspace", why);
    return -1;
  }
  return plan.bytes;
}

extern "C" int proj_attn(const proj_attn_args* args, proj_stream stream) {
  const char* const call = "proj_attn";
  if (!args) return kv_refuse(PROJ_EINVAL, call, "args is NULL");
  const proj_attn_args& a = *args;
  Plan plan;
  int status = PROJ_OK;
  if (const char* why = make_plan(a.cache, a.m, a.heads, &plan, &status)) return kv_refuse(status, call, why);
  const proj_kv_cache& c = *a.cache;
  const int64_t width = a.heads * c.D;
  if (a.gate_act != PROJ_GATE_LINEAR && a.gate_act != PROJ_GATE_SIGMOID)
    return kv_refuse(PROJ_EINVAL, call, "unknown gate_act");
  const float scale_log2 = static_cast<float>(a.scale * 1.4426950408889634);
  if (!std::isfinite(scale_log2))
    return kv_refuse(PROJ_EINVAL, call, "scale, or scale log2(e), is no finite number");
  if (a.m > 0 && c.sequences > 0 && (!a.q || !a.out || !a.offsets || !a.start))
    return kv_refuse(PROJ_EINVAL, call, "q, out, offsets or start is NULL");
  if (a.ldq < width || a.ldo < width || (a.gate && a.ldg < width))
    return kv_refuse(PROJ_EINVAL, call, "a row stride is below heads D");
  if (a.mask && (a.words < 1 || a.ldm < a.words))
    return kv_refuse(PROJ_EINVAL, call, "words < 1, or ldm below words");
  if ((a.out == a.q && a.ldo != a.ldq) || (a.gate && a.out == a.gate && a.ldo != a.ldg))
    return kv_refuse(PROJ_EINVAL, call, "out is q or the gate, but with another stride");
  if (a.mask && a.words > 1024) return kv_refuse(PROJ_EUNSUPPORTED, call, "words > 1024");
  const int64_t most = int64_t{1} << 31;
  if (a.ldq >= most || a.ldo >= most || a.ldg >= most || a.ldm >= most)
    return kv_refuse(PROJ_EUNSUPPORTED, call, "a row stride of 2^31 or more");
  if (!kv_aligned(a.q, 16) || !kv_aligned(a.out, 16) || !kv_aligned(a.gate, 16) || a.ldq % 8 ||
      a.ldo % 8 || (a.gate && a.ldg % 8))
    return kv_refuse(PROJ_EALIGN, call, "rows of q, out or the gate do not start on 16 bytes");
  if (!kv_aligned(a.offsets, 4) || !kv_aligned(a.start, 4) || !kv_aligned(a.mask, 4) ||
      !kv_aligned(a.lse, 4))
    return kv_refuse(PROJ_EALIGN, call, "offsets, start, mask or lse is not aligned to 4 bytes");
  if (a.m == 0 || c.sequences == 0) return PROJ_OK;
  if (!a.workspace || a.workspace_bytes < plan.bytes)
    return kv_refuse(PROJ_EINVAL, call, "workspace is NULL or smaller than proj_attn_workspace");
  if (!kv_aligned(a.workspace, 16)) return kv_refuse(PROJ_EALIGN, call, "workspace is not aligned to 16 bytes");
  AttnParams p = {};
  p.c = device_cache(c);
  p.q = static_cast<const uint8_t*>(a.q);
  p.ldq = a.ldq * 2;
  p.offsets = a.offsets;
  p.start = a.start;
  p.mask = a.mask;
  p.ldm = a.ldm;
  p.words = static_cast<int>(a.words);
  p.scale_log2 = scale_log2;
  p.gate = static_cast<const uint8_t*>(a.gate);
  p.ldg = a.ldg * 2;
  p.sigmoid = a.gate_act == PROJ_GATE_SIGMOID;
  p.out = static_cast<uint8_t*>(a.out);
  p.ldo = a.ldo * 2;
  p.lse = a.lse;
  p.m = static_cast<int>(a.m);
  p.heads = static_cast<int>(a.heads);
  p.D = static_cast<int>(c.D);
  p.group = make_divisor(static_cast<uint32_t>(a.heads / c.heads));
  p.tile_rows = plan.tile_rows;
  p.unit = plan.unit;
  p.ctas = plan.ctas;
  p.solo = plan.solo;
  while ((1 << p.min_shift) < plan.min_units) ++p.min_shift;
  while ((1 << p.tile_shift) < p.tile_rows) ++p.tile_shift;
  while ((1 << p.unit_shift) < p.unit) ++p.unit_shift;
  void* status_word = nullptr;
  cudaError_t e = cudaGetSymbolAddress(&status_word, g_attn_status);
  if (e != cudaSuccess) return record_cuda(e, call);
  p.status = static_cast<uint32_t*>(status_word);
  p.splits = static_cast<Split*>(a.workspace);
  p.part_o = reinterpret_cast<float*>(p.splits + kWarps * plan.sms);
  p.part_ml = p.part_o + int64_t{2} * plan.ctas * plan.tile_rows * c.D;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (plan.tc)
    e = attn_tc_launch(p, c.dtype, c.format, s);
  else if (c.dtype == PROJ_BF16)
    e = c.D == 64 ? stream_format<__nv_bfloat16, 64>(c.format, p, s)
                  : stream_format<__nv_bfloat16, 128>(c.format, p, s);
  else
    e = c.D == 64 ? stream_format<__half, 64>(c.format, p, s) : stream_format<__half, 128>(c.format, p, s);
  if (e != cudaSuccess) return record_cuda(e, call);
  // No more items than this, and as many CTAs to one as its rows keep at work.
  const int64_t rows = std::min<int64_t>(plan.tile_rows, plan.rows);
  const int64_t items = (a.m * (a.heads / c.heads) / plan.tile_rows + c.sequences) * c.heads;
  const int sets = kThreads / (static_cast<int>(c.D) / 4);
  const int64_t x = std::min<int64_t>(items, plan.ctas);
  // 16 CTAs an SM (16 items of 8 rows in 10 parts each: the call
  // 24.7 us with a set a row, 19.9 with a CTA)
  p.spread = x * rows <= 16 * plan.sms;
  const int64_t y = p.spread ? rows : (rows + sets - 1) / sets;
  const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>(std::max<int64_t>(1, y)));
  if (c.dtype == PROJ_BF16)
    e = c.D == 64 ? launch(attn_join_kernel<__nv_bfloat16, 64>, grid, 0, p, s)
                  : launch(attn_join_kernel<__nv_bfloat16, 128>, grid, 0, p, s);
  else
    e = c.D == 64 ? launch(attn_join_kernel<__half, 64>, grid, 0, p, s)
                  : launch(attn_join_kernel<__half, 128>, grid, 0, p, s);
  return e == cudaSuccess ? PROJ_OK : record_cuda(e, call);
}

extern "C" int proj_attn_describe(const proj_kv_cache* cache, int64_t m, int64_t heads, char* buf,
                                  size_t cap) {
  const char* const call = "proj_attn_describe";
  Plan plan;
  int status = PROJ_OK;
  if (const char* why = make_plan(cache, m, heads, &plan, &status)) return kv_refuse(status, call, why);
  if (!buf || cap == 0) return kv_refuse(PROJ_EINVAL, call, "buf is NULL or cap 0");
  std::snprintf(buf, cap, "attn %s, items of %d rows, units of %d keys, up to %d %s, join",
                plan.tc ? "tcgen05" : "stream", plan.tile_rows, plan.unit, plan.ctas, plan.solo ? "warps" : "CTAs");
  return PROJ_OK;
}

extern "C" int proj_attn_device_status(proj_stream stream, uint32_t* code) {
  const char* const call = "proj_attn_device_status";
  void* at = nullptr;
  uint32_t word = 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaGetSymbolAddress(&at, g_attn_status);
  if (e == cudaSuccess) e = cudaMemcpyAsync(&word, at, 4, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(at, 0, 4, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return record_cuda(e, call);
  if (code) *code = word;
  return word ? kv_refuse(PROJ_EDEVICE, call, "a kernel recorded a fault") : PROJ_OK;
}
