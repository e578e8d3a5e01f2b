// attn_tc.cu -- attention of drafted tokens over the cache on tcgen05, for
// items of many rows (a group's heads times a sequence's drafts above 32; 17 to 32 of
// 16-bit entries too, attn.cu's make_plan) over long caches.
//
// Rows are the M side of both products, a row in each of 128 lanes of tensor
// memory; a tile is 64 keys:
//   S [128 x 64] = Q K^T     A = Q, held in tensor memory for an item
//   O [128 x D] += P V       A = P, written to tensor memory by the softmax
// K and V are the B operands in shared memory, both as [key][64 dimensions]
// rows of 128 bytes in the 128-byte swizzle: K-major for the first product,
// N-major for the second, so V needs no transposition.
//
// Roles (20 warps): 0-3 and 4-7 are two softmax groups, a thread a row, which
// take the tiles in turn and have an S, a P and an O each -- so one group's
// exponentials run beside the other's products, and neither waits for the
// other's sums; they meet at the item's end.  8-15 bring the cache by 16-byte
// asynchronous copies, in teams that take the tiles in turn: 16-bit entries to their
// stage, 8-bit codes to a ring of their own, from where the thread that copied them
// takes them to their stage as fp16, which holds them exactly.  16 and 19 issue the
// MMAs.  17 walks the CTA's share: it looks up pages, and hands each tile's addresses
// to the loading warps and each segment to the others, so that no other warp divides
// or waits for a table.  18 brings the scales.
//
// Softmax as in the streaming kernel: a reference per row that moves only when
// a score is well above it, whereupon O is scaled in tensor memory;
// probabilities are fp16 (bf16 caches: bf16, since V may leave fp16's range).  A
// second number for what that rounding leaves has no room: with 128 dimensions Q, two
// S, two P and two O fill all 512 columns.  (Error against 64 bits 0.0003 in fp16,
// where the output's own rounding is 0.0002; 0.0017 in bf16, as that rounding alone;
// 0.0023 over a bf16 cache.)  Scales of K multiply the fp32
// score; those of V the probability, relative to a power-of-two reference that
// warp 18 keeps (and that tiles of drafts turn into one of each row's own: attn.h,
// kRoom; by the largest scale and the largest score that the row sees of 32 keys).
//
// What bounds it is none of the units (issue slots 39-44 % used, tensor pipe 20-31 %,
// HBM a tenth to three quarters) but how long a tile's chain of hand-offs takes a warp:
// some 3100 cycles in a softmax group, half of that a tile with two groups, where
// HBM would deliver 64 keys of e4m3 in 700.  32 sequences of 8 drafts, 64 heads on
// 8, 16-bit: 140 us (4.9 TB/s); 16 of 8 drafts over up to 32768 keys, 8 heads on 1,
// e4m3: 60 us, of which some 25 are a call's ends (share, pages, queries, sums and
// their join); 32 of up to 64 drafts: 141 us (0.36 PFLOP/s).  What the steps there
// were worth: short loops (five roles share a scheduler's instruction cache; with
// loops unrolled over tiles two thirds of the cycles went to waiting for
// instructions) 103 -> 74 us in the second case, no spills in any loop 82 -> 65,
// teams of loading warps 191 -> 157 in the first, lane halves that share the item's
// end 157 -> 141, the join's CTAs 62 -> 59 in the second.
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "attn.h"
#include "kernels.h"
#include "kv_num.cuh"

namespace proj {
namespace {

constexpr int kSoftWarps = 8, kLoadWarp = 8, kLoadWarps = 8, kMmaWarp = 16, kWalkWarp = 17, kScaleWarp = 18,
              kPvWarp = 19;
constexpr int kThreads = 32 * 20;
// Registers a thread: at launch, and of the three kinds of warpgroups (two of
// softmax, two of loading, one of the others).  Spills cost: beside this much shared
// memory L1 does not hold those of 640 threads.  16-bit and int8 instances have up to
// 16 bytes of them, e4m3's 48 to 64.
constexpr int kRegs = 96, kSoftRegs = 160, kLoadRegs = 48, kOtherRegs = 64;
static_assert(2 * kSoftRegs + 2 * kLoadRegs + kOtherRegs <= 5 * kRegs && 5 * kRegs * 128 <= 65536, "registers");
// The loading warps are teams that take the tiles in turn: what one warp does for a
// tile is a chain of waits, some two tiles' time long, whatever its share.
template <int kFormat>
constexpr int kTeams = kFormat == PROJ_KV_ROWS ? 4 : 2;
constexpr int kKeys = kAttnTcUnit;
constexpr int kTmemCols = 512;
constexpr int kRaw = 4;        // tiles of 8-bit codes in shared memory or on their way there
constexpr int kRawScales = 4;  // of scales
constexpr int kIds = 4;        // of page ids
constexpr int kSlots = 8;      // tiles whose addresses are known
constexpr int kSegments = 4;   // segments that are known

// What the walking warp says of a tile.
struct alignas(16) Tile {
  int64_t at[kKeys], scale[kKeys];  // offsets of entries (-1: no page) and scales
  uint32_t valid[2];
  int kind;  // 0: no more tiles, 1: a tile, + 2: of drafts, + 4: a segment's first
  int pad;
};

// A part of an item.
struct alignas(16) Segment {
  int tiles;  // 0: no more segments
  int b, lo, start, len, head, row0, rows, u0, whole;
  int pad[2];
};

// Beside a stage: scales of K and V, the reference of V's, keys that exist; of
// drafts: keys whose scale of V, and keys of which a value is no finite number.
constexpr int kSide = 640, kVScale = 256, kRef = 512, kValid = 520, kOddScale = 528, kOdd = 576;

template <int kFormat, int D>
struct Tc {
  static constexpr int kHalves = D / 64;            // of 64 dimensions
  static constexpr int kHalf = kKeys * 128;         // bytes
  static constexpr int kOperand = kHalves * kHalf;  // K or V of a tile
  static constexpr int kStage = 2 * kOperand;
  static constexpr bool kCoded = kFormat != PROJ_KV_ROWS;
  static constexpr int kStages = kCoded ? (D == 128 ? 4 : 6) : (D == 128 ? 6 : 8);
  static constexpr int kRawTile = 2 * kKeys * D;  // codes of K and V
  static constexpr int kRawAt = kStages * kStage;
  static constexpr int kSideAt = kRawAt + (kCoded ? kRaw * kRawTile : 0);
  static constexpr int kMl = kSideAt + kStages * kSide;  // float[2][128][3]
  static constexpr int kRawScaleAt = kMl + 2 * 128 * 12;  // float[kRawScales][2][kKeys]
  static constexpr int kSwapAt = kRawScaleAt + (kCoded ? kRawScales * 8 * kKeys : 0);  // float[2][2][16][64]: by group and giving half
  static constexpr int kIdsAt = kSwapAt + 16384;  // int[kIds][kKeys]
  static constexpr int kTiles = kIdsAt + kIds * kKeys * 4;
  static constexpr int kSegs = kTiles + kSlots * static_cast<int>(sizeof(Tile));
  static constexpr int kBarsAt = kSegs + kSegments * static_cast<int>(sizeof(Segment));
  static constexpr int kBars = 2 * kStages + 9 + 2 * kSlots + 2 * kSegments;
  static constexpr int kSmem = 1024 + kBarsAt + kBars * 8 + 16;
  // tensor memory, in columns
  static constexpr int kQ = 0, kS = D / 2, kP = kS + 2 * kKeys, kO = kP + kKeys;
  static_assert(kO + 2 * D <= kTmemCols && kSmem <= 232448, "room");
};

__device__ __forceinline__ void tmem_ld32(uint32_t addr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,"
      "%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// D[tmem] (+)= A[tmem] B[smem], kind::f16.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// B in N-major order: rows of 64 n (128 bytes) for each k, eight rows to a
// swizzle atom of 1024 bytes, atoms along k 1024 bytes apart (stride offset),
// the next 64 n `n_stride` bytes further (leading offset).
__device__ __forceinline__ uint64_t smem_desc_n_major(uint32_t saddr, uint32_t n_stride) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(n_stride >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

// Instruction descriptor as idesc_bf16_f32, with the type (0: fp16, 1: bf16)
// and B's order (bit 16: N-major).
constexpr uint32_t instruction(int bf16, int n_major, int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(bf16) << 7) | (static_cast<uint32_t>(bf16) << 10) |
         (static_cast<uint32_t>(n_major) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(r));
  return r != 0;
}

// Bounded wait; the polls read the clock only now and then.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, uint32_t* status,
                                         uint32_t code) {
  if (mbar_try_wait(bar, parity)) return true;
  uint64_t t0 = 0;
  for (uint32_t n = 1;; ++n) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((n & 255u) == 0) {
      const uint64_t now = globaltimer_ns();
      if (!t0) t0 = now;
      if (now - t0 > kWaitLimitNs) {
        atomicOr(status, code);
        return false;
      }
    }
  }
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copies_sealed() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void st_shared_u4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                             uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ float4 ld_shared_f4(uint32_t addr) {
  const uint4 v = ld_shared_u4(addr);
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                     __uint_as_float(v.w));
}
__device__ __forceinline__ void st_shared_f(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ float ld_shared_f(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ void st_shared_u(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_shared_u(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ void st_shared_byte(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint2 ld_shared_u2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

// A pair of 16-bit numbers with what is no finite number taken out.
template <bool kBf16>
__device__ __forceinline__ uint32_t finite_pair(uint32_t w, uint32_t& odd) {
  constexpr uint32_t e = kBf16 ? 0x7F80u : 0x7C00u;
  if ((w & e) == e) {
    odd = 1;
    w &= 0xFFFF0000u;
  }
  if ((w & (e << 16)) == (e << 16)) {
    odd = 1;
    w &= 0xFFFFu;
  }
  return w;
}

// The CTA's segments in order: parts of items.
struct Walk {
  Share share;
  int64_t at;
  Sequence seq;
  int head, row0, u0, u1, rows;
  __device__ __forceinline__ void begin(const AttnParams& p, const Share& s) {
    share = s;
    at = s.first;
    seq = sequence_at(p, s.b);
  }
  __device__ __forceinline__ bool next(const AttnParams& p) {
    if (at >= share.end) return false;
    for (int64_t u; at >= share.before + (u = units_of(p, seq));) {
      share.before += u;
      if (++share.b >= p.c.sequences) return false;
      seq = sequence_at(p, share.b);
    }
    const int64_t local = at - share.before;
    const int64_t item = item_of(local, seq.units);
    u0 = static_cast<int>(local - item * seq.units);
    u1 = static_cast<int>(min(static_cast<int64_t>(seq.units), u0 + (share.end - at)));
    head = static_cast<int>(item_of(item, seq.tiles));
    row0 = static_cast<int>(item - static_cast<int64_t>(head) * seq.tiles) * kAttnTcRows;
    rows = min(kAttnTcRows, seq.rows * static_cast<int>(p.group.d) - row0);
    at += u1 - u0;
    return true;
  }
};

__device__ __forceinline__ uint64_t low_bits(int n) {
  return n <= 0 ? 0 : n >= 64 ? ~uint64_t{0} : (uint64_t{1} << n) - 1;
}
// What row `token` of a sequence (whose first row is lo) sees of 64 keys, the
// first of which is draft `draft` (below 0: before the drafts).
__device__ __forceinline__ uint64_t seen_of(const AttnParams& p, int lo, int token, int draft) {
  uint64_t own;
  if (p.mask) {
    const uint32_t* row = p.mask + static_cast<int64_t>(lo + token) * p.ldm;
    const int w = draft >> 5, shift = draft & 31;
    uint32_t v[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) v[i] = w + i >= 0 && w + i < p.words ? row[w + i] : 0u;
    own = static_cast<uint64_t>(__funnelshift_r(v[0], v[1], shift)) |
          static_cast<uint64_t>(__funnelshift_r(v[1], v[2], shift)) << 32;
  } else {
    own = low_bits(token - draft + 1);
  }
  return own | low_bits(-draft);
}

// The same of keys that exist (`valid`), and whether one that it sees is noted as
// having a value or a scale that is no finite number.  Not inlined: few tiles are
// asked, and the loop around it is short.
template <int kFormat>
__device__ __noinline__ uint64_t seen_here(const AttnParams& p, int lo, int token, int draft, uint2 valid,
                                           uint32_t odd_scale, uint32_t odd_keys, bool& odd) {
  const uint64_t seen = seen_of(p, lo, token, draft) & (valid.x | static_cast<uint64_t>(valid.y) << 32);
  if (draft + kKeys > 0) {
    if (kFormat != PROJ_KV_ROWS) {
      const uint2 w = ld_shared_u2(odd_scale);
      odd |= (seen & (w.x | static_cast<uint64_t>(w.y) << 32)) != 0;
    }
    if (kFormat != PROJ_KV_INT8) {
#pragma unroll 1
      for (int j = 0; j < kKeys; j += 4) {
        const uint32_t w = ld_shared_u(odd_keys + j);
        if (w == 0) continue;
        const uint32_t here = static_cast<uint32_t>(seen >> j);
        odd |= (w & 0xFFu && here & 1u) || (w & 0xFF00u && here & 2u) ||
               (w & 0xFF0000u && here & 4u) || (w & 0xFF000000u && here & 8u);
      }
    }
  }
  return seen;
}

// The values of V at columns c .. c + 15 that are no finite numbers, of keys that
// the row sees in the segment's tiles of drafts, added to o.  The first of these
// tiles begins with the last keys before the drafts (d < 0), which every row sees.
template <typename T, int kFormat>
__device__ __noinline__ void add_odd(const AttnParams& p, const Segment& seg, int token, int c, float* o) {
  const int d0 = max(seg.start / kKeys, seg.u0) * kKeys - seg.start;
  const int d1 = min(seg.len - seg.start, (seg.u0 + seg.tiles) * kKeys - seg.start);
#pragma unroll 1
  for (int d = d0; d < d1; ++d) {
    bool sees = d < 0;
    if (!sees)
      sees = p.mask ? (d >> 5) < p.words && (p.mask[static_cast<int64_t>(seg.lo + token) * p.ldm + (d >> 5)] >> (d & 31) & 1)
                    : d <= token;
    int id, spot;
    if (!sees || !page_of(p.c, seg.b, seg.start + d, id, spot)) continue;
    const Entry e = entry_at(p.c, id, spot, seg.head);
    const uint8_t* v = p.c.v + e.at;
    const bool fine = kFormat == PROJ_KV_ROWS || fabsf(p.c.v_scale[e.scale]) < INFINITY;
#pragma unroll 1
    for (int j = 0; j < 16; ++j) {
      float x;
      if constexpr (kFormat != PROJ_KV_ROWS)
        x = !fine || (kFormat == PROJ_KV_E4M3 && (v[c + j] & 0x7F) == 0x7F) ? __uint_as_float(0x7FC00000u) : 0.f;
      else
        x = to_f32(reinterpret_cast<const T*>(v)[c + j]);
      if (!(fabsf(x) < INFINITY)) o[j] += x;
    }
  }
}

template <typename T, int kFormat, int D>
__global__ void __launch_bounds__(kThreads, 1) attn_tc_kernel(const __grid_constant__ AttnParams p) {
  using F = Tc<kFormat, D>;
  constexpr bool kCoded = kFormat != PROJ_KV_ROWS;
  using C = std::conditional_t<kCoded, __half, T>;
  constexpr bool kBf16 = std::is_same_v<C, __nv_bfloat16>;
  constexpr int NS = F::kStages;
  constexpr int kTeam = kLoadWarps / kTeams<kFormat>;  // warps
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + F::kBarsAt + F::kBars * 8);
  const uint32_t base = smem_u32(smem);
  const uint32_t full = base + F::kBarsAt, empty = full + 8 * NS;
  const uint32_t s_full = empty + 8 * NS, s_free = s_full + 16, p_full = s_free + 16;
  const uint32_t o_done = p_full + 16, q_full = o_done + 16;
  const uint32_t t_full = q_full + 8, t_empty = t_full + 8 * kSlots;
  const uint32_t g_full = t_empty + 8 * kSlots, g_empty = g_full + 8 * kSegments;
  Tile* const s_tiles = reinterpret_cast<Tile*>(smem + F::kTiles);
  Segment* const s_segs = reinterpret_cast<Segment*>(smem + F::kSegs);
  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(full + 8 * s, kTeam + 1);
      mbar_init(empty + 8 * s, 1);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(s_full + 8 * g, 1);
      mbar_init(s_free + 8 * g, 4);
      mbar_init(p_full + 8 * g, 4);
      mbar_init(o_done + 8 * g, 1);
    }
    mbar_init(q_full, kSoftWarps);
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(t_full + 8 * s, 1);
      mbar_init(t_empty + 8 * s, kTeam + 1);
    }
    for (int s = 0; s < kSegments; ++s) {
      mbar_init(g_full + 8 * s, 1);
      mbar_init(g_empty + 8 * s, kSoftWarps + 2);
    }
    fence_mbar_init();
  }
  touch(p);
  // Tensor memory is taken when the kernel before has completed (it might hold
  // some), and the next one may start once it is taken here.
  griddep_wait();
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_launch_dependents();

  // Only the walking warp looks for the CTA's share; the others learn of it from
  // the segments and tiles that it names.
  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kMmaWarp || warp == kPvWarp) {
      // --------------------------------------------------------------- MMA
      // One warp each for the two products, so that neither waits for what the other
      // waits for.
      const bool one = elect_one(), first = warp == kMmaWarp;
      constexpr uint32_t kIdQk = instruction(kBf16, 0, 128, kKeys), kIdPv = instruction(kBf16, 1, 128, D);
      bool ok = true;
      int stage = 0;
      uint32_t phase = 0;
      uint32_t turn[2] = {0u, 0u};  // tiles that each group has had
      for (int n = 0;; ++n) {
        const int seg = n % kSegments;
        ok = ok && wait_bar(g_full + 8 * seg, n / kSegments & 1u, p.status, kStatusTimeoutMma);
        const int tiles = ok ? s_segs[seg].tiles : 0;
        __syncwarp();
        if (lane == 0) mbar_arrive(g_empty + 8 * seg);
        if (tiles == 0) break;
        if (first) ok = ok && wait_bar(q_full, n & 1u, p.status, kStatusTimeoutMma);
#pragma unroll 1
        for (int i = 0; i < tiles; ++i) {
          const int g = i & 1;
          if (first) {
            // S of the group's tile before has been read
            if (i >= 2) ok = ok && wait_bar(s_free + 8 * g, (turn[g] - 1) & 1u, p.status, kStatusTimeoutMma);
            ok = ok && wait_bar(full + 8 * stage, phase, p.status, kStatusTimeoutMma);
            tc_fence_after();
            if (one && ok) {
              const uint32_t k = base + stage * F::kStage;
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                mma_ts(tmem + F::kS + g * kKeys, tmem + F::kQ + kk * 8,
                       smem_desc_sw128(k + (kk >> 2) * F::kHalf + (kk & 3) * 32), kIdQk, kk > 0);
              tc_commit(s_full + 8 * g);
            }
          } else {
            ok = ok && wait_bar(p_full + 8 * g, turn[g] & 1u, p.status, kStatusTimeoutMma);
            tc_fence_after();
            if (one && ok) {
              const uint32_t v = base + stage * F::kStage + F::kOperand;
#pragma unroll
              for (int kk = 0; kk < kKeys / 16; ++kk)
                mma_ts(tmem + F::kO + g * D, tmem + F::kP + g * (kKeys / 2) + kk * 8,
                       smem_desc_n_major(v + kk * 2048, F::kHalf), kIdPv, i >= 2 || kk > 0);
              tc_commit(o_done + 8 * g);
              tc_commit(empty + 8 * stage);
            }
          }
          ++turn[g];
          __syncwarp();
          if (++stage == NS) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    } else if (warp == kWalkWarp) {
      // ---------------------------------------------------- the CTA's share
      Share share;
      const bool mine = find_share_walk(p, blockIdx.x, share);
      Walk walk;
      if (mine) walk.begin(p, share);
      bool ok = true;
      int slot = 0;
      uint32_t phase = 0;
      for (int n = 0;; ++n) {
        const bool more = ok && mine && walk.next(p);
        const int seg = n % kSegments;
        ok = ok && wait_bar(g_empty + 8 * seg, (n / kSegments & 1u) ^ 1u, p.status, kStatusTimeoutProducer);
        if (lane == 0) {
          Segment& s = s_segs[seg];
          s.tiles = more ? walk.u1 - walk.u0 : 0;
          if (more) {
            s.b = walk.share.b;
            s.lo = walk.seq.lo;
            s.start = walk.seq.start;
            s.len = walk.seq.len;
            s.head = walk.head;
            s.row0 = walk.row0;
            s.rows = walk.rows;
            s.u0 = walk.u0;
            s.whole = walk.u0 == 0 && walk.u1 == walk.seq.units;
          }
          mbar_arrive(g_full + 8 * seg);
        }
        __syncwarp();
        if (!more) {
          // the end, for each team that goes by tiles
#pragma unroll 1
          for (int i = 0; i < kTeams<kFormat>; ++i) {
            ok = ok && wait_bar(t_empty + 8 * slot, phase ^ 1u, p.status, kStatusTimeoutProducer);
            if (lane == 0) {
              s_tiles[slot].kind = 0;
              mbar_arrive(t_full + 8 * slot);
            }
            if (++slot == kSlots) {
              slot = 0;
              phase ^= 1u;
            }
          }
          if (lane == 0) p.splits[blockIdx.x] = mine ? split_of(p, share, blockIdx.x) : Split{};
          break;
        }
        // Page ids come through shared memory, kIds - 1 tiles ahead; lanes have keys
        // lane and lane + 32.
        const int32_t* const table = p.c.table + walk.share.b * p.c.ldt;
        const int64_t head_at = walk.head * p.c.head_stride;
        const int64_t head_scale = static_cast<int64_t>(walk.head) * p.c.page.d;
        const uint32_t ids = base + F::kIdsAt + lane * 4;
        const auto ask = [&](int u) {
          if (u < walk.u1) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int key = u * kKeys + j * 32 + lane;
              const bool here = key < walk.seq.len;
              copy4(ids + u % kIds * (4 * kKeys) + j * 128, here ? table + quotient(key, p.c.page) : table, here ? 4 : 0);
            }
          }
          copies_sealed();
        };
#pragma unroll 1
        for (int i = 0; i < kIds - 1; ++i) ask(walk.u0 + i);
#pragma unroll 1
        for (int u = walk.u0; u < walk.u1; ++u) {
          const int key0 = u * kKeys;
          ask(u + kIds - 1);
          ok = ok && wait_bar(t_empty + 8 * slot, phase ^ 1u, p.status, kStatusTimeoutProducer);
          copies_wait<kIds - 1>();
          Tile& tile = s_tiles[slot];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int key = key0 + j * 32 + lane;
            const int id = static_cast<int>(ld_shared_u(ids + u % kIds * (4 * kKeys) + j * 128));
            const bool good = key < walk.seq.len && id >= 0 && id < p.c.pages;
            const int spot = key - quotient(key, p.c.page) * static_cast<int>(p.c.page.d);
            tile.at[j * 32 + lane] = good ? head_at + static_cast<int64_t>(id) * static_cast<int>(p.c.page_stride) +
                                                static_cast<int64_t>(spot) * static_cast<int>(p.c.token_stride)
                                          : -1;
            if (kCoded) tile.scale[j * 32 + lane] = head_scale + static_cast<int64_t>(id) * p.c.page_scales + spot;
            const uint32_t valid = __ballot_sync(0xFFFFFFFFu, good);
            if (lane == 0) tile.valid[j] = valid;
          }
          if (lane == 0) tile.kind = 1 + (key0 + kKeys > walk.seq.start ? 2 : 0) + (u == walk.u0 ? 4 : 0);
          __syncwarp();
          if (lane == 0) mbar_arrive(t_full + 8 * slot);
          if (++slot == kSlots) {
            slot = 0;
            phase ^= 1u;
          }
        }
        copies_wait<0>();
      }
    } else if (warp == kScaleWarp) {
      // ------------------------------------------------------------- scales
      // A lane has keys lane and lane + 32, from the copy to what the softmax reads.
      bool ok = true;
      int slot = 0, from_slot = 0, stage = 0;
      uint32_t t_phase = 0, phase = 0;
      float ref = 0.f;
      bool open = true;
      const uint32_t raw = base + F::kRawScaleAt + lane * 4;
      const auto fetch = [&] {
        if (open) {
          ok = ok && wait_bar(t_full + 8 * slot, t_phase, p.status, kStatusTimeoutDecode);
          const Tile& tile = s_tiles[slot];
          open = ok && tile.kind != 0;
          if (kCoded && open) {
            const uint32_t to = raw + slot % kRawScales * (8 * kKeys);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int bytes = tile.valid[j] >> lane & 1 ? 4 : 0;
              const int64_t at = bytes ? tile.scale[j * 32 + lane] : 0;
              copy4(to + j * 128, p.c.k_scale + at, bytes);
              copy4(to + 4 * kKeys + j * 128, p.c.v_scale + at, bytes);
            }
          }
          if (++slot == kSlots) {
            slot = 0;
            t_phase ^= 1u;
          }
        }
        copies_sealed();
      };
      static_assert(kSlots % kRawScales == 0, "a slot's scales have one place");
#pragma unroll 1
      for (int s = 0; s < kRawScales - 1; ++s) fetch();
#pragma unroll 1
      for (;;) {
        fetch();
        if (!ok) break;
        copies_wait<kRawScales - 1>();
        const Tile& tile = s_tiles[from_slot];
        const int kind = tile.kind;
        if (kind == 0) break;
        ok = ok && wait_bar(empty + 8 * stage, phase ^ 1u, p.status, kStatusTimeoutProducer);
        const uint32_t side = base + F::kSideAt + stage * kSide;
        if (lane < 2) st_shared_u(side + kValid + 4 * lane, tile.valid[lane]);
        if constexpr (kCoded) {
          const uint32_t at = raw + from_slot % kRawScales * (8 * kKeys);
          if (kind & 4) ref = 0.f;
          float w[2];
          uint32_t top_bits = 0;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            w[j] = ld_shared_f(at + 4 * kKeys + j * 128);
            const uint32_t size = __float_as_uint(w[j]) & 0x7FFFFFFFu;
            const bool fine = size < 0x7F800000u;
            if (fine) top_bits = max(top_bits, size);
            // before the drafts every row sees the key, and NaN is what all of them get
            if (!fine) w[j] = kind & 2 ? 0.f : __uint_as_float(0x7FC00000u);
            if (kind & 2) {
              const uint32_t odd = __ballot_sync(0xFFFFFFFFu, !fine);
              if (lane == 0) st_shared_u(side + kOddScale + 4 * j, odd);
            }
          }
          const float top = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, top_bits));
          // a power of two not above the largest scale: its reciprocal is exact, and
          // what is stored is at most 2
          if (top > 2.f * ref) ref = __uint_as_float(max(__float_as_uint(top) & 0x7F800000u, 0x00800000u));
          const float inv = ref > 0.f ? __frcp_rn(ref) : 0.f;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            st_shared_f(side + j * 128 + lane * 4, ld_shared_f(at + j * 128));
            st_shared_f(side + kVScale + j * 128 + lane * 4, w[j] * inv);
          }
          if (lane == 0) st_shared_f(side + kRef, ref);
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(full + 8 * stage);
          mbar_arrive(t_empty + 8 * from_slot);
        }
        if (++from_slot == kSlots) from_slot = 0;
        if (++stage == NS) {
          stage = 0;
          phase ^= 1u;
        }
      }
      copies_wait<0>();
    }
  } else if (warp >= kLoadWarp) {
    // --------------------------------------------------------------- cache
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLoadRegs));
    constexpr int kLoadThreads = 32 * kTeam, TM = kTeams<kFormat>;
    const int team = (warp - kLoadWarp) / kTeam, tid = threadIdx.x - 32 * (kLoadWarp + team * kTeam);
    constexpr int kRow = kCoded ? D : 2 * D, kPieces = kRow / 16, kTurn = kLoadThreads / kPieces;
    constexpr int kPasses = kKeys / kTurn;
    const int piece = tid % kPieces, key_of = tid / kPieces;
    const uint8_t* const from_k = p.c.k + piece * 16;
    const uint8_t* const from_v = p.c.v + piece * 16;
    // Tiles of a team on their way when it hands one over.  A tile is handed over
    // before the next one is asked for: its stage may still be busy with a tile that
    // waits for nothing but this one's turn.
    static_assert(kSlots % TM == 0 && NS % 2 == 0 && (!kCoded || kRaw % TM == 0), "a team's places");
    constexpr int kLag = kCoded ? kRaw / TM : (NS - 1) / TM > 0 ? (NS - 1) / TM : 1;
    uint32_t kinds = 0;  // of the tiles issued: three bits each, the oldest lowest
    bool ok = true, open = true;
    int stage = team % NS, slot = team;
    uint32_t phase = team / NS, t_phase = 0;
    const auto place = [&](int key, int half, int chunk) {
      return half * F::kHalf + key * 128 + ((chunk ^ (key & 7)) << 4);
    };
    const auto landed = [&] {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full + 8 * stage);
      if ((stage += TM) >= NS) {
        stage -= NS;
        phase ^= 1u;
      }
    };
    // Tiles of drafts: what is no finite number is taken out of this thread's own
    // chunks of V, and the keys that had some are noted.
    const auto finite_only = [&](int key) {
      const uint32_t v = base + stage * F::kStage + F::kOperand;
      uint32_t odd = 0;
#pragma unroll 1
      for (int i = 0; i < (kCoded ? 2 : 1); ++i) {
        const uint32_t at = v + (kCoded ? place(key, piece >> 2, 2 * (piece & 3) + i) : place(key, piece >> 3, piece & 7));
        const uint4 w = ld_shared_u4(at);
        uint32_t o = 0;
        const uint32_t a = finite_pair<kBf16>(w.x, o), b = finite_pair<kBf16>(w.y, o);
        const uint32_t c = finite_pair<kBf16>(w.z, o), d = finite_pair<kBf16>(w.w, o);
        if (o) st_shared_u4(at, a, b, c, d);
        odd |= o;
      }
      const uint32_t who = __ballot_sync(0xFFFFFFFFu, odd) >> (lane - piece) & ((1u << kPieces) - 1u);
      if (piece == 0) st_shared_byte(base + F::kSideAt + stage * kSide + kOdd + key, who ? 1u : 0u);
    };
    static_assert(!kCoded || kTurn % 8 == 0, "a thread's rows have one place in the swizzle");
    // 8-bit codes: the second half's lanes store their two chunks in the other
    // order, so the eight lanes of a key meet eight different banks
    const int swap = kCoded ? piece >> 2 & 1 : 0;
    const uint32_t put_a = place(key_of, piece >> 2, 2 * (piece & 3) + swap);
    const uint32_t put_b = place(key_of, piece >> 2, 2 * (piece & 3) + 1 - swap);
    int in = team;  // raw slot, or stage, of the tile that is issued
    uint32_t in_phase = 0;
    const auto issue = [&] {
      int kind = 0;
      if (open) {
        ok = ok && wait_bar(t_full + 8 * slot, t_phase, p.status, kStatusTimeoutDecode);
        kind = ok ? s_tiles[slot].kind : 0;
        open = kind != 0;
      }
      if (kind) {
        if constexpr (!kCoded)
          ok = ok && wait_bar(empty + 8 * in, in_phase ^ 1u, p.status, kStatusTimeoutProducer);
        const uint32_t to = kCoded ? base + F::kRawAt + in * F::kRawTile + tid * 16 : base + in * F::kStage;
#pragma unroll
        for (int j = 0; j < kPasses; ++j) {
          const int key = j * kTurn + key_of;
          const int64_t at = s_tiles[slot].at[key];
          const int64_t from = at >= 0 ? at : 0;
          const int bytes = at >= 0 ? 16 : 0;
          const uint32_t dst = to + (kCoded ? j * kLoadThreads * 16 : place(key, piece >> 3, piece & 7));
          copy16(dst, from_k + from, bytes);
          copy16(dst + (kCoded ? F::kRawTile / 2 : F::kOperand), from_v + from, bytes);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(t_empty + 8 * slot);
        if ((slot += TM) >= kSlots) {
          slot -= kSlots;
          t_phase ^= 1u;
        }
        if ((in += TM) >= (kCoded ? kRaw : NS)) {
          in -= kCoded ? kRaw : NS;
          in_phase ^= 1u;
        }
      }
      copies_sealed();
      kinds = kinds >> 3 | static_cast<uint32_t>(kind) << (3 * kLag - 3);
    };
#pragma unroll 1
    for (int i = 0; i < kLag; ++i) issue();
    int raw = team;
#pragma unroll 1
    for (;;) {
      const uint32_t kind = kinds & 7u;
      if (kind == 0) break;
      copies_wait<kLag - 1>();
      if constexpr (kCoded) {
        // this thread's own pieces: codes to fp16
        ok = ok && wait_bar(empty + 8 * stage, phase ^ 1u, p.status, kStatusTimeoutProducer);
        const uint32_t from = base + F::kRawAt + raw * F::kRawTile + tid * 16;
        const uint32_t to = base + stage * F::kStage;
#pragma unroll
        for (int j = 0; j < 2 * kPasses; ++j) {
          const int pass = j % kPasses;
          const uint32_t src = from + j / kPasses * (F::kRawTile / 2) + pass * kLoadThreads * 16;
          const uint32_t dst = to + j / kPasses * F::kOperand + pass * kTurn * 128;
          const uint2 a = ld_shared_u2(src + swap * 8), b = ld_shared_u2(src + 8 - swap * 8);
          st_shared_u4(dst + put_a, decode_pair<kFormat>(a.x, 0), decode_pair<kFormat>(a.x, 1),
                       decode_pair<kFormat>(a.y, 0), decode_pair<kFormat>(a.y, 1));
          st_shared_u4(dst + put_b, decode_pair<kFormat>(b.x, 0), decode_pair<kFormat>(b.x, 1),
                       decode_pair<kFormat>(b.y, 0), decode_pair<kFormat>(b.y, 1));
        }
        if ((raw += TM) >= kRaw) raw -= kRaw;
      }
      if (kFormat != PROJ_KV_INT8 && (kind & 2u)) {
#pragma unroll 1
        for (int j = 0; j < kPasses; ++j) finite_only(j * kTurn + key_of);
      }
      landed();
      issue();
    }
    copies_wait<0>();
  } else {
    // ------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    const int group = warp >> 2, quad = warp & 3, lane_row = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t my_s = tmem + lanes + F::kS + group * kKeys, my_p = tmem + lanes + F::kP + group * (kKeys / 2);
    const uint32_t my_o = tmem + lanes + F::kO + group * D;
    const int G = static_cast<int>(p.group.d);
    bool ok = true;
    uint32_t turn = 0;   // tiles that this group has had
    int tile_stage = 0;  // of the item's first tile
    uint32_t tile_phase = 0;
    for (int n = 0;; ++n) {
      const int slot_of = n % kSegments;
      ok = ok && wait_bar(g_full + 8 * slot_of, n / kSegments & 1u, p.status, kStatusTimeoutEpilogue);
      // A wait that gave up ends the loop for all: they meet at barriers below.
      if (named_bar_sync_or(5, 32 * kSoftWarps, !ok)) break;
      // (stays in shared memory until its end: registers are short)
      const Segment& seg = s_segs[slot_of];
      const int tiles = seg.tiles;
      if (tiles == 0) break;
      const int before_drafts = seg.start - seg.u0 * kKeys;  // keys of the segment
      // Up to 64 rows: both halves of the lanes hold them, the MMAs make their scores
      // twice at no cost, and each half takes 32 of a tile's 64 keys (of the other
      // 32 its probabilities are zero): half the softmax for a warp.
      const bool halves = seg.rows <= 64;
      const int row = halves ? lane_row & 63 : lane_row;
      const bool real = row < seg.rows;
      const bool busy = (halves ? quad & 1 : quad) * 32 < seg.rows;  // one of the warp's rows is real
      const int c0 = halves ? quad >> 1 : 0, c1 = halves ? c0 + 1 : 2;  // columns / 32
      const int r = seg.row0 + (real ? row : 0);
      const int token = quotient(r, p.group), head = seg.head * G + r - token * G;
      // -------------------------------------------------------- queries --
      float fq = 1.f;
      // Each group brings half of the columns.  The factor of a row's scores is
      // positive (its sign goes to the queries, and so does a zero), so the largest
      // product is the largest score.
      constexpr bool kNarrow = kCoded && std::is_same_v<T, __nv_bfloat16>;
      uint32_t q[D / 4];
      if (busy) {
        const uint8_t* from = p.q + static_cast<int64_t>(seg.lo + token) * p.ldq + static_cast<int64_t>(head) * D * 2 + group * D;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint4 w = *reinterpret_cast<const uint4*>(from + i * 16);
          q[4 * i] = w.x;
          q[4 * i + 1] = w.y;
          q[4 * i + 2] = w.z;
          q[4 * i + 3] = w.w;
        }
      }
      float f = 1.f;
      F2 up = f2(1.f);
      if constexpr (kNarrow) {
        // bf16 to fp16: the row's largest magnitude is brought to 2^14 .. 2^15
        uint32_t pairs = 0;
        const uint32_t room = base + F::kMl + lane_row * 4;
        if (busy) {
#pragma unroll
          for (int i = 0; i < D / 4; ++i) pairs = __vmaxu2(pairs, q[i] & 0x7FFF7FFFu);
          st_shared_u(room + group * 512, pairs);
        }
        named_bar_sync(1, 32 * kSoftWarps);
        if (busy) pairs = __vmaxu2(pairs, ld_shared_u(room + (1 - group) * 512));
        const uint32_t most = max(pairs & 0xFFFFu, pairs >> 16);
        int e = 0;
        if (most > 0 && most < 0x7F80u) e = min(126, 14 - ilogbf(__uint_as_float(most << 16)));
        const float s = scalbnf(1.f, e);
        up = f2(p.scale_log2 > 0.f ? s : p.scale_log2 < 0.f ? -s : 0.f);
        f = scalbnf(1.f, -e);
      }
      if (busy) {
        if constexpr (kNarrow) {
#pragma unroll
          for (int i = 0; i < D / 4; ++i) {
            float x, y;
            widen2(q[i], x, y, __nv_bfloat16());
            parts(mul2(f2(x, y), up), x, y);
            q[i] = pack2(x, y, __half());
          }
        } else if (p.scale_log2 <= 0.f) {
          const uint32_t keep = p.scale_log2 == 0.f ? 0u : 0xFFFFFFFFu;
#pragma unroll
          for (int i = 0; i < D / 4; ++i) q[i] = (q[i] ^ 0x80008000u) & keep;
        }
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
          tmem_st16(tmem + lanes + F::kQ + group * (D / 4) + i * 16, q + i * 16);
        tmem_st_wait();
        fq = fmaxf(f * fabsf(p.scale_log2), 1.17549435e-38f);
      }
      if (halves && busy) {
        const uint32_t zero[16] = {};
        tmem_st16(my_p + 16 * (1 - c0), zero);
        tmem_st_wait();
      }
      tc_fence_before();
      named_bar_sync(1, 32 * kSoftWarps);
      if (lane == 0) mbar_arrive(q_full);

      // ---------------------------------------------------------- tiles --
      float ref = kNoScore, sum = 0.f, v_ref = 0.f;
      bool odd = false;
      int stage = tile_stage + group;
      uint32_t phase = tile_phase;
      if (stage >= NS) {
        stage -= NS;
        phase ^= 1u;
      }
      for (int i = group; i < tiles; i += 2) {
        const uint32_t side = base + F::kSideAt + stage * kSide;
        ok = ok && wait_bar(s_full + 8 * group, turn & 1u, p.status, kStatusTimeoutEpilogue);
        tc_fence_after();
        if (busy) {
          // what stands beside the stage
          const int draft = i * kKeys - before_drafts;  // of the first key
          uint64_t seen = ~uint64_t{0};
          ok = ok && wait_bar(full + 8 * stage, phase, p.status, kStatusTimeoutEpilogue);
          const uint2 valid = ld_shared_u2(side + kValid);
          const bool partial = (valid.x & valid.y) != 0xFFFFFFFFu || draft + kKeys > 0;
          if (__builtin_expect(partial, 0))
            seen = seen_here<kFormat>(p, seg.lo, token, draft, valid, side + kOddScale, side + kOdd, odd);
          float down = 1.f, tile_sum = 0.f;
          if constexpr (kCoded) {
            const float now = ld_shared_f(side + kRef);
            if (now != v_ref) {
              down = v_ref / now;  // both powers of two, or v_ref 0 and nothing of V summed yet
              if (partial && v_ref > 0.f) {
                // not every row sees the key: this row's reference goes down instead
                const int low = lowered(sum, exponent_of(now) - exponent_of(v_ref));
                ref -= static_cast<float>(low);
                sum *= power_of_two(low);
                down *= power_of_two(low);
              }
              v_ref = now;
            }
          }
          const F2 q2 = f2(fq);
#pragma unroll 1
          for (int c = c0; c < c1; ++c) {
            float f[32];
            tmem_ld32(my_s + c * 32, f);
            tmem_ld_wait();
            if (halves) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(s_free + 8 * group);
            }
            if constexpr (kCoded) {
#pragma unroll
              for (int j = 0; j < 32; j += 16) {
                float4 ks[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) ks[x] = ld_shared_f4(side + c * 128 + (j + 4 * x) * 4);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                  float* y = f + j + 4 * x;
                  parts(mul2(f2(y[0], y[1]), f2(ks[x].x, ks[x].y)), y[0], y[1]);
                  parts(mul2(f2(y[2], y[3]), f2(ks[x].z, ks[x].w)), y[2], y[3]);
                }
              }
            }
            float by_scale = 0.f;  // of what is seen here, logarithm of V's largest scale
            if (__builtin_expect(partial, 0)) {
              const uint32_t here = static_cast<uint32_t>(c ? seen >> 32 : seen);
              float most = 0.f;
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                float4 vs = make_float4(0.f, 0.f, 0.f, 0.f);
                if constexpr (kCoded) vs = ld_shared_f4(side + kVScale + c * 128 + j * 4);
                const float v[4] = {vs.x, vs.y, vs.z, vs.w};
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                  if (here >> (j + x) & 1)
                    most = fmaxf(most, fabsf(v[x]));
                  else
                    f[j + x] = -INFINITY;
                }
              }
              if constexpr (kCoded) by_scale = fmaxf(__log2f(most), -kRoom);
            }
            float tops[4] = {f[0], f[1], f[2], f[3]};
#pragma unroll
            for (int j = 4; j < 32; ++j) tops[j & 3] = fmaxf(tops[j & 3], f[j]);
            const float top = fmaf(fq, fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])), by_scale);
            if (__builtin_expect(__any_sync(0xFFFFFFFFu, top > ref + kSlack), 0)) {
              if (top > ref + kSlack) {
                const float step = exp2_fast(ref - top);
                ref = top;
                sum *= step;
                down *= step;
              }
              if (c > c0) {
                // the tile's first half again, relative to the new reference
                c = c0 - 1;
                tile_sum = 0.f;
                continue;
              }
            }
            if (!halves && c == c1 - 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(s_free + 8 * group);
            }
            const F2 low = f2(kLift - ref);
            F2 total[2] = {f2(0.f), f2(0.f)};
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 32; j += 16) {
              float4 vs[4];
              if constexpr (kCoded) {
#pragma unroll
                for (int x = 0; x < 4; ++x) vs[x] = ld_shared_f4(side + kVScale + c * 128 + (j + 4 * x) * 4);
              }
              float e[16];
#pragma unroll
              for (int x = 0; x < 16; x += 2) parts(fma2(f2(f[j + x], f[j + x + 1]), q2, low), e[x], e[x + 1]);
#pragma unroll
              for (int x = 0; x < 16; ++x) e[x] = exp2_fast(e[x]);
#pragma unroll
              for (int x = 0; x < 16; x += 4) {
                const F2 e0 = f2(e[x], e[x + 1]), e1 = f2(e[x + 2], e[x + 3]);
                total[0] = add2(total[0], e0);
                total[1] = add2(total[1], e1);
                if constexpr (kCoded) {
                  parts(mul2(e0, f2(vs[x / 4].x, vs[x / 4].y)), e[x], e[x + 1]);
                  parts(mul2(e1, f2(vs[x / 4].z, vs[x / 4].w)), e[x + 2], e[x + 3]);
                }
                w[(j + x) / 2] = pack2(e[x], e[x + 1], C());
                w[(j + x) / 2 + 1] = pack2(e[x + 2], e[x + 3], C());
              }
            }
            float a, b;
            parts(add2(total[0], total[1]), a, b);
            tile_sum += a + b;
            // the group's products before: P is free, and O complete
            if (c == c0 && turn > 0)
              ok = ok && wait_bar(o_done + 8 * group, (turn - 1) & 1u, p.status, kStatusTimeoutEpilogue);
            tc_fence_after();
            tmem_st16(my_p + c * 16, w);
          }
          sum += tile_sum;
          if (__builtin_expect(i >= 2 && __any_sync(0xFFFFFFFFu, down != 1.f), 0)) {
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              float o[16];
              tmem_ld16(my_o + c, o);
              tmem_ld_wait();
              uint32_t w[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) w[j] = __float_as_uint(o[j] * down);
              tmem_st16(my_o + c, w);
            }
          }
          tmem_st_wait();
        } else {
          if (lane == 0) mbar_arrive(s_free + 8 * group);
          if (turn > 0) ok = ok && wait_bar(o_done + 8 * group, (turn - 1) & 1u, p.status, kStatusTimeoutEpilogue);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + 8 * group);
        ++turn;
        stage += 2;
        if (stage >= NS) {
          stage -= NS;
          phase ^= 1u;
        }
      }
      tile_stage += tiles;
      while (tile_stage >= NS) {
        tile_stage -= NS;
        tile_phase ^= 1u;
      }

      // ----------------------------------------------- the groups' sums joined --
      const uint32_t ml = base + F::kMl;
      st_shared_f(ml + (group * 128 + lane_row) * 12, ref - kLift);
      st_shared_f(ml + (group * 128 + lane_row) * 12 + 4, sum);
      st_shared_f(ml + (group * 128 + lane_row) * 12 + 8, kCoded ? v_ref : 1.f);
      if (tiles > group) ok = ok && wait_bar(o_done + 8 * group, (turn - 1) & 1u, p.status, kStatusTimeoutEpilogue);
      // a value of V that is no finite number, seen by this row
      const bool any_odd = named_bar_sync_or(2, 32 * kSoftWarps, odd);
      tc_fence_after();
      {
        // the row's sums: of both groups, and of both halves of the lanes
        float m[4], l[4], up[2];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const uint32_t mine = ml + (g * 128 + lane_row) * 12, other = ml + (g * 128 + (lane_row ^ 64)) * 12;
          m[g] = ld_shared_f(mine);
          l[g] = ld_shared_f(mine + 4);
          up[g] = ld_shared_f(mine + 8);
          m[2 + g] = halves ? ld_shared_f(other) : -INFINITY;
          l[2 + g] = halves ? ld_shared_f(other + 4) : 0.f;
        }
        const float top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
        float all = 0.f;
#pragma unroll
        for (int g = 0; g < 4; ++g) all += l[g] * exp2_fast(m[g] - top);
        const float a0 = exp2_fast(m[0] - top) * up[0], a1 = exp2_fast(m[1] - top) * up[1];
        const bool whole = seg.whole;
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (seg.u0 == 0 ? 1 : 0);
        float* part = p.part_o + (slot * kAttnTcRows + row) * D;
        // Each group writes half of the columns, and of those, where the lanes hold two
        // halves of each row, each half a half: it gives the other its sums of the
        // other's columns.
        const bool writes = real && busy;
        const int side = halves ? quad >> 1 : 0, width = halves ? D / 4 : D / 2;
        const int first = group * (D / 2) + side * width, given = group * (D / 2) + (1 - side) * width;
        const uint32_t swap = base + F::kSwapAt + group * 8192 + row * 4;
        const bool gated = writes && whole && p.gate;
        const T* const gates = reinterpret_cast<const T*>(p.gate + static_cast<int64_t>(seg.lo + token) * p.ldg) + head * D;
        const auto sums = [&](int c, float (&o)[16]) {
          float o1[16];
          tmem_ld16(tmem + lanes + F::kO + c, o);
          if (tiles > 1) tmem_ld16(tmem + lanes + F::kO + D + c, o1);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) o[j] = tiles > 1 ? o[j] * a0 + o1[j] * a1 : o[j] * a0;
        };
#pragma unroll 1
        for (int x = 0; x < width; x += 16) {
          const int c = first + x;
          Vec<T, 8> gate[2];
          if (gated) {
            gate[0] = load_vec<T, 8>(gates + c);
            gate[1] = load_vec<T, 8>(gates + c + 8);
          }
          float o[16];
#pragma unroll 1
          for (int own = halves ? 0 : 1; own < 2; ++own) {
            if (busy) sums(own ? c : given + x, o);
            if (!own) {
              if (busy) {
#pragma unroll
                for (int j = 0; j < 16; ++j) st_shared_f(swap + side * 4096 + j * 256, o[j]);
              }
              named_bar_sync(3 + group, 128);
            }
          }
          if (halves && busy) {
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] += ld_shared_f(swap + (1 - side) * 4096 + j * 256);
          }
          if (__builtin_expect(any_odd && writes, 0)) {
            float with[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) with[j] = o[j];
            add_odd<T, kFormat>(p, seg, token, c, with);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = with[j];
          }
          if (writes && whole) {
            write_out<T>(p, static_cast<int64_t>(seg.lo + token), head * D + c, o, all, gate);
          } else if (writes) {
#pragma unroll
            for (int j = 0; j < 16; j += 4)
              *reinterpret_cast<float4*>(part + c + j) = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
          }
          // what was given has been read
          if (halves && x + 16 < width) named_bar_sync(3 + group, 128);
          __syncwarp();
        }
        if (writes && group == 0 && side == 0) {
          if (whole) {
            if (p.lse) p.lse[static_cast<int64_t>(seg.lo + token) * p.heads + head] = lse_of(top, all);
          } else {
            *reinterpret_cast<float2*>(p.part_ml + (slot * kAttnTcRows + row) * 2) = make_float2(top, all);
          }
        }
      }
      tc_fence_before();
      // both groups are done with the item's Q, O and sums
      named_bar_sync(1, 32 * kSoftWarps);
      tc_fence_after();
      if (lane == 0) mbar_arrive(g_empty + 8 * slot_of);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <typename T, int kFormat, int D>
cudaError_t tc_run(const AttnParams& p, cudaStream_t s) {
  const auto kernel = attn_tc_kernel<T, kFormat, D>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), Tc<kFormat, D>::kSmem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(p.ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Tc<kFormat, D>::kSmem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename T>
cudaError_t tc_format(const AttnParams& p, int format, cudaStream_t s) {
  if (p.D == 64)
    return format == PROJ_KV_ROWS   ? tc_run<T, PROJ_KV_ROWS, 64>(p, s)
           : format == PROJ_KV_E4M3 ? tc_run<T, PROJ_KV_E4M3, 64>(p, s)
                                    : tc_run<T, PROJ_KV_INT8, 64>(p, s);
  return format == PROJ_KV_ROWS   ? tc_run<T, PROJ_KV_ROWS, 128>(p, s)
         : format == PROJ_KV_E4M3 ? tc_run<T, PROJ_KV_E4M3, 128>(p, s)
                                  : tc_run<T, PROJ_KV_INT8, 128>(p, s);
}

}  // namespace

cudaError_t attn_tc_launch(const AttnParams& p, int dtype, int format, cudaStream_t s) {
  return dtype == PROJ_BF16 ? tc_format<__nv_bfloat16>(p, format, s) : tc_format<__half>(p, format, s);
}

}  // namespace proj
