// attn_tc.cu -- attention of drafted tokens over the cache on tcgen05, for
// items of many rows (a group's heads times a sequence's drafts above 32).
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
// other's sums; they meet at the item's end.  8-15 bring the cache: 8-bit
// codes come to registers by 16-byte loads, four tiles ahead, and go to shared
// memory as fp16, which holds them exactly (through shared memory twice they
// would cost it half as much again as the MMAs' own reads); 16-bit entries by
// asynchronous copies.  Warp 16 issues the MMAs; 17-19 only complete its
// warpgroup, which gives registers to the others.
//
// Softmax as in the streaming kernel: a reference per row that moves only when
// a score is more than 6 above it (in powers of two), whereupon O is scaled in
// tensor memory; probabilities are 2^8 at the reference, in fp16 (bf16 caches:
// bf16).  Scales of K multiply the fp32 score; those of V the probability,
// relative to a power-of-two reference that the loading warps keep.
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "attn.h"
#include "kernels.h"
#include "kv_num.cuh"

namespace proj {
namespace {

constexpr int kSoftWarps = 8, kLoadWarp = 8, kLoadWarps = 8, kMmaWarp = 16;
constexpr int kThreads = 32 * 20;
// Registers a thread: at launch, and of the three kinds of warpgroups (two of
// softmax, two of loading, one of the MMA warp).
constexpr int kRegs = 96, kSoftRegs = 128, kLoadRegs = 88, kMmaRegs = 48;
static_assert(2 * kSoftRegs + 2 * kLoadRegs + kMmaRegs <= 5 * kRegs && 5 * kRegs * 128 <= 65536, "registers");
constexpr int kLoadThreads = 32 * kLoadWarps;
constexpr int kKeys = kAttnTcUnit;
constexpr int kTmemCols = 512;
constexpr int kAhead = 4;  // tiles on their way to registers

template <int D>
struct Tc {
  static constexpr int kHalves = D / 64;            // of 64 dimensions
  static constexpr int kHalf = kKeys * 128;         // bytes
  static constexpr int kOperand = kHalves * kHalf;  // K or V of a tile
  static constexpr int kStage = 2 * kOperand;
  static constexpr int kStages = D == 128 ? 6 : 8;
  // beside a stage: scales of K and V, the reference of V's, keys that exist, keys
  // of drafts with a value that is no finite number
  static constexpr int kSide = 640, kVScale = 256, kRef = 512, kValid = 520, kOdd = 576;
  static constexpr int kSideAt = kStages * kStage;
  static constexpr int kFq = kSideAt + kStages * kSide;  // float[128]
  static constexpr int kMl = kFq + 512;                  // float[2][128][3]
  static constexpr int kBarsAt = kMl + 3072;
  static constexpr int kBars = 2 * kStages + 9;
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
    if (mbar_try_wait_hint(bar, parity, 1000u)) return true;
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
    const int64_t item = local / seq.units;
    u0 = static_cast<int>(local - item * seq.units);
    u1 = static_cast<int>(min(static_cast<int64_t>(seq.units), u0 + (share.end - at)));
    head = static_cast<int>(item / seq.tiles);
    row0 = static_cast<int>(item - static_cast<int64_t>(head) * seq.tiles) * kAttnTcRows;
    rows = min(kAttnTcRows, seq.rows * static_cast<int>(p.group.d) - row0);
    at += u1 - u0;
    return true;
  }
};

// What row `token` of a sequence sees of the 64 keys from key0 on.
__device__ __forceinline__ uint64_t low_bits(int n) {
  return n <= 0 ? 0 : n >= 64 ? ~uint64_t{0} : (uint64_t{1} << n) - 1;
}
__device__ __forceinline__ uint64_t seen_of(const AttnParams& p, const Sequence& s, int token,
                                            int key0) {
  const int draft = key0 - s.start;  // of the first key
  uint64_t own;
  if (p.mask) {
    const uint32_t* row = p.mask + (s.lo + token) * p.ldm;
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

template <typename T, int kFormat, int D>
__global__ void __launch_bounds__(kThreads, 1) attn_tc_kernel(const AttnParams p) {
  using F = Tc<D>;
  constexpr bool kCoded = kFormat != PROJ_KV_ROWS;
  using C = std::conditional_t<kCoded, __half, T>;
  constexpr bool kBf16 = std::is_same_v<C, __nv_bfloat16>;
  constexpr int NS = F::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + F::kBarsAt + F::kBars * 8);
  const uint32_t base = smem_u32(smem);
  const uint32_t full = base + F::kBarsAt, empty = full + 8 * NS;
  const uint32_t s_full = empty + 8 * NS, s_free = s_full + 16, p_full = s_free + 16;
  const uint32_t o_done = p_full + 16, q_full = o_done + 16;
  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(full + 8 * s, kLoadWarps);
      mbar_init(empty + 8 * s, 1);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(s_full + 8 * g, 1);
      mbar_init(s_free + 8 * g, 4);
      mbar_init(p_full + 8 * g, 4);
      mbar_init(o_done + 8 * g, 1);
    }
    mbar_init(q_full, kSoftWarps);
    fence_mbar_init();
  }
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

  Share share;
  const bool mine = find_share<kThreads>(p, blockIdx.x, share);
  Walk walk;
  if (mine) walk.begin(p, share);

  if (!mine) {
    // nothing to do but to give the tensor memory back
  } else if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMmaRegs));
    // ----------------------------------------------------------------- MMA
    const bool one = elect_one();
    bool ok = true;
    int stage = 0;        // of the next tile of keys
    uint32_t phase = 0;
    uint32_t turn[2] = {0u, 0u};  // tiles that each group has had
    uint32_t items = 0;
    constexpr uint32_t kIdQk = instruction(kBf16, 0, 128, kKeys), kIdPv = instruction(kBf16, 1, 128, D);
    const auto qk = [&](int g) {
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
      __syncwarp();
      if (++stage == NS) {
        stage = 0;
        phase ^= 1u;
      }
    };
    int pv_stage = 0;
    while (warp == kMmaWarp && walk.next(p)) {
      const int tiles = walk.u1 - walk.u0;
      ok = ok && wait_bar(q_full, items & 1u, p.status, kStatusTimeoutMma);
      ++items;
      tc_fence_after();
      qk(0);
      if (tiles > 1) qk(1);
      for (int i = 0; i < tiles; ++i) {
        const int g = i & 1;
        if (i + 2 < tiles) {
          ok = ok && wait_bar(s_free + 8 * g, turn[g] & 1u, p.status, kStatusTimeoutMma);
          qk(g);
        }
        ok = ok && wait_bar(p_full + 8 * g, turn[g] & 1u, p.status, kStatusTimeoutMma);
        ++turn[g];
        tc_fence_after();
        if (one && ok) {
          const uint32_t v = base + pv_stage * F::kStage + F::kOperand;
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            mma_ts(tmem + F::kO + g * D, tmem + F::kP + g * (kKeys / 2) + kk * 8,
                   smem_desc_n_major(v + kk * 2048, F::kHalf), kIdPv, i >= 2 || kk > 0);
          tc_commit(o_done + 8 * g);
          tc_commit(empty + 8 * pv_stage);
        }
        __syncwarp();
        if (++pv_stage == NS) pv_stage = 0;
      }
    }
  } else if (warp >= kLoadWarp) {
    // --------------------------------------------------------------- cache
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLoadRegs));
    const int tid = threadIdx.x - 32 * kLoadWarp, lwarp = warp - kLoadWarp;
    constexpr int kRow = kCoded ? D : 2 * D, kPieces = kRow / 16, kTurn = kLoadThreads / kPieces;
    constexpr int kPasses = kKeys / kTurn;
    const int piece = tid % kPieces, key_of = tid / kPieces;
    bool ok = true;
    int stage = 0;
    uint32_t phase = 0;
    // The tile that is fetched next, and the pages of its keys.
    bool more = walk.next(p);
    int unit = more ? walk.u0 : 0;
    bool first = true;
    int ids[kPasses], side_ids[2];
    const auto id_of = [&](int key) {
      return key < walk.seq.len ? p.c.table[walk.share.b * p.c.ldt + quotient(key, p.c.page)] : -1;
    };
    const auto pages = [&] {
      if (!more) return;
#pragma unroll
      for (int j = 0; j < kPasses; ++j) ids[j] = id_of(unit * kKeys + j * kTurn + key_of);
      if (lwarp < 2) {
        side_ids[0] = id_of(unit * kKeys + lane);
        side_ids[1] = id_of(unit * kKeys + 32 + lane);
      }
    };
    const auto entry_of = [&](int id, int key, Entry& e) {
      const bool good = id >= 0 && id < p.c.pages;
      const int spot = key - quotient(key, p.c.page) * static_cast<int>(p.c.page.d);
      e = good ? entry_at(p.c, id, spot, walk.head) : Entry{0, 0};
      return good;
    };
    const auto advance = [&] {
      first = false;
      if (++unit == walk.u1) {
        more = walk.next(p);
        unit = more ? walk.u0 : 0;
        first = true;
      }
      pages();
    };
    const auto place = [&](int key, int half, int chunk) {
      return half * F::kHalf + key * 128 + ((chunk ^ (key & 7)) << 4);
    };
    const auto landed = [&] {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full + 8 * stage);
      if (++stage == NS) {
        stage = 0;
        phase ^= 1u;
      }
    };
    pages();
    if constexpr (kCoded) {
      uint4 rk[kAhead][kPasses], rv[kAhead][kPasses];
      float scale[kAhead][2];
      uint32_t valid[kAhead][2];
      int kind[kAhead];  // 0: no tile, 1: a tile, + 2: of drafts, + 4: an item's first
      float ref = 0.f;
      const auto fetch = [&](int s) {
        kind[s] = 0;
        if (!more) return;
        const int key0 = unit * kKeys;
        kind[s] = 1 + (key0 + kKeys > walk.seq.start ? 2 : 0) + (first ? 4 : 0);
#pragma unroll
        for (int j = 0; j < kPasses; ++j) {
          Entry e;
          const bool good = entry_of(ids[j], key0 + j * kTurn + key_of, e);
          rk[s][j] = rv[s][j] = make_uint4(0u, 0u, 0u, 0u);
          if (good) {
            rk[s][j] = *reinterpret_cast<const uint4*>(p.c.k + e.at + piece * 16);
            rv[s][j] = *reinterpret_cast<const uint4*>(p.c.v + e.at + piece * 16);
          }
        }
        if (lwarp < 2) {
          const float* from = lwarp ? p.c.v_scale : p.c.k_scale;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            Entry e;
            const bool good = entry_of(side_ids[j], key0 + j * 32 + lane, e);
            scale[s][j] = good ? from[e.scale] : 0.f;
            valid[s][j] = __ballot_sync(0xFFFFFFFFu, good);
          }
        }
        advance();
      };
      const auto spread = [&](uint32_t to, const uint4& w, int key, bool check, uint32_t& odd) {
        const uint32_t word[4] = {w.x, w.y, w.z, w.w};
        uint32_t h[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          h[2 * i] = decode_pair<kFormat>(word[i], 0);
          h[2 * i + 1] = decode_pair<kFormat>(word[i], 1);
        }
        if (kFormat == PROJ_KV_E4M3 && check) {
#pragma unroll
          for (int i = 0; i < 8; ++i) h[i] = finite_pair<false>(h[i], odd);
        }
        // the second half's lanes store their two chunks in the other order: the
        // eight lanes of a key then meet eight different banks
        const int half = piece >> 2, c = 2 * (piece & 3), x = half & 1;
        st_shared_u4(to + place(key, half, c + x), x ? h[4] : h[0], x ? h[5] : h[1], x ? h[6] : h[2],
                     x ? h[7] : h[3]);
        st_shared_u4(to + place(key, half, c + 1 - x), x ? h[0] : h[4], x ? h[1] : h[5],
                     x ? h[2] : h[6], x ? h[3] : h[7]);
      };
      const auto store = [&](int s) {
        ok = ok && wait_bar(empty + 8 * stage, phase ^ 1u, p.status, kStatusTimeoutProducer);
        const uint32_t to = base + stage * F::kStage, side = base + F::kSideAt + stage * F::kSide;
        const bool check = kind[s] & 2;
#pragma unroll
        for (int j = 0; j < kPasses; ++j) {
          const int key = j * kTurn + key_of;
          uint32_t odd = 0;
          spread(to, rk[s][j], key, false, odd);
          spread(to + F::kOperand, rv[s][j], key, check, odd);
          if (kFormat == PROJ_KV_E4M3 && check) {
            const uint32_t who = __ballot_sync(0xFFFFFFFFu, odd) >> (lane - piece) & ((1u << kPieces) - 1u);
            if (piece == 0) st_shared_byte(side + F::kOdd + key, who ? 1u : 0u);
          }
        }
        if (lwarp == 0) {
          st_shared_f(side + lane * 4, scale[s][0]);
          st_shared_f(side + 128 + lane * 4, scale[s][1]);
          if (lane == 0) {
            st_shared_u(side + F::kValid, valid[s][0]);
            st_shared_u(side + F::kValid + 4, valid[s][1]);
          }
        } else if (lwarp == 1) {
          if (kind[s] & 4) ref = 0.f;
          float v[2] = {scale[s][0], scale[s][1]};
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (!(fabsf(v[j]) < INFINITY)) v[j] = __uint_as_float(0x7FC00000u);
          float top = fmaxf(fabsf(v[0]), fabsf(v[1]));
#pragma unroll
          for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
          // a power of two not above the largest scale: its reciprocal is exact, and
          // what is stored is at most 2
          if (top > 2.f * ref) ref = __uint_as_float(max(__float_as_uint(top) & 0x7F800000u, 0x00800000u));
          const float inv = ref > 0.f ? 1.f / ref : 0.f;
          st_shared_f(side + F::kVScale + lane * 4, v[0] * inv);
          st_shared_f(side + F::kVScale + 128 + lane * 4, v[1] * inv);
          if (lane == 0) st_shared_f(side + F::kRef, ref);
        }
        landed();
      };
#pragma unroll
      for (int s = 0; s < kAhead; ++s) fetch(s);
      for (bool going = true; going;) {
#pragma unroll
        for (int s = 0; s < kAhead; ++s) {
          if (kind[s] == 0) {
            going = false;
            break;
          }
          store(s);
          fetch(s);
        }
      }
    } else {
      // copies two tiles behind their issue
      constexpr int kLag = 3;
      int kind[kLag + 1];
      int in_stage = 0, slot = 0;
      uint32_t in_phase = 0;
      const auto issue = [&](int s) {
        kind[s] = 0;
        if (more) {
          ok = ok && wait_bar(empty + 8 * in_stage, in_phase ^ 1u, p.status, kStatusTimeoutProducer);
          const int key0 = unit * kKeys;
          kind[s] = 1 + (key0 + kKeys > walk.seq.start ? 2 : 0);
          const uint32_t to = base + in_stage * F::kStage, side = base + F::kSideAt + in_stage * F::kSide;
#pragma unroll
          for (int j = 0; j < kPasses; ++j) {
            Entry e;
            const int key = j * kTurn + key_of;
            const int bytes = entry_of(ids[j], key0 + key, e) ? 16 : 0;
            const uint32_t at = to + place(key, piece >> 3, piece & 7);
            copy16(at, p.c.k + e.at + piece * 16, bytes);
            copy16(at + F::kOperand, p.c.v + e.at + piece * 16, bytes);
          }
          if (lwarp == 0) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              Entry e;
              const uint32_t v = __ballot_sync(0xFFFFFFFFu, entry_of(side_ids[j], key0 + j * 32 + lane, e));
              if (lane == 0) st_shared_u(side + F::kValid + 4 * j, v);
            }
          }
          if (++in_stage == NS) {
            in_stage = 0;
            in_phase ^= 1u;
          }
          advance();
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      (void)slot;
#pragma unroll
      for (int s = 0; s < kLag; ++s) issue(s);
      for (bool going = true; going;) {
#pragma unroll
        for (int s = 0; s <= kLag; ++s) {
          if (kind[s] == 0) {
            going = false;
            break;
          }
          issue((s + kLag) % (kLag + 1));
          asm volatile("cp.async.wait_group %0;" ::"n"(kLag) : "memory");
          if (kind[s] & 2) {
            // this thread's own pieces of V: what is no finite number is taken out
            const uint32_t v = base + stage * F::kStage + F::kOperand;
            const uint32_t side = base + F::kSideAt + stage * F::kSide;
#pragma unroll
            for (int j = 0; j < kPasses; ++j) {
              const int key = j * kTurn + key_of;
              const uint32_t at = v + place(key, piece >> 3, piece & 7);
              const uint4 w = ld_shared_u4(at);
              uint32_t odd = 0;
              const uint32_t a = finite_pair<kBf16>(w.x, odd), b = finite_pair<kBf16>(w.y, odd);
              const uint32_t c = finite_pair<kBf16>(w.z, odd), d = finite_pair<kBf16>(w.w, odd);
              if (odd) st_shared_u4(at, a, b, c, d);
              const uint32_t who = __ballot_sync(0xFFFFFFFFu, odd) >> (lane - piece % 32) &
                                   ((1u << kPieces) - 1u);
              if (piece == 0) st_shared_byte(side + F::kOdd + key, who ? 1u : 0u);
            }
          }
          landed();
        }
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
  } else {
    // ------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    const int group = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t my_s = tmem + lanes + F::kS + group * kKeys, my_p = tmem + lanes + F::kP + group * (kKeys / 2);
    const uint32_t my_o = tmem + lanes + F::kO + group * D;
    const int G = static_cast<int>(p.group.d);
    bool ok = true;
    uint32_t turn = 0;   // tiles that this group has had
    int tile_stage = 0;  // of the item's first tile
    uint32_t tile_phase = 0;
    while (walk.next(p)) {
      const Sequence& seq = walk.seq;
      const int tiles = walk.u1 - walk.u0;
      const bool real = row < walk.rows;
      const bool busy = (warp & 3) * 32 < walk.rows;  // one of the warp's rows is real
      const int r = walk.row0 + (real ? row : 0);
      const int token = quotient(r, p.group), head = walk.head * G + r - token * G;
      // -------------------------------------------------------- queries --
      if (group == 0) {
        if (busy) {
          const uint8_t* from = p.q + (seq.lo + token) * p.ldq + static_cast<int64_t>(head) * D * 2;
          uint32_t q[D / 2];
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            const uint4 w = real ? *reinterpret_cast<const uint4*>(from + i * 16) : make_uint4(0u, 0u, 0u, 0u);
            q[4 * i] = w.x;
            q[4 * i + 1] = w.y;
            q[4 * i + 2] = w.z;
            q[4 * i + 3] = w.w;
          }
          float f = 1.f;
          if constexpr (kCoded && std::is_same_v<T, __nv_bfloat16>) {
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < D / 2; ++i) top = max(max(top, q[i] & 0x7FFFu), q[i] >> 16 & 0x7FFFu);
            int e = 0;
            if (top > 0 && top < 0x7F80u) e = 14 - ilogbf(__uint_as_float(top << 16));
            const float fa = scalbnf(1.f, e / 2), fb = scalbnf(1.f, e - e / 2);
#pragma unroll
            for (int i = 0; i < D / 2; ++i) {
              float x, y;
              widen2(q[i], x, y, __nv_bfloat16());
              q[i] = pack2(x * fa * fb, y * fa * fb, __half());
            }
            f = scalbnf(1.f, -e);
          }
          st_shared_f(base + F::kFq + row * 4, f * p.scale_log2);
#pragma unroll
          for (int i = 0; i < D / 32; ++i) tmem_st16(tmem + lanes + F::kQ + i * 16, q + i * 16);
          tmem_st_wait();
        }
        tc_fence_before();
      }
      named_bar_sync(1, 32 * kSoftWarps);
      if (lane == 0) mbar_arrive(q_full);
      const float fq = ld_shared_f(base + F::kFq + row * 4);

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
        const uint32_t side = base + F::kSideAt + stage * F::kSide;
        ok = ok && wait_bar(s_full + 8 * group, turn & 1u, p.status, kStatusTimeoutEpilogue);
        ok = ok && wait_bar(full + 8 * stage, phase, p.status, kStatusTimeoutEpilogue);
        tc_fence_after();
        if (busy) {
          float f[kKeys];
          tmem_ld32(my_s, f);
          tmem_ld32(my_s + 32, f + 32);
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(s_free + 8 * group);
          const int key0 = (walk.u0 + i) * kKeys;
          const uint2 valid = ld_shared_u2(side + F::kValid);
          const bool partial = (valid.x & valid.y) != 0xFFFFFFFFu || key0 + kKeys > seq.start;
          if constexpr (kCoded) {
            const F2 q2 = f2(fq);
#pragma unroll
            for (int j = 0; j < kKeys; j += 4) {
              const float4 ks = ld_shared_f4(side + j * 4);
              parts(mul2(f2(f[j], f[j + 1]), mul2(f2(ks.x, ks.y), q2)), f[j], f[j + 1]);
              parts(mul2(f2(f[j + 2], f[j + 3]), mul2(f2(ks.z, ks.w), q2)), f[j + 2], f[j + 3]);
            }
          } else {
            const F2 q2 = f2(fq);
#pragma unroll
            for (int j = 0; j < kKeys; j += 2) parts(mul2(f2(f[j], f[j + 1]), q2), f[j], f[j + 1]);
          }
          uint32_t seen[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
          if (partial) {
            const uint64_t all = seen_of(p, seq, token, key0);
            seen[0] = static_cast<uint32_t>(all) & valid.x;
            seen[1] = static_cast<uint32_t>(all >> 32) & valid.y;
#pragma unroll
            for (int j = 0; j < kKeys; ++j)
              if (!(seen[j >> 5] >> (j & 31) & 1)) f[j] = -INFINITY;
            if (kFormat != PROJ_KV_INT8 && key0 + kKeys > seq.start) {
#pragma unroll 1
              for (int j = 0; j < kKeys; j += 4) {
                uint32_t w;
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(side + F::kOdd + j));
                if (w == 0) continue;
                const uint32_t here = seen[j >> 5] >> (j & 31);
                odd |= (w & 0xFFu && here & 1u) || (w & 0xFF00u && here & 2u) ||
                       (w & 0xFF0000u && here & 4u) || (w & 0xFF000000u && here & 8u);
              }
            }
          }
          float top = f[0];
#pragma unroll
          for (int j = 1; j < kKeys; ++j) top = fmaxf(top, f[j]);
          float down = 1.f;
          if (top > ref + 6.f) {
            down = exp2_fast(ref - top);
            ref = top;
            sum *= down;
          }
          if constexpr (kCoded) {
            const float now = ld_shared_f(side + F::kRef);
            if (now != v_ref) {
              down *= v_ref / now;  // both powers of two, or v_ref 0 and nothing summed yet
              v_ref = now;
            }
          }
          // the group's products before: P is free, and O complete
          if (turn > 0) ok = ok && wait_bar(o_done + 8 * group, (turn - 1) & 1u, p.status, kStatusTimeoutEpilogue);
          tc_fence_after();
          if (i >= 2 && __any_sync(0xFFFFFFFFu, down != 1.f)) {
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
          const F2 low = f2(8.f - ref);
          F2 total = f2(0.f);
#pragma unroll
          for (int c = 0; c < kKeys; c += 32) {
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              float e[4];
              parts(add2(f2(f[c + j], f[c + j + 1]), low), e[0], e[1]);
              parts(add2(f2(f[c + j + 2], f[c + j + 3]), low), e[2], e[3]);
#pragma unroll
              for (int x = 0; x < 4; ++x) e[x] = exp2_fast(e[x]);
              total = add2(total, add2(f2(e[0], e[1]), f2(e[2], e[3])));
              if constexpr (kCoded) {
                const float4 vs = ld_shared_f4(side + F::kVScale + (c + j) * 4);
                parts(mul2(f2(e[0], e[1]), f2(vs.x, vs.y)), e[0], e[1]);
                parts(mul2(f2(e[2], e[3]), f2(vs.z, vs.w)), e[2], e[3]);
                if (partial) {
#pragma unroll
                  for (int x = 0; x < 4; ++x)
                    if (!(seen[c >> 5] >> (j + x) & 1)) e[x] = 0.f;
                }
              }
              w[j / 2] = pack2(e[0], e[1], C());
              w[j / 2 + 1] = pack2(e[2], e[3], C());
            }
            tmem_st16(my_p + c / 2, w);
          }
          float a, b;
          parts(total, a, b);
          sum += a + b;
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
      st_shared_f(ml + (group * 128 + row) * 12, ref - 8.f);
      st_shared_f(ml + (group * 128 + row) * 12 + 4, sum);
      st_shared_f(ml + (group * 128 + row) * 12 + 8, kCoded ? v_ref : 1.f);
      if (tiles > group) ok = ok && wait_bar(o_done + 8 * group, (turn - 1) & 1u, p.status, kStatusTimeoutEpilogue);
      // a value of V that is no finite number, seen by this row
      const bool any_odd = named_bar_sync_or(2, 32 * kSoftWarps, odd);
      tc_fence_after();
      if (busy) {
        float m[2], l[2], up[2];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          m[g] = ld_shared_f(ml + (g * 128 + row) * 12);
          l[g] = ld_shared_f(ml + (g * 128 + row) * 12 + 4);
          up[g] = ld_shared_f(ml + (g * 128 + row) * 12 + 8);
        }
        const float top = fmaxf(m[0], m[1]);
        const float f0 = exp2_fast(m[0] - top), f1 = exp2_fast(m[1] - top);
        const float all = l[0] * f0 + l[1] * f1;
        const float a0 = f0 * up[0], a1 = f1 * up[1];
        const bool whole = walk.u0 == 0 && walk.u1 == seq.units;
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (walk.u0 == 0 ? 1 : 0);
        float* part = p.part_o + (slot * kAttnTcRows + row) * D;
        constexpr int kCols = D / 2;  // each group writes half of the columns
#pragma unroll 1
        for (int c = group * kCols; c < (group + 1) * kCols; c += 16) {
          float o[16], o1[16];
          tmem_ld16(tmem + lanes + F::kO + c, o);
          if (tiles > 1) tmem_ld16(tmem + lanes + F::kO + D + c, o1);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) o[j] = tiles > 1 ? o[j] * a0 + o1[j] * a1 : o[j] * a0;
          if (kFormat != PROJ_KV_INT8 && any_odd && real) {
            // the drafts of this part once more: what is no finite number goes to
            // the rows that see it
            const int d0 = max(0, walk.u0 * kKeys - seq.start);
            const int d1 = min(seq.len - seq.start, walk.u1 * kKeys - seq.start);
            for (int d = d0; d < d1; ++d) {
              const bool sees = p.mask ? (d >> 5) < p.words && (p.mask[(seq.lo + token) * p.ldm + (d >> 5)] >> (d & 31) & 1)
                                       : d <= token;
              int id, spot;
              if (!sees || !page_of(p.c, walk.share.b, seq.start + d, id, spot)) continue;
              const uint8_t* v = p.c.v + entry_at(p.c, id, spot, walk.head).at;
              for (int j = 0; j < 16; ++j) {
                float x;
                if constexpr (kCoded)
                  x = (v[c + j] & 0x7F) == 0x7F ? __uint_as_float(0x7FC00000u) : 0.f;
                else
                  x = to_f32(reinterpret_cast<const T*>(v)[c + j]);
                if (!(fabsf(x) < INFINITY)) {
#pragma unroll
                  for (int y = 0; y < 16; ++y)
                    if (y == j) o[y] += x;
                }
              }
            }
          }
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const float v[4] = {o[j], o[j + 1], o[j + 2], o[j + 3]};
            if (real && whole)
              write_out<T>(p, seq.lo + token, head * D + c + j, v, all);
            else if (real)
              *reinterpret_cast<float4*>(part + c + j) = make_float4(v[0], v[1], v[2], v[3]);
          }
          __syncwarp();
        }
        if (real && group == 0) {
          if (whole) {
            if (p.lse) p.lse[static_cast<int64_t>(seq.lo + token) * p.heads + head] = lse_of(top, all);
          } else {
            *reinterpret_cast<float2*>(p.part_ml + (slot * kAttnTcRows + row) * 2) = make_float2(top, all);
          }
        }
      }
      tc_fence_before();
      // both groups are done with the item's Q, O and sums
      named_bar_sync(1, 32 * kSoftWarps);
      tc_fence_after();
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
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), Tc<D>::kSmem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(p.ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Tc<D>::kSmem;
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
