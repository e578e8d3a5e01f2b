// w4_tc.cu -- products with 4-bit weights for many tokens, on tcgen05.
//
// 128 weight rows are the M side of the MMA, up to TN tokens its N side.  The
// weights come to it through tensor memory: bulk copies bring them 4 bits wide
// to shared memory, decode warps turn them into pairs s (q - z), rounded to
// the type of x, and store those to tensor memory, from where the MMA reads
// its A operand -- so the 16-bit form of a weight never crosses shared memory,
// whose bandwidth is left to x (TN = 64: 16-byte copies of the tile's own rows
// by the decode warps; above: TMA; both in the 128-byte swizzle).
//
// The rounding of s (q - z) to 16 bits: the tensor cores take 16-bit
// operands, and the scale differs within the K of one accumulation, so it
// has to be applied before the MMA.  Many of the products are exact
// (q - z a power of two); the others add errors of the size of the
// output's own rounding.
//
// A CTA is persistent over items (token tile, 128-row tile); row tiles go
// fastest, so the CTAs that run together share the tokens of one expert.
// Roles (24 warps): 0 issues the copies of x, 1 those of the weights, 2 and 3
// MMAs, 4-11 drain accumulators, 12-23 decode (three groups of four warps, a
// group every third step, a warp 32 rows).  A role's loop runs in one or a few
// threads, at some five cycles an instruction; what a step and an item cost
// each of them is what the roles are split by.  Up to TN = 128 there are two
// accumulators, and each has its MMA warp and its four drain warps, which take
// the items in turn; at TN = 256 there is one, and the drain warps halve its
// columns.
// What bounds it: at few tokens the decode warps.  A pair of weights costs 0.75
// shifts, a mask-or, a subtraction and a multiplication, a step of 128 x 128
// some 350 issue slots of each scheduler, and waits come on top (a decode group
// asks for a step's x and waits for it within that step): a step takes about
// 1000 cycles, in which HBM would deliver more than twice its 8.5 KB.  (256
// experts of 8192 x 512 in groups of 32 with zeros, 8000 rows spread 1 / rank:
// 274 us, 2.83 TB/s of the 775 MB that it reads and writes;
// DRAM traffic is 742 MB, so nothing is read twice.)  At 256 tokens the MMAs
// and x: 64 KB of x a step from L2, eight MMAs of 128 x 256 x 16.  (8192 x
// 4096, 256 tokens: 18.8 us, 0.91 PFLOP/s, from L2 and from HBM alike.)
//
// Where there are few tiles, a cluster of C CTAs splits K, and the partial
// sums meet in rank order through distributed shared memory.
#include <cuda_runtime.h>

#include "cluster_common.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "splitk.cuh"
#include "vec.cuh"
#include "w4.h"
#include "w4_num.cuh"

namespace proj {
namespace {

constexpr int kDrainWarp = 4;    // first of eight
constexpr int kDecodeWarp = 12;  // first of 4 kGroups
constexpr int kGroups = 3;
constexpr int kThreads = 32 * (kDecodeWarp + 4 * kGroups);
constexpr int kTmemCols = 512;
constexpr int kTileTable = 1024;  // token tiles of experts that are looked up

// A step is 128 columns (two units): one hand-off each between the producers,
// the decode warps and the MMA warp, whose loops cost more than the work of
// 64 columns for few tokens.  Its weights: codes, scales, zeros (at most).
constexpr int kCodeBytes = 2 * kW4UnitBytes, kScaleBytes = 1024, kZeroBytes = 512;
constexpr int kWStage = kCodeBytes + kScaleBytes + kZeroBytes;

template <int TN>
struct Cfg {
  static constexpr int kHalf = TN * 128;          // x of one unit
  static constexpr int kStage = 2 * kHalf;
  // Few tokens: the decode warps copy x too, 16 bytes at a time and only the
  // tile's own rows, in the same stages as their A.  A tensor copy costs an
  // SM's copy engine some 75 ns per 32 rows of 64 columns, needed or not, and
  // the warp that issues it a round of waits per step: with it, tiles of a
  // dozen rows (the experts' down product of 1000 tokens) waited for x in
  // every step.
  static constexpr bool kRowCopies = TN == 64;
  // x in shared memory
  static constexpr int S = TN == 64 ? 6 : TN == 128 ? 4 : 3;
  static constexpr int SA = TN == 64 ? 6 : 3;     // A in tensor memory, 64 columns each
  static constexpr int SW = TN <= 128 ? 6 : 3;    // weights in shared memory
  // The decode groups take the steps in turn, and each waits for every phase
  // of its stages' barriers: both of their rings are multiples.
  static_assert(SA % kGroups == 0 && SW % kGroups == 0, "a stage belongs to one group");
  static constexpr int kAcc = TN <= 128 ? 2 : 1;
  static constexpr int kACol = kAcc * TN;         // behind the accumulators
  static constexpr int kBars = 2 * S + 2 * SA + 2 * SW + 6;
  static constexpr int kRing = S * kStage;        // the partial sums' staging afterwards
  static constexpr int kBarsAt = kRing + SW * kWStage;
  // rings, barriers, tensor-memory address, and for experts (TN up to 128) the
  // tile and row tables
  static constexpr int kTables = kBarsAt + kBars * 8 + 16;
  static constexpr int kSmem =
      1024 + kTables + (TN <= 128 ? (3 * kW4MaxExperts + 4) * 4 + kTileTable * 8 : 0);
  static_assert(!kRowCopies || S == SA, "x and A share their stages");
  static_assert(kACol + 64 * SA <= kTmemCols && TN * 512 <= kRing && kSmem <= 232448, "stages");
};

// A[16 rows x 64 columns] to tensor memory: lanes lane0 .. + 15, 32 columns.
// Register 4 i + 0, 1: row g, columns 8 i + 2 t, + 1; + 2, 3: row g + 8.
__device__ __forceinline__ void tmem_st_16x256b_x4(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Lane's row of 32 columns.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,"
      "%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// 16 bytes, of which `bytes` are read and the rest zeros.
__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}

__device__ __forceinline__ uint2 ld_shared_u2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t ld_shared_u16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}

// D[tmem] (+)= A[tmem] * B[smem desc]^T, kind::f16.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// True in one lane of a converged warp.  The compiler knows that code under
// it runs in one lane, and keeps the MMA's operands in uniform registers.
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

struct Item {
  int expert, row0, rows, rt;
};

// Items of this CTA's cluster in order: number cluster, + clusters, ...; item
// i is token tile i / RT, row tile i % RT.
struct Items {
  const int* pre;   // [E + 1] tiles before each expert (null: one matrix)
  const int* off;   // [E] first row
  const int* end;   // [E] row behind the last
  const int2* tile;  // by token tile: first row, expert << 9 | rows; or null: too many
  int tt, rt, step_t, step_r, RT, m;
  int e;
  __device__ __forceinline__ void begin(int first, int step) {
    tt = first / RT;
    rt = first - tt * RT;
    step_t = step / RT;
    step_r = step - step_t * RT;
    e = 0;
  }
  __device__ __forceinline__ void next() {
    tt += step_t;
    rt += step_r;
    if (rt >= RT) {
      rt -= RT;
      ++tt;
    }
  }
  template <int TN>
  __device__ __forceinline__ Item get() {
    Item it;
    it.rt = rt;
    if (tile) {
      const int2 v = tile[tt];
      it.row0 = v.x;
      it.rows = v.y & 511;
      it.expert = v.y >> 9;
    } else if (pre) {
      while (pre[e + 1] <= tt) ++e;
      it.expert = e;
      it.row0 = off[e] + (tt - pre[e]) * TN;
      it.rows = min(TN, end[e] - it.row0);
    } else {
      it.expert = 0;
      it.row0 = tt * TN;
      it.rows = min(TN, m - it.row0);
    }
    return it;
  }
};

template <typename T, bool kG32, bool kZeros, int TN>
__global__ void __launch_bounds__(kThreads, 1)
    w4_tc_kernel(const __grid_constant__ CUtensorMap tmap_x, const W4Params p, const int C,
                 const int box) {
  using F = Cfg<TN>;
  constexpr int S = F::S, SA = F::SA, SW = F::SW;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + F::kBarsAt);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + F::kBars);
  int* s_pre = reinterpret_cast<int*>(smem + F::kTables);
  int* s_off = s_pre + kW4MaxExperts + 1;
  int* s_end = s_off + kW4MaxExperts;
  int2* s_tile = reinterpret_cast<int2*>(s_end + kW4MaxExperts + 3);  // 8-byte aligned
  __shared__ int s_warp[kThreads / 32];

  const uint32_t ring = smem_u32(smem), wring = ring + F::kRing;
  const uint32_t xfull = smem_u32(bars), xempty = xfull + 8 * S;
  const uint32_t afull = xempty + 8 * S, aempty = afull + 8 * SA;
  const uint32_t wfull = aempty + 8 * SA, wempty = wfull + 8 * SW;
  const uint32_t accf = wempty + 8 * SW, acce = accf + 16, turn = acce + 16;
  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(blockIdx.x) % C;
  const int kb0 = static_cast<int>(static_cast<int64_t>(rank) * p.KU / C);
  const int kb1 = static_cast<int>(static_cast<int64_t>(rank + 1) * p.KU / C);
  const int steps = (kb1 - kb0 + 1) / 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(xfull + 8 * s, 1);
      mbar_init(xempty + 8 * s, 1);
    }
    for (int s = 0; s < SA; ++s) {
      mbar_init(afull + 8 * s, 4);  // decode warps
      mbar_init(aempty + 8 * s, 1);
    }
    for (int s = 0; s < SW; ++s) {
      mbar_init(wfull + 8 * s, 1);
      mbar_init(wempty + 8 * s, 4);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(accf + 8 * s, 1);
      mbar_init(acce + 8 * s, F::kAcc == 2 ? 128 : 256);
      mbar_init(turn + 8 * s, 1);
    }
    fence_mbar_init();
    if (!F::kRowCopies) prefetch_tmap(&tmap_x);
  }

  Items items;
  items.RT = p.RT;
  items.m = static_cast<int>(p.m);
  const int first = static_cast<int>(blockIdx.x) / C, step = static_cast<int>(gridDim.x) / C;
  items.begin(first, step);
  int all_items;
  if (p.offsets) {
    // tiles of each expert and the sums before it; offsets are clamped to
    // 0 .. m and taken as not decreasing, so no row outside x is named
    griddep_wait();
    constexpr int kPer = (kW4MaxExperts + kThreads - 1) / kThreads;
    int tiles[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = threadIdx.x * kPer + i;
      tiles[i] = 0;
      if (e < p.E) {
        const int lo = min(max(p.offsets[e], 0), items.m);
        const int hi = min(max(p.offsets[e + 1], lo), items.m);
        s_off[e] = lo;
        s_end[e] = hi;
        tiles[i] = (hi - lo + TN - 1) / TN;
      }
      sum += tiles[i];
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    int before = inc - sum;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w)
      if (w < warp) before += s_warp[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = threadIdx.x * kPer + i;
      if (e < p.E) {
        s_pre[e] = before;
        for (int k = 0; k < tiles[i] && before + k < kTileTable; ++k)
          s_tile[before + k] =
              make_int2(s_off[e] + k * TN, e << 9 | min(TN, s_end[e] - s_off[e] - k * TN));
        before += tiles[i];
        if (e == p.E - 1) s_pre[p.E] = before;
      }
    }
    __syncthreads();
    items.pre = s_pre;
    items.off = s_off;
    items.end = s_end;
    items.tile = s_pre[p.E] <= kTileTable ? s_tile : nullptr;
    // offsets that decrease all the same can claim rows twice: no more tiles are
    // worked on than the launch was planned for (with C > 1 one item a cluster)
    all_items = min(s_pre[p.E], min(p.E, items.m) + items.m / TN) * items.RT;
  } else {
    __syncthreads();  // the barriers are initialised
    items.pre = nullptr;
    items.off = nullptr;
    items.end = nullptr;
    items.tile = nullptr;
    all_items = (items.m + TN - 1) / TN * items.RT;
  }
  const int n_items = first < all_items ? (all_items - first + step - 1) / step : 0;

  // Every role passes the named barrier once its part of the set-up is done:
  // the barriers are initialised and the tensor memory is allocated.  Only then
  // may the stream's next kernel start beside this one (it might want tensor
  // memory too), and tensor memory is taken only when the kernel before has
  // completed (it might still have to allocate its own).
  if (warp == 0) {
    // --------------------------------------------------------- x producer
    griddep_wait();
    named_bar_sync(1, kThreads);
    int st = 0;
    uint32_t phase = 0;
    bool ok = !F::kRowCopies;
    for (int n = 0; n < n_items && ok; ++n, items.next()) {
      const Item im = items.get<TN>();
      const int boxes = (im.rows + box - 1) / box;
      const uint32_t bytes = static_cast<uint32_t>(boxes * box * 128);
      for (int kb = kb0; kb < kb1; kb += 2) {
        const int units = min(2, kb1 - kb);
        ok = __all_sync(0xFFFFFFFFu,
                        wait_bar(xempty + 8 * st, phase ^ 1u, p.status, kStatusTimeoutProducer));
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(xfull + 8 * st, bytes * units);
          for (int u = 0; u < units; ++u)
            for (int b = 0; b < boxes; ++b)
              tma_load_2d(ring + st * F::kStage + u * F::kHalf + b * box * 128, &tmap_x,
                          (kb + u) * 64, im.row0 + b * box, xfull + 8 * st);
        }
        __syncwarp();
        if (++st == S) {
          st = 0;
          phase ^= 1u;
        }
      }
    }
    // Every copy issued has to land before its buffer goes to other use: wait
    // until the MMAs have released each stage.
    for (int j = 0; j < S && !F::kRowCopies; ++j) {
      wait_bar(xempty + 8 * st, phase ^ 1u, p.status, kStatusTimeoutDrain);
      if (++st == S) {
        st = 0;
        phase ^= 1u;
      }
    }
  } else if (warp == 2 || warp == 3) {
    // ----------------------------------------------------------------- MMA
    griddep_wait();
    if (warp == 2) {
      tmem_alloc(smem_u32(tmem_slot), kTmemCols);
      tmem_relinquish();
    }
    tc_fence_before();
    named_bar_sync(1, kThreads);
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_launch_dependents();
    const int set = warp - 2;
    if (set) items.next();
    bool ok = true;
    for (int n = set; n < n_items && ok && set < F::kAcc; n += F::kAcc) {
      const Item im = items.get<TN>();
      for (int i = 0; i < F::kAcc; ++i) items.next();
      const uint32_t cols = static_cast<uint32_t>((im.rows + 15) & ~15);
      // D fp32, A and B K-major, M = 128, N = cols
      const uint32_t idesc =
          (1u << 4) | Num<T>::kIdescType | ((cols >> 3) << 17) | ((128u >> 4) << 24);
      ok = wait_bar(acce + 8 * set, static_cast<uint32_t>((n / F::kAcc) & 1) ^ 1u, p.status,
                    kStatusTimeoutMma);
      // A wait tells a phase from the one before it only, so the stages are
      // waited for in order: this warp's turn comes when the other has issued
      // the whole item before.
      if (F::kAcc == 2 && n > 0)
        ok = ok && wait_bar(turn + 8 * set, static_cast<uint32_t>(((n - 1) / 2) & 1), p.status,
                            kStatusTimeoutMma);
      tc_fence_after();
      const uint32_t d = tmem + set * TN;
      int it = n * steps;
      for (int step = 0; step < steps; ++step, ++it) {
        const int st = it % S, sa = it % SA;
        ok = __all_sync(0xFFFFFFFFu, ok &&
                            (F::kRowCopies ||
                             wait_bar(xfull + 8 * st, static_cast<uint32_t>((it / S) & 1),
                                      p.status, kStatusTimeoutMma)) &&
                            wait_bar(afull + 8 * sa, static_cast<uint32_t>((it / SA) & 1), p.status,
                                     kStatusTimeoutMma));
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t a = tmem + F::kACol + sa * 64;
          const uint64_t b = smem_desc_sw128(ring + st * F::kStage);
#pragma unroll
          for (int k = 0; k < 4; ++k)  // 16 columns: 8 of tensor memory, 32 bytes of x
            mma_ts(d, a + 8 * k, b + 2 * k, idesc, (step > 0 || k > 0) ? 1u : 0u);
          if (kb0 + 2 * step + 1 < kb1) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ts(d, a + 32 + 8 * k, b + (F::kHalf >> 4) + 2 * k, idesc, 1u);
          }
          if (!F::kRowCopies) tc_commit(xempty + 8 * st);
          tc_commit(aempty + 8 * sa);
          if (step == steps - 1) {
            tc_commit(accf + 8 * set);
            if (F::kAcc == 2) mbar_arrive(turn + 8 * (set ^ 1));
          }
        }
        __syncwarp();
      }
    }
  } else if (warp >= kDrainWarp && warp < kDecodeWarp) {
    // ------------------------------------------------------ accumulators
    griddep_wait();
    named_bar_sync(1, kThreads);
    tc_fence_after();
    const int q = warp & 3, set = (warp - kDrainWarp) >> 2;
    // both sets on every item, a half of its columns each, or items in turn
    const bool halves = F::kAcc == 1 || C > 1;
    const int stride = halves ? 1 : 2;
    if (!halves && set) items.next();
    const uint32_t lanes = *tmem_slot + (static_cast<uint32_t>(32 * q) << 16);
    const int ldo = static_cast<int>(p.ldo);
    for (int n = halves ? 0 : set; n < n_items; n += stride) {
      const Item im = items.get<TN>();
      for (int i = 0; i < stride; ++i) items.next();
      const int buf = n % F::kAcc;
      if (!wait_bar(accf + 8 * buf, static_cast<uint32_t>((n / F::kAcc) & 1), p.status,
                    kStatusTimeoutEpilogue))
        break;
      tc_fence_after();
      const int r = 32 * q + lane;  // row of the tile
      const int row = im.rt * 128 + r;
      T* out = static_cast<T*>(p.out) + static_cast<int64_t>(im.row0) * p.ldo + row;
      for (int c0 = halves ? 32 * set : 0; c0 < im.rows; c0 += halves ? 64 : 32) {
        // columns behind the last row's are not used, whatever they hold
        float v[32];
        tmem_ld32(lanes + buf * TN + c0, v);
        tmem_ld_wait();
        if (C > 1) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            st_shared_f32(ring + static_cast<uint32_t>(((c0 + j) * 128 + r) * 4), v[j]);
        } else {
          T* at = out + static_cast<int64_t>(c0) * ldo;
          const int left = row < p.N ? im.rows - c0 : 0;
#pragma unroll
          for (int j8 = 0; j8 < 32; j8 += 8) {
            if (im.rows - c0 <= j8) break;
#pragma unroll
            for (int j = j8; j < j8 + 8; ++j)
              if (j < left) at[static_cast<int64_t>(j) * ldo] = from_f32<T>(v[j]);
          }
        }
      }
      tc_fence_before();
      mbar_arrive(acce + 8 * buf);
    }
  } else if (warp == 1) {
    // --------------------------------------------------- weights' producer
    // The weights are constant: their copies need not wait for the kernel
    // before (with experts' offsets, everything here came after that wait).
    const uint64_t pol = policy_evict_first();
    int st = 0;
    uint32_t phase = 0;
    bool ok = true, synced = false;
    int ahead = 0;  // steps issued before the barrier: as many as there are stages
    for (int n = 0; n < n_items && ok; ++n, items.next()) {
      const Item im = items.get<TN>();
      const int64_t tile = static_cast<int64_t>(im.expert) * items.RT + im.rt;
      const uint8_t* codes = reinterpret_cast<const uint8_t*>(p.codes) +
                             (tile * p.KU + kb0) * kW4UnitBytes;
      for (int kb = kb0; kb < kb1; kb += 2, codes += kCodeBytes) {
        const int units = min(2, kb1 - kb);
        const int g0 = kG32 ? 2 * kb : p.group_of(kb);
        const int groups = kG32 ? 2 * units : p.group_of(kb + units - 1) - g0 + 1;
        if (!synced && ahead++ == SW) {
          named_bar_sync(1, kThreads);
          synced = true;
        }
        ok = __all_sync(0xFFFFFFFFu,
                        wait_bar(wempty + 8 * st, phase ^ 1u, p.status, kStatusTimeoutProducer));
        if (!ok) break;
        if (elect_one()) {
          const uint32_t bar = wfull + 8 * st, dst = wring + st * kWStage;
          mbar_arrive_expect_tx(bar, units * kW4UnitBytes + groups * (kZeros ? 384 : 256));
          bulk_g2s(dst, codes, units * kW4UnitBytes, bar, pol);
          const int64_t row = (tile * p.NGp + g0) * 128;
          bulk_g2s(dst + kCodeBytes, p.scales + row, groups * 256, bar, pol);
          if (kZeros) bulk_g2s(dst + kCodeBytes + kScaleBytes, p.zeros + row, groups * 128, bar, pol);
        }
        __syncwarp();
        if (++st == SW) {
          st = 0;
          phase ^= 1u;
        }
      }
    }
    if (!synced) named_bar_sync(1, kThreads);
    for (int j = 0; j < SW; ++j) {  // the copies issued have landed and been read
      wait_bar(wempty + 8 * st, phase ^ 1u, p.status, kStatusTimeoutDrain);
      if (++st == SW) {
        st = 0;
        phase ^= 1u;
      }
    }
  } else {
    // -------------------------------------------------------------- decode
    const int gi = (warp - kDecodeWarp) >> 2;  // steps gi, gi + kGroups, ... of the sequence
    const int q = warp & 3;
    const int g = lane >> 2;
    const int total = n_items * steps;
    if (F::kRowCopies) griddep_wait();  // these warps read x
    named_bar_sync(1, kThreads);
    tc_fence_after();
    const uint32_t a0 = *tmem_slot + (static_cast<uint32_t>(32 * q) << 16) + F::kACol;
    int step = gi;  // within the item
    while (step >= steps) {
      step -= steps;
      items.next();
    }
    Item im = {};
    if (F::kRowCopies && gi < total) im = items.get<TN>();
    // x: of the two units' 16 pieces of a row the (thread % 16)th, of every
    // eighth row; what K cuts off is filled with zeros
    const int piece = threadIdx.x & 15;
    const int r0 = static_cast<int>(threadIdx.x - 32 * kDecodeWarp) % 128 / 16;
    for (int it = gi; it < total; it += kGroups) {
      const int sa = it % SA, sw = it % SW;
      if constexpr (F::kRowCopies) {
        if (!wait_bar(aempty + 8 * sa, static_cast<uint32_t>((it / SA) & 1) ^ 1u, p.status,
                      kStatusTimeoutDecode))
          break;
        const int unit = kb0 + 2 * step + (piece >> 3);
        const int col = unit * 64 + (piece & 7) * 8;
        const int bytes = min(16, max(0, 2 * (p.K - col)));
        const char* from = static_cast<const char*>(p.x) +
                           2 * ((static_cast<int64_t>(im.row0) + r0) * p.ldx + (bytes ? col : 0));
        const uint32_t to = ring + sa * F::kStage + (piece >> 3) * F::kHalf;
        if (unit < kb1) {
          // rows 8 apart sit alike in the swizzle
          const uint32_t swizzled = to + r0 * 128 + (((piece ^ r0) & 7) << 4);
          for (int i = 0; i < im.rows - r0; i += 8, from += 16 * p.ldx)
            cp_async16_zfill(swizzled + i * 128, from, bytes);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      }
      if (!wait_bar(wfull + 8 * sw, static_cast<uint32_t>((it / SW) & 1), p.status,
                    kStatusTimeoutDecode))
        break;
      const int kb = kb0 + 2 * step;
      const int units = min(2, kb1 - kb);
      const uint32_t src = wring + sw * kWStage;
      bool ok = true;
#pragma unroll 1
      for (int u = 0; u < units; ++u) {
        uint4 code[2];
        uint32_t sc[2][2], ze[2][2];  // [row block][half]
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int rb = 2 * q + j;
          code[j] = ld_shared_u4(src + u * kW4UnitBytes + rb * 512 + lane * 16);
          if (kG32) {
            const uint32_t at = (u * 8 + rb) * 8 + g;
            const uint2 v = ld_shared_u2(src + kCodeBytes + 8 * at);
            sc[j][0] = v.x;
            sc[j][1] = v.y;
            if (kZeros) {
              ze[j][0] = ld_shared_u32(src + kCodeBytes + kScaleBytes + 4 * at);
              ze[j][1] = ze[j][0] >> 16;
            }
          } else {
            const uint32_t at = ((p.group_of(kb + u) - p.group_of(kb)) * 8 + rb) * 8 + g;
            sc[j][0] = sc[j][1] = ld_shared_u32(src + kCodeBytes + 4 * at);
            if (kZeros)
              ze[j][0] = ze[j][1] = ld_shared_u16(src + kCodeBytes + kScaleBytes + 2 * at);
          }
        }
        if (u == 0 && !F::kRowCopies) {
          ok = wait_bar(aempty + 8 * sa, static_cast<uint32_t>((it / SA) & 1) ^ 1u, p.status,
                        kStatusTimeoutDecode);
          tc_fence_after();
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t word[4] = {code[j].x, code[j].y, code[j].z, code[j].w};
          uint32_t r[16];
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
              const uint32_t zero = zero_pair<T>(kZeros ? ze[j][h] : 0x0808u, hi);
              const uint32_t s = __byte_perm(sc[j][h], 0u, hi ? 0x3232 : 0x1010);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                r[(2 * h + (i >> 1)) * 4 + 2 * hi + (i & 1)] =
                    Num<T>::mul(code_pair<T>(word[2 * h + hi], i, zero), s);
            }
          tmem_st_16x256b_x4(a0 + (static_cast<uint32_t>(16 * j) << 16) + sa * 64 + 32 * u, r);
        }
      }
      tmem_st_wait();
      if constexpr (F::kRowCopies) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        fence_proxy_async_smem();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(wempty + 8 * sw);
        mbar_arrive(afull + 8 * sa);
      }
      if (!ok) break;
      step += kGroups;
      if (step >= steps) {
        do {
          step -= steps;
          items.next();
        } while (step >= steps);
        if (F::kRowCopies && it + kGroups < total) im = items.get<TN>();
      }
    }
  }
  __syncwarp();
  if (C > 1) {
    // One item per cluster: the partial sums stand in the rings; rank r sums
    // its share of the tokens, in rank order.
    cluster_sync_all();
    griddep_wait();
    items.begin(first, step);
    if (n_items) {
      const Item im = items.get<TN>();
      const int j0 = im.rows * rank / C, j1 = im.rows * (rank + 1) / C;
      const int n = (j1 - j0) * 32;
      for (int base = threadIdx.x; base < n; base += 4 * kThreads) {
        // four items in flight: a round trip to another CTA's memory is long
        float4 sum[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) sum[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = 0; c < C; ++c) {
          const uint32_t peer = map_to_rank(ring, static_cast<uint32_t>(c));
          float4 v[4];
#pragma unroll
          for (int u = 0; u < 4; ++u)
            v[u] = ld_dsmem_v4(peer + 16 * (j0 * 32 + min(base + u * kThreads, n - 1)));
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            sum[u].x += v[u].x;
            sum[u].y += v[u].y;
            sum[u].z += v[u].z;
            sum[u].w += v[u].w;
          }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int i = base + u * kThreads;
          if (i >= n) break;
          const float v[4] = {sum[u].x, sum[u].y, sum[u].z, sum[u].w};
          const int64_t row = static_cast<int64_t>(im.rt) * 128 + i % 32 * 4;
          T* out = static_cast<T*>(p.out) + (im.row0 + j0 + i / 32) * p.ldo + row;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (row + j < p.N) out[j] = from_f32<T>(v[j]);
        }
      }
    }
    cluster_sync_all();  // no CTA leaves while another reads its partial sums
  } else {
    __syncthreads();
  }
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(*tmem_slot, kTmemCols);
  }
}

template <typename T, bool kG32, bool kZeros, int TN>
cudaError_t launch(const CUtensorMap& map, const W4Params& p, int grid, int C, int box,
                   cudaStream_t s) {
  auto kernel = w4_tc_kernel<T, kG32, kZeros, TN>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), Cfg<TN>::kSmem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<TN>::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(C);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, map, p, C, box);
}

template <typename T, int TN>
cudaError_t launch_form(const CUtensorMap& map, const W4Params& p, int grid, int C, int box,
                        cudaStream_t s) {
  if (p.group == 32)
    return p.zeros ? launch<T, true, true, TN>(map, p, grid, C, box, s)
                   : launch<T, true, false, TN>(map, p, grid, C, box, s);
  return p.zeros ? launch<T, false, true, TN>(map, p, grid, C, box, s)
                 : launch<T, false, false, TN>(map, p, grid, C, box, s);
}

template <typename T>
cudaError_t launch_any(int tn, const CUtensorMap& map, const W4Params& p, int grid, int C, int box,
                       cudaStream_t s) {
  switch (tn) {
    case 64: return launch_form<T, 64>(map, p, grid, C, box, s);
    case 128: return launch_form<T, 128>(map, p, grid, C, box, s);
    default: return launch_form<T, 256>(map, p, grid, C, box, s);
  }
}

}  // namespace

cudaError_t w4_tc_launch(bool fp16, int tn, const W4Params& p, int64_t grid, int C,
                         cudaStream_t s) {
  CUtensorMap map = {};
  // An expert's rows are few: boxes of 32 keep the rows behind them out.  One
  // matrix has whole tiles, and a copy's issue costs more than its rows.
  int box = 32;
  while (!p.offsets && box < tn && box < p.m) box *= 2;
  if (tn != 64 && !make_rows_map(&map, p.x, p.m, p.K, p.ldx, fp16, box))
    return cudaErrorInvalidValue;
  const int n = static_cast<int>(grid);
  return fp16 ? launch_any<__half>(tn, map, p, n, C, box, s)
              : launch_any<__nv_bfloat16>(tn, map, p, n, C, box, s);
}

int w4_tc_max_clusters(int C) {
  // every form takes an SM to itself: one stands for all
  auto kernel = w4_tc_kernel<__nv_bfloat16, false, false, 256>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<256>::kSmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(C);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           Cfg<256>::kSmem) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

}  // namespace proj
