/*
 * proj.h -- C ABI of libproj: weight-bandwidth-bound dense projections on
 * GB300 (sm_103a).
 *
 * The operation (muse_bf16_proj guide, ch. 1, §1.1 "What is computed"):
 *
 *     out[i, n] = sum over k of x[i, k] * W[n, k]        (out = x @ W.T, no bias)
 *
 * for five fixed layers (§1.1 table):
 *
 *     layer      N x K         W dtype   out dtype
 *     qkv_gate   2304 x 8192   bf16      bf16
 *     o          8192 x 1024   bf16      bf16
 *     pooler     4096 x 8192   bf16      bf16
 *     unpooler   8192 x 4096   bf16      bf16   (only rows 0..1023 at m <= 8)
 *     router      256 x 8192   fp32      fp32
 *
 * Accumulation is in fp32; the dense layers round the fp32 sum to bf16
 * (round-to-nearest-even) on output.  The router keeps fp32 weights and an
 * fp32 sum: at every token count the dispatch runs it on the CUDA cores, the
 * bf16 input (widened exactly) meeting the fp32 weights in fp32 fused
 * multiply-adds (no TF32 truncation anywhere).  On request only
 * (PROJ_VARIANT_PLANES3) the router runs on the tensor cores instead, its
 * weights split at prepare into three bf16 planes with hi + mid + lo == W
 * exactly, so every product x * plane is exact and only the fp32
 * accumulation rounds.
 *
 * Interface shape (guide ch. 1, §1.6 "Rules that shaped the code"):
 * prepare(weights) runs once, untimed, and may repack or losslessly recode
 * W; the timed call is replayed as a CUDA graph, so it branches on shapes
 * only, performs no host synchronisation, no allocation and no memset, and
 * caches nothing derived from x.  Split-K bookkeeping is reset on the GPU.
 *
 * Threading: a handle is not thread-safe and must not run on two streams
 * at the same time (its split-K workspace and counters are shared by calls).
 * Different handles are independent.
 *
 * Errors: every call validates its arguments before touching the GPU and
 * returns a proj_status (or NULL + proj_last_status() for constructors).
 * A CUDA error raised while enqueuing maps to PROJ_ECUDA.  Nothing aborts
 * the process and no C++ exception crosses this boundary.
 */
#ifndef PROJ_H_
#define PROJ_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Opaque, library-owned state of one prepared layer. */
typedef struct proj_ctx *proj_handle;

/* A CUDA stream (cudaStream_t / CUstream).  NULL means the legacy default
 * stream of the calling thread. */
typedef struct CUstream_st *proj_stream;

enum proj_layer {
    PROJ_QKV_GATE = 0,
    PROJ_O = 1,
    PROJ_POOLER = 2,
    PROJ_UNPOOLER = 3,
    PROJ_ROUTER = 4
};

/* PROJ_FP16 serves the 4-bit products, the expert sort and the norms below; the
 * five layers keep PROJ_BF16 and PROJ_FP32. */
enum proj_dtype { PROJ_BF16 = 0, PROJ_FP32 = 1, PROJ_FP16 = 2 };

enum proj_flags {
    /* Also keep a lossless 12-bit exponent-window copy of a bf16 W and use
     * it for the token counts its kernel covers (project report, "Round 5 --
     * lossless 12-bit compressed weights", "Format"): per weight the raw low
     * byte plus a 4-bit (sign, 3-bit window code) field; the 8 window values
     * of the 7 high exponent bits are chosen per matrix to cover the most
     * weights; weights outside the window are restored exactly from a
     * per-tile escape list.  Results are bit-identical to the uncompressed
     * kernel.  If any tile holds more escapes than the format's per-tile
     * capacity, the encoding is declined and the handle runs uncompressed
     * (proj_info reports it).  Where K is a multiple of 1024 (<= 8192) a
     * second 12-bit copy in 1024-column row chunks (same window, escapes per
     * chunk, at most 7, else that copy is declined) serves the register GEMV
     * at m <= 2, and the same format over the warp-MMA GEMV's fragment-order
     * copy serves that GEMV from 3 tokens; both are bit-identical to their
     * dense forms, and proj_describe_ex names them "expwin12rc". */
    PROJ_ENCODE_EXPWIN12 = 1u << 0
};

enum proj_status {
    PROJ_OK = 0,
    PROJ_EINVAL = 1,        /* bad argument (NULL, wrong shape or dtype, m < 0) */
    PROJ_EUNSUPPORTED = 2,  /* valid request this build does not serve (m > m_max) */
    PROJ_EALIGN = 3,        /* a pointer is not 16-byte aligned */
    PROJ_ENOMEM = 4,        /* device or host allocation failed (prepare only) */
    PROJ_ECUDA = 5,         /* a CUDA call failed; see proj_last_cuda_error() */
    PROJ_EDEVICE = 6        /* a kernel reported a fault in its status word */
};

/* Variant selection for proj_run_ex (testing and tuning). */
enum proj_variant {
    PROJ_VARIANT_AUTO = 0,      /* the dispatch table's choice */
    PROJ_VARIANT_DENSE = 1,     /* uncompressed weights */
    PROJ_VARIANT_EXPWIN12 = 2,  /* 12-bit weights (handle must hold them): the row-chunk
                                   copy on the register GEMV at m <= 2, the recoded
                                   fragment copy on the warp-MMA GEMV where x fits its
                                   shared memory (m <= 32), else the tile records on the
                                   tensor cores (stream-K tile kernel, token tiles of
                                   at most 128: any m); each where it was built */
    PROJ_VARIANT_PLANES3 = 3    /* router only: the fp32 weights as three bf16 planes,
                                   hi + mid + lo == W exactly, on the tensor cores */
};

/* How CTAs sharing a tile combine their fp32 partials (both deterministic:
 * the summation order depends only on the partition). */
enum proj_reduce {
    PROJ_REDUCE_AUTO = 0,        /* the dispatch table's choice */
    PROJ_REDUCE_OWNER = 1,       /* the CTA holding the tile's first k-range sums
                                    the others' partials (small m) */
    PROJ_REDUCE_DISTRIBUTED = 2  /* every contributor sums 1/S of the tile */
};

/* Kernel family for proj_run_ex (testing and tuning). */
enum proj_kernel {
    PROJ_KERNEL_AUTO = 0,   /* the dispatch table's choice */
    PROJ_KERNEL_GEMV = 1,   /* row-streaming CUDA-core GEMV, m <= 2 */
    PROJ_KERNEL_TILE = 2,   /* tiled kernels: tensor cores (bf16) / FMA tiles (router),
                               split-K across CTAs through global memory */
    PROJ_KERNEL_MMA = 5,    /* bf16 layers, m <= 32 (as far as x fits shared memory: K <=
                               8192 / 4096 / 1024 at 8 / 16 / 32 tokens): weight-streaming
                               GEMV on the warp-level tensor-core MMA (mma.sync m16n8k16)
                               from a copy of W in fragment order; CTAs own whole 16-row
                               blocks (at most 4), proj_run_opts.grid = CTAs; the dispatch
                               form at 3 <= m <= 8 (not the pooler) and on o to 16 */
    PROJ_KERNEL_GEMV_REG = 4, /* m <= 2 (the router: m <= 16): CUDA-core GEMV with the
                                 weights loaded straight into registers, whole rows per
                                 CTA (PROJ_KERNEL_GEMV: through a shared-memory ring fed
                                 by bulk copies); for the router at 3 <= m <= 16, FP32
                                 FMAs with x in passes of eight tokens (the dispatch
                                 form at 3 <= m <= 8) */
    PROJ_KERNEL_GEMV_SPLITK = 6, /* router, m <= 32: the FP32-FMA weight-streaming GEMV with K
                                    split across a thread-block cluster (K / 1024 CTAs, one
                                    1024-column chunk of eight rows each, x staged per CTA for
                                    its chunk only), partials summed in rank order through
                                    distributed shared memory; the dispatch form at
                                    9 <= m <= 24; PROJ_EUNSUPPORTED elsewhere */
    PROJ_KERNEL_CLUSTER = 3, /* tensor cores (dense bf16 weights; the router's bf16 planes),
                               split-K inside a thread-block cluster combined through
                               distributed shared memory, and optionally across several
                               clusters per tile through global memory:
                               proj_run_opts.grid = cluster size (1..16),
                               proj_run_opts.groups = clusters per tile (1..8) */
    PROJ_KERNEL_ROWS = 8,   /* bf16 layers, m <= 32: weight-streaming GEMV on the warp-level
                               tensor-core MMA over whole row runs per CTA (CTA c of
                               proj_run_opts.grid, default the SM count, owns rows
                               [c N / grid, (c + 1) N / grid), at most 64), W and x
                               brought from their row-major layouts into a shared-memory
                               ring by tensor copies; proj_run_opts.groups = 32-column
                               steps per ring stage (a power of two dividing K / 32, at
                               most 64; 0 = chosen for the most bytes in flight);
                               PROJ_EUNSUPPORTED elsewhere */
    PROJ_KERNEL_PAIR = 7    /* bf16 layers (dense weights): tensor cores on CTA pairs
                               (tcgen05 cta_group::2, 256 weight rows per MMA, each CTA
                               holding half of the token tile's x), K split across
                               proj_run_opts.groups pairs per 256-row tile (1..8; 0 = cost
                               model), one thread-block cluster of 2 x groups CTAs whose
                               partials meet in L2; proj_run_opts.tile_n = 64, 128 or 256
                               tokens per tile; grid and reduce must be 0; groups > 1
                               needs the grid within one CTA per SM (the partials'
                               exchange is sized for that), else PROJ_EUNSUPPORTED; the
                               dispatch form on o above 128 tokens and on the unpooler
                               from 192 */
};

typedef struct proj_run_opts {
    int variant;    /* enum proj_variant */
    int grid;       /* CTAs of the partition (1 .. SMs), or the cluster size for
                       PROJ_KERNEL_CLUSTER; 0 = dispatch table */
    int reduce;     /* enum proj_reduce (tiled kernels); owner needs m <= 32 on bf16 */
    int kernel;     /* enum proj_kernel */
    int groups;     /* PROJ_KERNEL_CLUSTER: clusters sharing one output tile's K
                       (1..16); PROJ_KERNEL_PAIR: pairs sharing one 256-row tile's K
                       (1..8); 0 = dispatch table */
    int tile_n;     /* token tile width of the tensor-core kernels (16, 32, 64, 128
                       or 256; the 12-bit kernel 16 or 32); 0 = dispatch table */
    void *stamps;   /* optional, for measurement: a device buffer of 8 uint64 per
                       CTA of the launch that the row-run kernel (PROJ_KERNEL_ROWS)
                       and the tensor-core cluster and CTA-pair kernels fill with
                       %globaltimer readings (ns): [0] entry, [1] the wait on the
                       previous kernel of the stream passed, [2] first stage landed
                       (tensor-core issuer), [3] last MMA issued, [4] accumulator
                       complete, [5] accumulator staged (row-run: main loop done),
                       [6] past the cluster barrier before the combine, [7] exit;
                       slots a kernel has no phase for are left as they are;
                       NULL = none; ignored by the other kernels */
} proj_run_opts;

typedef struct proj_info_t {
    int layer;               /* enum proj_layer */
    int dtype;               /* enum proj_dtype of W */
    int64_t N, K;
    int64_t m_max;
    int expwin12;            /* 1 if the 12-bit copy is present and used */
    int expwin12_declined;   /* 1 if requested but declined (escape overflow) */
    int expwin12_e0;         /* window base: high7 in [e0, e0 + 7] */
    int64_t expwin12_escapes;        /* weights outside the window */
    int64_t expwin12_bytes;          /* bytes of the 12-bit stream incl. escapes */
    int64_t dense_bytes;             /* bytes of the packed uncompressed W */
    int64_t workspace_bytes;         /* split-K partials + counters */
    int num_sms;
    int reserved[7];
} proj_info_t;

/*
 * Prepare a layer.  Untimed; may allocate and synchronise.
 *   layer : enum proj_layer.
 *   W     : device pointer to row-major [N, K] weights, 16-byte aligned;
 *           bf16 for every layer but the router, fp32 for the router.  It is
 *           only read, and fully consumed before return: the caller may free
 *           it afterwards.
 *   N, K  : must equal the layer's fixed shape (table above).
 *   dtype : PROJ_FP32 for the router, PROJ_BF16 otherwise.
 * Returns NULL on error; proj_last_status() then says why.
 */
proj_handle proj_prepare(int layer, const void *W, int64_t N, int64_t K, int dtype);

/*
 * As proj_prepare, plus:
 *   flags  : enum proj_flags.
 *   m_max  : largest token count proj_run will be called with; sizes the
 *            workspace.  0 selects the default, 1024.
 *   status : optional out-parameter (may be NULL).
 */
proj_handle proj_prepare_ex(int layer, const void *W, int64_t N, int64_t K, int dtype,
                            uint32_t flags, int64_t m_max, int *status);

/*
 * Timed call.  Enqueues the projection on `stream` and returns; no
 * allocation, no host synchronisation, no memset; capturable in a CUDA graph.
 * Branches on m only.
 *   x   : device pointer, bf16 row-major [m, K], contiguous, 16-byte aligned.
 *   m   : token count, 0 <= m <= m_max (m = 0 returns PROJ_OK, no launch).
 *   out : device pointer, row-major [m, proj_out_features(h, m)], contiguous,
 *         16-byte aligned; bf16 for the dense layers, fp32 for the router.
 *         Every element is written.
 * x and out must not overlap.  Returns PROJ_OK or an error status.
 */
int proj_run(proj_handle h, const void *x, int64_t m, void *out, proj_stream stream);

/* proj_run with an explicit variant and split-K grid (opts may be NULL). */
int proj_run_ex(proj_handle h, const void *x, int64_t m, void *out, proj_stream stream,
                const proj_run_opts *opts);

/*
 * End-to-end call on HOST buffers: copies x_host [m, K] bf16 to a
 * handle-owned device buffer, runs the projection, and delivers the result to
 * out_host [m, proj_out_features(h, m)], all enqueued on `stream`.  For a
 * page-locked x_host (16-byte aligned) the copy in is a copy kernel reading
 * the buffer's device mapping; for a page-locked out_host the projection
 * kernel stores the result straight into its device mapping (every element
 * written once, as on device memory); other host memory goes through
 * cudaMemcpyAsync and a handle-owned staging buffer (asynchronous only for
 * page-locked memory).  The caller synchronises `stream` before reading
 * out_host.  Same m rules as proj_run.
 */
int proj_run_host(proj_handle h, const void *x_host, int64_t m, void *out_host,
                  proj_stream stream);

/* Output width at m tokens: N, except the unpooler's 1024 at m <= 8
 * (guide ch. 1, §1.1 table).  Returns -1 for a NULL handle. */
int64_t proj_out_features(proj_handle h, int64_t m);

/* Fill *info with the handle's facts.  Returns PROJ_OK or PROJ_EINVAL. */
int proj_info(proj_handle h, proj_info_t *info);

/*
 * Describe the kernel and launch shape proj_run would use at m (for
 * reports): writes a NUL-terminated string of at most `cap` bytes to `buf`.
 */
int proj_describe(proj_handle h, int64_t m, char *buf, size_t cap);

/* The same for proj_run_ex with these options (opts may be NULL): the kernel
 * and launch shape that call would use, or the status it would refuse with
 * (PROJ_EINVAL / PROJ_EUNSUPPORTED, nothing written). */
int proj_describe_ex(proj_handle h, int64_t m, const proj_run_opts *opts, char *buf, size_t cap);

/*
 * Decode the handle's packed weights back to row-major [N, K] at W_out
 * (device, same dtype as prepared).  With the 12-bit copy present it
 * decodes that copy, so a bitwise comparison with the original W checks
 * that the recode is lossless.  For the router, PROJ_VARIANT_PLANES3 sums
 * the three bf16 planes back to fp32 (the same check for the plane split).
 * variant = PROJ_UNPACK_FRAG16 decodes the bf16 layers' copy in warp-MMA
 * fragment order (the few-token GEMV's layout; PROJ_EUNSUPPORTED where it
 * was not built), and variant = PROJ_UNPACK_RC12 the 12-bit row-chunk copy
 * (bf16 layers with PROJ_ENCODE_EXPWIN12; PROJ_EUNSUPPORTED where it was
 * not built or was declined), and variant = PROJ_UNPACK_FRAG12 the 12-bit
 * recode of the fragment-order copy (same conditions; it uses a temporary
 * device buffer of N x K bf16 and synchronises `stream`).  variant =
 * PROJ_UNPACK_RUNS decodes the row-run copy of the few-token GEMV
 * (PROJ_KERNEL_ROWS: each CTA's rows as [K / 32 steps][rows][32 columns])
 * into all N rows, and PROJ_UNPACK_RUNS_SLICE the unpooler's copy of its
 * first 1024 rows into [1024, K] (PROJ_EUNSUPPORTED where not built).
 * Otherwise enqueued on `stream`.
 */
#define PROJ_UNPACK_FRAG16 16
#define PROJ_UNPACK_RC12 32
#define PROJ_UNPACK_FRAG12 64
#define PROJ_UNPACK_RUNS 128
#define PROJ_UNPACK_RUNS_SLICE 256
int proj_unpack_weights(proj_handle h, int variant, void *W_out, proj_stream stream);

/* Read and clear the handle's device status word (synchronises `stream`).
 * Returns PROJ_OK or PROJ_EDEVICE; *code receives the raw word if non-NULL. */
int proj_device_status(proj_handle h, proj_stream stream, uint32_t *code);

/* Free everything the handle owns (synchronises the device first). */
void proj_destroy(proj_handle h);

/* Status of the last failing call on this thread, and its text. */
int proj_last_status(void);
const char *proj_status_string(int status);
/* Last error text recorded on this thread: a CUDA error, or the reason an
 * argument was rejected ("" if none). */
const char *proj_last_cuda_error(void);

/*
 * Streaming read of `bytes` bytes at device pointer `buf` (16-byte aligned,
 * bytes a multiple of 16), with every byte reaching the SMs: the HBM read
 * floor of the timing harness, and, on a buffer larger than L2, the flush
 * that makes the next call cold.  Writes one 32-bit checksum per CTA to
 * `sink` (device, >= grid + 1 words; the last one is a status word).
 * grid = 0 picks two CTAs per SM for mode 0 and one for mode 1.
 * mode 0 = 128-bit register loads, mode 1 = bulk copies into shared memory;
 * adding PROJ_READ_PDL (4) launches it the way proj_run launches the
 * projection kernels, as a programmatic dependent launch (it may start as
 * the previous kernel's CTAs exit; it reads nothing that kernel writes).
 * Any other mode is PROJ_EINVAL.
 */
#define PROJ_READ_PDL 4
int proj_read_floor(const void *buf, int64_t bytes, void *sink, int grid, int mode,
                    proj_stream stream);

/*
 * FP32 FMA probe: the measured ceiling of the CUDA cores' fp32 fused
 * multiply-adds, the denominator for the router's FP32-FMA path (guide ch. 1,
 * §1.5).  Launches `grid` CTAs of 256 threads (grid = 0: eight per SM), each
 * thread running 8 independent chains of packed `fma.rn.f32x2` for `iters`
 * steps (1 <= iters <= 2^24); enqueued on `stream`, time it with events
 * there.  `sink` (device, >= 4 bytes, 4-byte aligned) is never written in
 * practice: it keeps the arithmetic alive.  *flops (if non-NULL) receives the
 * launch's floating-point operations, grid x 256 x 8 x 2 x 2 x iters.
 * Returns PROJ_OK; PROJ_EINVAL (NULL sink, iters or grid out of range);
 * PROJ_EALIGN; PROJ_ECUDA.
 */
int proj_fma_peak(void *sink, int iters, int grid, proj_stream stream, double *flops);

/* Number of SMs of the current device (0 on error). */
int proj_num_sms(void);

/*
 * Allocation-free GEMV for one or two tokens on caller-owned weights.
 * The method's pages have no counterpart of this call: it exists for callers
 * that may not allocate device memory -- a plugin or custom operator that a
 * host framework hands only its input and output buffers while that
 * framework's allocator owns the device memory, or latency-critical code
 * that must not call cudaMalloc/cudaFree (they can stall the whole device and
 * can fail at run time).  Such callers cannot use proj_prepare, which
 * allocates repacked weights and a workspace.
 *
 *   out[i, n] = sum over k of x[i, k] * W[n, k],  0 <= i < m,  0 <= n < N
 *
 *   W       : device, row-major [N, K], contiguous, 16-byte aligned; any N >= 1.
 *   w_dtype : PROJ_BF16 (out is bf16, fp32 sum rounded to nearest even) or
 *             PROJ_FP32 (out is fp32).
 *   K       : a multiple of 1024 in [1024, 8192].
 *   x       : device, bf16 row-major [m, K], 16-byte aligned.
 *   m       : 0, 1 or 2 (0 returns PROJ_OK and launches nothing).
 *   out     : device, row-major [m, N], 16-byte aligned; every element written.
 *
 * The kernel is the ring-form streaming GEMV that proj_run_ex runs with
 * kernel = PROJ_KERNEL_GEMV: with grid = min(SMs, 256) that call splits W over
 * the same min(SMs, 256, N) CTAs and gives bit-identical results (on devices
 * of at most 256 SMs the default grid is the same).  Its scratch is a
 * 4 KB static device array inside the library (hand-off flags, partial row
 * sums and a status word for at most 256 CTAs); each device that loads the
 * library holds it until the process exits.  Nothing is allocated by any
 * call: the first call on a device (the current device when it is made) looks
 * up the array's device address and sets the kernels' shared-memory limit, so
 * make that first call before capturing any stream.  Every call then clears
 * the flags and status word with an asynchronous memset on `stream` and
 * launches one kernel.  All calls on a device share the one array, so calls
 * that overlap on the GPU (different streams, or threads without ordering)
 * race and give wrong results; serialise them.  A stall of the kernel's
 * bounded waits is recorded in that array's status word, which this call
 * does not report: read it with proj_gemv_static_status.
 *
 * Returns PROJ_OK; PROJ_EINVAL for NULL pointers, N < 1, m < 0 or a bad
 * w_dtype; PROJ_EUNSUPPORTED for m > 2 or K outside the rule above (the
 * static scratch is sized for those limits); PROJ_EALIGN; PROJ_ECUDA.  The
 * reason for a rejection is readable through proj_last_cuda_error().
 */
int proj_gemv_static(const void *W, int w_dtype, int64_t N, int64_t K, const void *x,
                     int64_t m, void *out, proj_stream stream);

/* The status word of the last proj_gemv_static call on the current device
 * (each call clears it when it starts; its kernel sets it if a bounded wait
 * gave up, in which case some rows of `out` are not written).  Synchronises
 * `stream` -- the stream of that call -- then reads the word; not for use
 * while `stream` is being captured.  *code receives the raw word if
 * non-NULL.  Returns PROJ_OK (word zero), PROJ_EDEVICE (non-zero) or
 * PROJ_ECUDA; allocates nothing. */
int proj_gemv_static_status(proj_stream stream, uint32_t *code);

/*
 * ---------------------------------------------------------------------------
 * Operators around the projections: products with 4-bit weights, tokens
 * sorted by expert and back, and the norms at a block's two ends.  They take
 * any size (no layer table), work on the caller's buffers, enqueue on
 * `stream` without host synchronisation or allocation, may be captured in a
 * CUDA graph, and give the same bits for the same inputs on every call.  Row
 * strides (ld*) count elements.  Data pointers need the alignment stated
 * with each call; a call that moves nothing (m = 0) returns PROJ_OK.
 * Indices that a buffer holds on the device (offsets, slots, expert ids) are
 * checked in the kernels: one out of range is treated as documented and
 * never read or written through.  Between a row's end and the next row's start
 * (ld > width) nothing is written; what stands there may be read, as part of a
 * 16-byte word, but does not enter any result.
 * ---------------------------------------------------------------------------
 *
 * Products with 4-bit weights and group scales.  A handle holds E matrices
 * [N, K] (E = 1: one layer; E > 1: one matrix per expert) with
 *
 *     w[e, n, k] = s[e, n, k / group] * (q[e, n, k] - z[e, n, k / group]),
 *
 * q and z whole numbers in 0..15.  proj_w4_run computes out = x w^T, and
 * proj_w4_run_experts the same for rows sorted by expert.  Products are
 * summed in fp32 and rounded once, to the type of x.  Up to a few tokens per
 * matrix, s multiplies the fp32 sum of its group, so the 4-bit numbers enter
 * exactly.  For more (and for many experts with K below 4096, whatever their
 * rows) s (q - z) is first rounded to the type of x, as in a checkpoint that
 * was dequantised to it, which adds errors of the size of the output's own
 * rounding.  proj_w4_describe says which of the two a call does.
 * PROJ_W4_EXACT keeps a handle to the first at any number of rows, and so does
 * a scale with which s (q - z) would leave the range of the type.
 */
typedef struct proj_w4_ctx *proj_w4_handle;

enum proj_w4_flags {
    /* No rounding of s (q - z) in any call.  Beyond some 16 rows a matrix the
     * weights are decoded again for every 16 rows, and calls take longer. */
    PROJ_W4_EXACT = 1u << 0
};

/*
 * Repack E matrices (device to device; the sources are consumed before the
 * call returns, which synchronises the legacy default stream).
 *   codes  : [E, N, ceil(K / 2)] bytes; column 2 j of a row is the low half of
 *            its byte j, column 2 j + 1 the high half.
 *   scales : [E, N, ceil(K / group)] in `dtype`.
 *   zeros  : the same shape in bytes (the low four bits count), or NULL: all 8.
 *   group  : columns per scale: 32 or a multiple of 64.
 *   dtype  : PROJ_BF16 or PROJ_FP16, the type of x, scales and out.
 * 1 <= E <= 1024, 1 <= N, K <= 2^20.  A handle holds the packed weights and a
 * status word, nothing else of a call: calls on several streams may overlap.
 * Returns NULL on error (*status, if
 * non-NULL, and proj_last_status() say why).
 */
proj_w4_handle proj_w4_prepare(const void *codes, const void *scales, const void *zeros,
                               int64_t experts, int64_t N, int64_t K, int64_t group, int dtype,
                               int *status);

/* As proj_w4_prepare, with flags of enum proj_w4_flags. */
proj_w4_handle proj_w4_prepare_ex(const void *codes, const void *scales, const void *zeros,
                                  int64_t experts, int64_t N, int64_t K, int64_t group, int dtype,
                                  uint32_t flags, int *status);

/*
 * out[i, n] = sum over k of x[i, k] w[0, n, k], i < m (E must be 1).
 *   x   : m rows of K values, ldx >= K a multiple of 8, 16-byte aligned.
 *   out : m rows of N values, ldo >= N, aligned to an element.
 * x and out must not overlap.  m <= 2^20, strides below 2^31.
 */
int proj_w4_run(proj_w4_handle h, const void *x, int64_t ldx, int64_t m, void *out, int64_t ldo,
                proj_stream stream);

/*
 * Rows offsets[e] .. offsets[e + 1] - 1 of x meet matrix e.  offsets: E + 1
 * int32 on the device, not decreasing, 0 .. m (values outside are moved into
 * that range; if they decrease all the same, a row that several experts claim
 * meets some of them or none).  Rows that belong to no expert are not read, and
 * their rows of out keep what they held.
 */
int proj_w4_run_experts(proj_w4_handle h, const void *x, int64_t ldx, int64_t m,
                        const int32_t *offsets, void *out, int64_t ldo, proj_stream stream);

/* The kernel and launch shape a call with m rows uses (at most `cap` bytes,
 * NUL-terminated; 256 are enough).  For a handle of one matrix that is
 * proj_w4_run's, and where proj_w4_run_experts differs, "; with offsets: " and
 * its own behind it. */
int proj_w4_describe(proj_w4_handle h, int64_t m, char *buf, size_t cap);

/* Read and clear the handle's device status word (synchronises `stream`), as
 * proj_device_status. */
int proj_w4_device_status(proj_w4_handle h, proj_stream stream, uint32_t *code);

/* Free the handle (synchronises the device first; NULL is ignored). */
void proj_w4_destroy(proj_w4_handle h);

/*
 * Tokens sorted by expert and back.  m tokens each choose k of E experts;
 * entry (t, j) is token t's j-th choice, flat index t k + j.  The sort is
 * stable: rows of one expert stand in the order of their flat indices.
 * 1 <= E <= 1024, 1 <= k <= min(E, 32), m * k < 2^31, D <= 2^30.
 */
enum proj_route_mode {
    PROJ_ROUTE_CHOSEN = 0, /* weights: softmax over the chosen logits */
    PROJ_ROUTE_ALL = 1     /* weights: softmax over all logits, at the chosen ones */
};

/* Bytes of workspace that proj_moe_route and proj_moe_sort want (0 is
 * possible); -1 for arguments they refuse. */
int64_t proj_moe_workspace(int64_t m, int64_t experts, int64_t k);

/*
 * Choose and sort.
 *   logits  : fp32 [m, E], stride ldl >= E, aligned to an element.
 *   expert  : int32 [m, k], the k largest logits in descending order, equal
 *             ones by ascending index.  Logits of -infinity and NaN are never
 *             chosen: where a row has fewer than k others, the rest is -1.
 *   weight  : fp32 [m, k]; 0 where expert is -1.
 *   offsets : int32 [E + 1]: rows offsets[e] .. offsets[e + 1] - 1 of the
 *             sorted order are expert e's.
 *   order   : int32 [m k]: the flat index of each sorted row; -1 from
 *             offsets[E] on.
 *   slot    : int32 [m, k]: the sorted row of each entry; -1 where expert is -1.
 * offsets, order and slot may be NULL together: then nothing is sorted.  The
 * workspace (16-byte aligned) is free again when the call's work is done.
 */
int proj_moe_route(const float *logits, int64_t ldl, int64_t m, int64_t experts, int64_t k,
                   int mode, int32_t *expert, float *weight, int32_t *offsets, int32_t *order,
                   int32_t *slot, void *workspace, int64_t workspace_bytes, proj_stream stream);

/* The sort alone, of the caller's choices (ids outside 0 .. E - 1 are no
 * expert's: slot -1). */
int proj_moe_sort(const int32_t *expert, int64_t m, int64_t experts, int64_t k, int32_t *offsets,
                  int32_t *order, int32_t *slot, void *workspace, int64_t workspace_bytes,
                  proj_stream stream);

/*
 * xs[slot[t, j], :] = x[t, :].  x: m rows of D, xs: m k rows of D, both
 * `dtype` (any of proj_dtype), aligned to an element (16-byte aligned
 * pointers and strides are faster).  Rows of xs that no entry names keep
 * what they held; slots outside 0 .. m k - 1 are skipped.
 */
int proj_moe_gather(const void *x, int64_t ldx, const int32_t *slot, int64_t m, int64_t D,
                    int64_t k, int dtype, void *xs, int64_t ldxs, proj_stream stream);

/*
 * out[t, :] = sum over j of weight[t, j] ys[slot[t, j], :], in fp32 in the
 * order of j, rounded once; a token without a valid slot gets zeros.  weight
 * NULL: all ones -- the gradient of proj_moe_gather.
 */
int proj_moe_combine(const void *ys, int64_t ldys, const int32_t *slot, const float *weight,
                     int64_t m, int64_t D, int64_t k, int dtype, void *out, int64_t ldo,
                     proj_stream stream);

/*
 * Gradient of proj_moe_combine: dys[slot[t, j], :] = weight[t, j] dout[t, :]
 * and dweight[t, j] = sum over d of dout[t, d] ys[slot[t, j], d] (0 for a slot
 * outside 0 .. m k - 1).  dys or dweight may be NULL (then ys may be, with
 * dweight); rows of dys that no entry names keep what they held.
 */
int proj_moe_combine_backward(const void *dout, int64_t lddo, const void *ys, int64_t ldys,
                              const int32_t *slot, const float *weight, int64_t m, int64_t D,
                              int64_t k, int dtype, void *dys, int64_t lddys, float *dweight,
                              proj_stream stream);

/*
 * Gradient of the weights of proj_moe_route with respect to the logits, with
 * the choice held fixed.  expert and weight: as proj_moe_route gave them;
 * logits are read in PROJ_ROUTE_ALL mode only (may be NULL otherwise).
 * dlogits: fp32 [m, E], every element written.
 */
int proj_moe_route_backward(const float *logits, int64_t ldl, int64_t m, int64_t experts,
                            int64_t k, int mode, const int32_t *expert, const float *weight,
                            const float *dweight, float *dlogits, int64_t lddl,
                            proj_stream stream);

/*
 * The norms after one block and before the next, with the block's gate and
 * the residual scale, in one pass.  Row by row, in fp32, each output rounded
 * once:
 *
 *     n      = y rsqrt(mean(y^2) + eps) w_post      (y_plain: n = y)
 *     out    = alpha residual + beta g n,           g = act(gate)
 *     normed = out' rsqrt(mean(out'^2) + eps) w_pre (out' = out before rounding)
 */
enum proj_gate_mode {
    PROJ_GATE_NONE = 0,    /* g = 1 */
    PROJ_GATE_CHANNEL = 1, /* gate [D] */
    PROJ_GATE_ELEMENT = 2, /* gate [m, D], stride ldg */
    PROJ_GATE_TOKEN = 3    /* gate [m] */
};
enum proj_gate_act { PROJ_GATE_LINEAR = 0, PROJ_GATE_SIGMOID = 1 };

typedef struct proj_norm_args {
    int64_t m, D;          /* 1 <= D <= 16384 */
    int dtype;             /* of every tensor but the statistics: any of proj_dtype */
    int gate_mode;         /* enum proj_gate_mode */
    int gate_act;          /* enum proj_gate_act */
    int y_plain;           /* 1: no norm after the block (w_post and rstd_post NULL) */
    float eps, alpha, beta;
    const void *y;         /* the block's output [m, D]; NULL: no block, out = alpha residual
                              (then w_post, rstd_post NULL and gate_mode NONE) */
    int64_t ldy;
    const void *residual;  /* [m, D] */
    int64_t ldr;
    const void *gate;      /* by gate_mode; NULL for NONE */
    int64_t ldg;
    const void *w_post;    /* [D], NULL: ones */
    const void *w_pre;     /* [D], NULL: ones */
    void *out;             /* [m, D]; may be `residual` itself (same stride), or NULL */
    int64_t ldo;
    void *normed;          /* [m, D]; may be `y` itself (same stride), or NULL; one of out
                              and normed is not NULL, and they do not overlap */
    int64_t ldn;
    float *rstd_post;      /* [m], optional: the two rsqrt factors, which the gradient wants */
    float *rstd_pre;
} proj_norm_args;

/* Pointers are aligned to an element; rows that all start on 16 bytes, with D
 * a multiple of 16 bytes, are faster. */
int proj_norm(const proj_norm_args *args, proj_stream stream);

typedef struct proj_norm_grad_args {
    int64_t m, D;          /* the forward call's values, down to rstd_pre */
    int dtype, gate_mode, gate_act, y_plain;
    float eps, alpha, beta;
    const void *y;
    int64_t ldy;
    const void *residual;
    int64_t ldr;
    const void *gate;
    int64_t ldg;
    const void *w_post;
    const void *w_pre;
    const float *rstd_post; /* as the forward call wrote them (rstd_post: unless y is NULL or */
    const float *rstd_pre;  /* y_plain; rstd_pre: unless dnormed is NULL) */
    const void *dout;       /* gradient of out [m, D], NULL: zero */
    int64_t lddo;
    const void *dnormed;    /* gradient of normed [m, D], NULL: zero (not both NULL) */
    int64_t lddn;
    void *dy;               /* gradients, each optional; none may overlap an input */
    int64_t lddy;
    void *dresidual;
    int64_t lddr;
    void *dgate;            /* CHANNEL: fp32 [D]; ELEMENT: dtype [m, D], stride lddg;
                               TOKEN: dtype [m] */
    int64_t lddg;
    float *dw_post;         /* fp32 [D] */
    float *dw_pre;          /* fp32 [D] */
    void *workspace;        /* proj_norm_workspace(m, D) bytes, 16-byte aligned; wanted for
                               dw_post, dw_pre and a CHANNEL dgate */
    int64_t workspace_bytes;
} proj_norm_grad_args;

/* Bytes of workspace of proj_norm_backward; -1 for m < 0 or a bad D. */
int64_t proj_norm_workspace(int64_t m, int64_t D);

/* Gradients of proj_norm; sums over tokens are taken in a fixed order. */
int proj_norm_backward(const proj_norm_grad_args *args, proj_stream stream);

/*
 * ---------------------------------------------------------------------------
 * The cache of keys and values between the qkv_gate and o projections: rows
 * quantised as they are written, read back, moved when drafts are accepted,
 * and attention of drafted tokens over it.  What stands above for the
 * operators around the projections holds here too.
 *
 * A cache is pages of `page` tokens.  For each token and head of keys and
 * values it keeps D entries of keys and D of values, 16 bits wide or 8 bits
 * with one fp32 scale:
 *
 *     value = code * scale,   scale = max(amax / top, 2^-126),
 *     code  = round(x * (1 / scale)),  top = 448 (e4m3) or 127 (int8),
 *
 * with amax the row's largest magnitude, each step rounded to fp32 and the
 * code to nearest even.  A row with a NaN or an infinity gets codes 0 and the
 * scale NaN: it reads back as NaN.
 *
 * The pages of sequence b are table[b, 0 .. width - 1]: position p stands in
 * page table[b, p / page] at place p % page.  A page id outside 0 .. pages - 1
 * is no page: nothing is written there, it reads back as zeros and no query
 * sees it.  Sequences may share pages that no call writes.
 *
 * Rows of a call belong to sequences by `offsets` [sequences + 1] on the
 * device, 0 <= offsets[b] <= offsets[b + 1] <= m (values outside are moved
 * into that range): row offsets[b] + i stands for position start[b] + i.  Rows
 * before offsets[0] and from offsets[sequences] on are no sequence's and left
 * alone.  A negative start counts as 0 in proj_attn; the other calls leave the
 * rows of negative positions as rows without a page.
 * ---------------------------------------------------------------------------
 */
enum proj_kv_format {
    PROJ_KV_ROWS = 0, /* entries of the cache's dtype, no scales */
    PROJ_KV_E4M3 = 1, /* 8-bit floating point, 4 bits of exponent, no infinities */
    PROJ_KV_INT8 = 2  /* -127 .. 127 */
};

typedef struct proj_kv_cache {
    int format;            /* enum proj_kv_format */
    int dtype;             /* PROJ_BF16 or PROJ_FP16: rows written and read back, queries, outputs */
    int64_t pages, page;   /* pages in all; tokens of one, 1 .. 65536 */
    int64_t heads, D;      /* heads of keys and values, 1 .. 1024; D = 64 or 128 */
    void *k, *v;           /* entries, 16-byte aligned */
    float *k_scale;        /* [pages, heads, page]; NULL for PROJ_KV_ROWS */
    float *v_scale;
    int64_t page_stride;   /* entry (page, head, place) starts at page page_stride + head head_stride */
    int64_t head_stride;   /* + place token_stride entries; multiples of 16 bytes, at least D */
    int64_t token_stride;  /* page and token: below 2^31 bytes */
    const int32_t *table;  /* device [sequences, width], row stride ldt >= width */
    int64_t ldt, width;    /* width page < 2^30 */
    int64_t sequences;     /* 0 .. 65536 */
} proj_kv_cache;

/*
 * Write rows k and v (m rows of heads D values, dtype; 16-byte aligned, strides
 * multiples of 8) to their positions; m < 2^30.  No two rows of a call may
 * stand in one place (of a page that the table names twice): what it holds
 * afterwards is not defined.
 */
int proj_kv_write(const proj_kv_cache *cache, const int32_t *offsets, const int32_t *start,
                  int64_t m, const void *k, int64_t ldk, const void *v, int64_t ldv,
                  proj_stream stream);

/* Read the same rows back, rounded once to dtype.  k or v may be NULL. */
int proj_kv_read(const proj_kv_cache *cache, const int32_t *offsets, const int32_t *start,
                 int64_t m, void *k, int64_t ldk, void *v, int64_t ldv, proj_stream stream);

/*
 * Accepted drafts to their places: entry i of path[b] (row stride ldp >=
 * depth) moves from position start[b] + path[b, i] to start[b] + i, codes and
 * scales as they are.  A path ascends from 0 or more (a draft comes after its
 * parent); the first entry that does not, or is negative, ends it.  Where one
 * of the two positions has no page, that entry is not moved.
 *   next_start : optional [sequences], start[b] + the number of entries; not
 *                `start` itself.
 */
int proj_kv_move(const proj_kv_cache *cache, const int32_t *start, const int32_t *path,
                 int64_t ldp, int64_t depth, int32_t *next_start, proj_stream stream);

/*
 * Attention of drafted tokens over the cache, which holds their own keys and
 * values already (proj_kv_write with the same offsets and start).  Query head
 * j meets head j / (heads / cache heads) of keys and values.  Row i of a
 * sequence sees all start[b] positions before the drafts, and of draft d
 *
 *     mask given : bit d % 32 of mask[row, d / 32] (d < 32 words), else
 *     mask NULL  : d <= i.
 *
 *     out = (softmax(scale q k^T over what the row sees) v) act(gate)
 *
 * A row that sees nothing, or only keys whose score is -infinity, gets zeros and
 * lse = -infinity.  What a row does not
 * see does not reach it, NaN and infinities included; where it sees a value that
 * is no finite number, that column of it is none either (an infinity or NaN).
 * Scores, their maximum and sums are fp32 (|v| below 2^90 keeps those of V there);
 * the products of 8-bit caches and of fp16 are computed in fp16 with codes and
 * queries exact in it (a row of bf16 queries is brought to its range by a power of
 * two; what is 2^-29 below the row's largest loses digits) and probabilities rounded
 * to it; those of bf16 caches in bf16, to which probabilities are rounded as well.
 * (The streaming kernel rounds them to a sum of two numbers of a 16-bit cache's
 * type.)  With 8-bit caches it is the product of probability and V's scale that is
 * rounded, to 2^-11 of itself or 2^-29 of the largest |v| that the row sees, whichever
 * is more; drafts that it does not see count for nothing in that as long as their
 * values are not beyond 2^60 times those that it does.
 * The gate is applied in fp32 and the result rounded once.
 *
 * How many rows and positions a sequence has is read on the device.  Which kernel
 * runs goes by m, sequences and heads, and by the table's width as the most that
 * a sequence can hold (proj_attn_describe): the results are good either way.
 */
typedef struct proj_attn_args {
    const proj_kv_cache *cache;
    int64_t m, heads;        /* rows of q, at most 2^20; query heads, a multiple of the cache's, at most 1024 */
    const void *q;           /* [m, heads D], dtype; 16-byte aligned, strides multiples of 8 */
    int64_t ldq;
    const int32_t *offsets;  /* device [sequences + 1] */
    const int32_t *start;    /* device [sequences] */
    const uint32_t *mask;    /* device [m, words], row stride ldm, or NULL */
    int64_t ldm, words;      /* words: 1 .. 1024 */
    float scale;             /* finite, and scale log2(e) too */
    int gate_act;            /* enum proj_gate_act */
    const void *gate;        /* [m, heads D], dtype, as q; NULL: none */
    int64_t ldg;
    void *out;               /* [m, heads D], dtype, as q; may be q itself or the gate (same stride) */
    int64_t ldo;
    float *lse;              /* [m, heads] natural logarithm of each row's sum, or NULL */
    void *workspace;         /* proj_attn_workspace bytes, 16-byte aligned */
    int64_t workspace_bytes;
} proj_attn_args;

/* Bytes of workspace of proj_attn on this device, no less for more rows of the
 * same cache; -1 for arguments it refuses.
 * A workspace holds nothing between calls, and calls that may overlap need one
 * each. */
int64_t proj_attn_workspace(const proj_kv_cache *cache, int64_t m, int64_t heads);

int proj_attn(const proj_attn_args *args, proj_stream stream);

/* The kernel and launch shape of proj_attn for m rows (at most `cap` bytes,
 * NUL-terminated; 256 are enough). */
int proj_attn_describe(const proj_kv_cache *cache, int64_t m, int64_t heads, char *buf, size_t cap);

/* Read and clear the status word of the current device's proj_attn calls
 * (synchronises `stream`; not while it is being captured), as
 * proj_device_status: PROJ_EDEVICE where a kernel's bounded wait gave up. */
int proj_attn_device_status(proj_stream stream, uint32_t *code);

#ifdef __cplusplus
}
#endif

#endif /* PROJ_H_ */
