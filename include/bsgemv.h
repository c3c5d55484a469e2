/*
 * bsgemv.h -- C ABI of the fused dequantize-and-multiply small-M GEMV for one NVIDIA GB300
 * (sm_103a):
 *
 *     y[M, N] = A[M, K] . deq(W)[N, K]^T,        1 <= M <= 32
 *
 * A is fp16 or bf16.  W is block-quantised along K and stored in the [N, blocks, blob] layout
 * ("[CUDA] Batched small-M GEMV for MatMulNBits (4-bit/8-bit)", Description), in one of:
 *
 *   BSGEMV_INT4      4-bit codes, two per byte (low nibble = even k); deq = (q - zp) * s with an
 *                    fp16 scale per (row, block) and an optional packed 4-bit zero point
 *                    ("[CUDA] MatMulNBits 8-bit: wide fp16 M=1 kernel for decode GEMVs",
 *                    Description; batched small-M page, Description and review)
 *   BSGEMV_INT8      8-bit codes; deq = (q - zp) * s, fp16 scale, optional 8-bit zero point
 *                    (wide M=1 page, Description)
 *   BSGEMV_FP8_E4M3  E4M3 codes; deq = e4m3 * s with one fp32 scale per 128 k
 *                    ("[CUDA] Block-scaled MatMul decode GEMV: tensor cores, packed FP4 decode
 *                    and M-tiling", description, FP8 tensor-core paragraph)
 *   BSGEMV_NVFP4     E2M1 codes two per byte (low nibble = even k), one E4M3 scale per 16 k and
 *                    one fp32 global scale g; deq = e2m1 * e4m3 * g (same page, NVFP4
 *                    tensor-core paragraph)
 *
 * Every call accumulates in fp32 and rounds the result once, round-to-nearest-even, to the
 * activation dtype.  The library has no CPU fallback: without an sm_103a device every entry
 * point that needs one returns an error.
 *
 * Layouts (all row-major, all tensors caller-owned):
 *   A       [M, K] fp16/bf16, device memory, 16-byte aligned
 *   W       int4/nvfp4: [N, K/2] bytes; int8/fp8: [N, K] bytes; device, 16-byte aligned
 *   scales  int4/int8: fp16 [N, K/bs]; fp8: fp32 [N, K/128]; nvfp4: E4M3 bytes [N, K/16]
 *   zp      int4: [N, ceil((K/bs)/2)] bytes, block b in nibble (b & 1) of byte b/2 (low nibble =
 *           even block); int8: [N, K/bs] bytes; NULL when has_zp == 0 (implicit zero point 8
 *           for int4, 128 for int8).  For NVFP4 this slot carries the device pointer of the one
 *           fp32 global scale.  For FP8 it must be NULL.
 *   y       [M, N] in the activation dtype, device memory, 16-byte aligned
 *
 * Streams are passed as `void*` holding a cudaStream_t (NULL = the legacy default stream).
 * All entry points are host functions; bsgemv_run only enqueues work and never synchronises.
 * A plan may be used by one stream at a time: its cross-CTA reduction workspace is shared by
 * every call made with it.  Status codes are returned; no exception crosses the ABI.
 */
#ifndef BSGEMV_H_
#define BSGEMV_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct bsgemv_plan_s* bsgemv_plan_t; /* opaque; owned by the library */

enum bsgemv_format {
  BSGEMV_INT4 = 1,
  BSGEMV_INT8 = 2,
  BSGEMV_FP8_E4M3 = 3,
  BSGEMV_NVFP4 = 4
};
/* OR-ed into `format`: the activations (and the output) are bf16 instead of fp16. */
#define BSGEMV_ACT_BF16 0x100

enum bsgemv_status {
  BSGEMV_OK = 0,
  BSGEMV_ERR_INVALID_ARG = -1,    /* NULL pointer, M out of range for the call, bad enum ... */
  BSGEMV_ERR_UNSUPPORTED = -2,    /* shape / block size / format combination not provided,
                                     or no sm_103a device */
  BSGEMV_ERR_MISALIGNED = -3,     /* A, W or y not 16-byte aligned */
  BSGEMV_ERR_M_TOO_LARGE = -4,    /* M > the plan's max_M */
  BSGEMV_ERR_CUDA = -5,           /* a CUDA runtime/driver call failed */
  BSGEMV_ERR_WRONG_DEVICE = -6,   /* the current device is not the plan's device */
  BSGEMV_ERR_DEVICE_TIMEOUT = -7, /* a kernel gave up a bounded wait (reported by
                                     bsgemv_device_status) */
  BSGEMV_ERR_SCRATCH_LIMIT = -8   /* bsgemv_run_noalloc: the problem needs more than the fixed
                                     scratch area holds */
};

/* Variants a plan can run (bsgemv_geometry.variant, bsgemv_plan_set_override). */
enum bsgemv_variant {
  BSGEMV_VARIANT_AUTO = 0,
  BSGEMV_VARIANT_MMA = 1,        /* tensor-core mma.sync m16n8k16, fp32 accumulate */
  BSGEMV_VARIANT_CUDA_CORE = 2   /* CUDA-core packed fp32 FMA (fma.rn.f32x2) over the same
                                    copies, decoders and reductions; plans with max_M <= 8.  A
                                    measured alternative: the tensor-core variant is faster for
                                    every format and M */
};

/* What a plan chose.  Filled by bsgemv_plan_describe / bsgemv_geometry_for. */
typedef struct {
  int variant;           /* enum bsgemv_variant */
  int rows_per_tile;     /* output columns n per CTA tile */
  int k_per_stage;       /* k elements per pipeline stage */
  int stages;            /* depth of the shared-memory ring */
  int consumer_warps;    /* warps that decode and multiply; one more warp issues the copies */
  int ctas;              /* persistent CTAs launched */
  int ctas_per_sm;       /* CTAs resident per SM the geometry was sized for */
  int sm_count;          /* SM count the geometry was derived for */
  int64_t tiles;         /* ceil(N / rows_per_tile) */
  int64_t stages_per_tile;
  int64_t total_stages;  /* tiles * stages_per_tile: the work split evenly over the CTAs */
  int smem_bytes;        /* dynamic shared memory per CTA */
  int64_t workspace_bytes;
  int cluster;           /* how a tile's K is split: 0 = stream-K over all CTAs with a global
                            last-arriver reduction; C >= 1 = C CTAs per tile in one thread-block
                            cluster, reduced in the cluster leader's shared memory */
} bsgemv_geometry;

/* How a plan splits the K of a tile over CTAs (bsgemv_plan_set_split). */
enum bsgemv_split {
  BSGEMV_SPLIT_AUTO = 0,      /* cluster split where its per-CTA work is within one stage of
                                 stream-K's, else stream-K */
  BSGEMV_SPLIT_STREAM_K = 1,  /* the tiles x stages space cut into equal ranges over all CTAs */
  BSGEMV_SPLIT_CLUSTER = 2    /* each tile split over the CTAs of one cluster, shares differing
                                 by at most one stage */
};

/*
 * Create a plan for one weight shape.  format = enum bsgemv_format, optionally | BSGEMV_ACT_BF16.
 * block_size: int4/int8 one of 16, 32, 64, 128, 256; fp8 128; nvfp4 16.
 * has_zp: 0 or 1 (int formats only; must be 0 for fp8 and nvfp4).
 * N >= 1 (any tail); K >= 64 with K % 64 == 0 and K % block_size == 0; 1 <= max_M <= 32 (the
 * pages' decode GEMVs take M <= 16; a plan for up to 24 rows runs three n8 activation tiles at
 * 3 CTAs per SM, or four at 2 CTAs per SM where that keeps a cluster split of its tiles; a plan
 * for up to 32 rows runs four at 2 CTAs per SM.  Size a plan for the largest M it serves).
 * Uses the current CUDA device, which must be sm_103 (GB300).  Allocates the plan's own device
 * workspace (cross-CTA partial sums, arrival counters and an error word, all zeroed here) with
 * cudaMalloc; every call reuses it and the kernels leave the counters at zero.
 * On success *out holds the plan; on error *out is NULL and a status < 0 is returned.
 */
int bsgemv_plan(bsgemv_plan_t* out, int format, int block_size, int has_zp, int64_t N, int64_t K,
                int max_M);

/*
 * Enqueue y = A . deq(W)^T for the first M (1 <= M <= max_M) rows of A on `stream`.
 * Pointers as in the layout table above (device memory).  Checks arguments, alignment and the
 * current device, launches one kernel and returns cudaGetLastError's result; it does not wait.
 * Results depend only on the plan and the inputs: the same row of A gives bit-identical
 * output for every M, and repeated calls are bit-identical.
 */
int bsgemv_run(bsgemv_plan_t plan, const void* A, const void* W, const void* scales,
               const void* zp, void* y, int M, void* stream);

/*
 * y = A . deq(W)^T + bias: as bsgemv_run, plus `bias`, N values in the activation dtype (device
 * memory, 2-byte aligned, caller-owned), added to every row's fp32 sum before the one rounding.
 * ("[CUDA] Block-scaled MatMul decode GEMV: tensor cores, packed FP4 decode and M-tiling",
 * Tests: the FP8 and FP4 operators take an optional bias; "[CUDA] Pin FP8 GEMV residency for
 * grids just past two blocks per SM", Tests.)  NULL bias: BSGEMV_ERR_INVALID_ARG (call
 * bsgemv_run instead).  Same determinism as bsgemv_run: rows are bit-identical across M.
 */
int bsgemv_run_bias(bsgemv_plan_t plan, const void* A, const void* W, const void* scales,
                    const void* zp, const void* bias, void* y, int M, void* stream);

/*
 * Same as bsgemv_run, but A and y are HOST memory (pinned memory gives asynchronous copies):
 * A is copied into the plan's device staging buffer, the GEMV runs, y is copied back, and the
 * call returns after the stream has finished (the host buffers are ready on return).  W,
 * scales and zp stay device pointers.  The staging buffer (max_M * (K + N) activation
 * elements) is allocated by the first call and freed by bsgemv_destroy.  When both host
 * buffers are pinned and 16-byte aligned they are used through their device mapping: a small
 * kernel copies A into the staging buffer (its start-up overlaps the neighbouring kernels like
 * the GEMV's own) and the GEMV writes y straight into y_host; otherwise A and y go through the
 * staging buffer by copy-engine transfers (cudaMemcpyAsync).
 */
int bsgemv_run_host(bsgemv_plan_t plan, const void* A_host, const void* W, const void* scales,
                    const void* zp, void* y_host, int M, void* stream);

/*
 * bsgemv_run_host without the final wait: the copy of A in, the GEMV and the copy of y out are
 * enqueued on `stream` and the call returns.  y_host holds the result once the stream has been
 * synchronised, and A_host must not change before then.  With pinned host memory the copies are
 * asynchronous, so a step of several GEMVs costs one synchronisation, not one per GEMV.  Calls
 * on one plan share its staging buffer: issue them on one stream (stream order keeps each
 * call's copy of A after the previous call's copy of y).
 */
int bsgemv_run_host_async(bsgemv_plan_t plan, const void* A_host, const void* W,
                          const void* scales, const void* zp, void* y_host, int M, void* stream);

/* Free the plan and its device memory (synchronises the device first).  NULL is a no-op. */
int bsgemv_destroy(bsgemv_plan_t plan);

/* Static, human-readable name of a status code. */
const char* bsgemv_status_string(int status);

/*
 * Test hook: write the dequantised weight deq(W) as fp32 [N, K] to `out` (device, caller-owned,
 * N * K floats), through the same register decoders and fragment mapping as the GEMV.  Each
 * value is the exact dequantised weight rounded once to fp32 (exact for int4/int8; for fp8 and
 * nvfp4 one rounding of the exact product).  Enqueued on `stream`.
 */
int bsgemv_debug_dequant(bsgemv_plan_t plan, const void* W, const void* scales, const void* zp,
                         float* out, void* stream);

/*
 * Choose how the plan splits each tile's K over CTAs (no counterpart on the pages, whose kernels
 * use a fixed split-K or none: an A/B and testing aid like bsgemv_plan_set_override).
 * split = enum bsgemv_split; cluster_size (CLUSTER only) = CTAs per tile, 1..16, 0 = chosen by
 * the plan from the SM count.  Returns BSGEMV_ERR_UNSUPPORTED when the tiles x cluster_size
 * CTAs do not fit one wave of the device or cluster_size exceeds the stages of a tile; the plan
 * is then unchanged.  Not thread-safe with bsgemv_run on the same plan.
 */
int bsgemv_plan_set_split(bsgemv_plan_t plan, int split, int cluster_size);

/*
 * A/B override for measurements: variant (enum bsgemv_variant, 0 = keep; CUDA_CORE needs a plan
 * with max_M <= 8, else BSGEMV_ERR_UNSUPPORTED), ctas (persistent
 * CTAs of a stream-K split, 0 = keep; under BSGEMV_SPLIT_AUTO a CTA count selects stream-K),
 * rows_per_tile (output columns per CTA tile: 64 or 128, 0 = keep; 128 needs a plan with
 * max_M <= 16 and the tensor-core variant, else BSGEMV_ERR_UNSUPPORTED), stages (ring depth,
 * 0 = keep).
 * Changes the summation order, so results are bit-identical only between calls made under the
 * same settings.  Returns BSGEMV_ERR_UNSUPPORTED for a setting the plan cannot run.
 */
int bsgemv_plan_set_override(bsgemv_plan_t plan, int variant, int ctas, int rows_per_tile,
                             int stages);

/*
 * Measure this plan's candidate geometries on the device and keep the fastest (the "online
 * profiler" that "[CUDA] Batched small-M GEMV for MatMulNBits (4-bit/8-bit)", review, proposes
 * instead of thresholds tuned on one GPU).  Candidates, in two rounds: first the K split under
 * each tile height (the automatic one, 64 and 128 rows) -- the automatic choice, stream-K over the
 * default grid and over 1 .. 4 CTAs per SM, and thread-block clusters of 2 .. 8 CTAs per tile --
 * then the ring depth of the fastest (2, 3, 4, 6, 8 or 12 stages, at the same CTAs per SM);
 * candidates the plan cannot run are skipped.  They are timed in the regime the calls run in:
 * back to back on one stream (a CUDA graph of `reps` (1 .. 100) rounds over R copies of W,
 * scales and zp, R copies >= 3x the L2, at most 8, so that no call finds its weights in L2),
 * with the caller's A and y (y is overwritten): calls of M rows plus, when M > 1, calls of one
 * row in a graph of their own (the chosen geometry serves every M of the plan).  The copies, a private
 * stream and the graphs are made and freed here.  Another geometry replaces the automatic
 * choice only if it is more than 1 % faster, in the search and again when the two are timed in
 * turn, twice each, at the end.
 * Synchronises `stream` first and returns when done; not for use inside stream capture.
 * Afterwards every call of the plan runs the chosen geometry, so rows stay bit-identical across
 * M from then on (results may differ in the last bits from calls made before, as the
 * summation order can change).  On an error the plan keeps its previous settings.
 */
int bsgemv_plan_autotune(bsgemv_plan_t plan, const void* A, const void* W, const void* scales,
                         const void* zp, void* y, int M, int reps, void* stream);

/* Copy the plan's current geometry into *g. */
int bsgemv_plan_describe(bsgemv_plan_t plan, bsgemv_geometry* g);

/*
 * Pure host function, no CUDA call: the geometry bsgemv_plan would choose for this problem on a
 * device with `sm_count` SMs (and the sm_103 shared-memory budget).  Returns the same status
 * bsgemv_plan would return for invalid arguments.
 */
int bsgemv_geometry_for(int format, int block_size, int has_zp, int64_t N, int64_t K, int max_M,
                        int sm_count, bsgemv_geometry* g);

/*
 * Synchronise `stream`, then read and clear the plan's device error word.  Returns BSGEMV_OK,
 * BSGEMV_ERR_DEVICE_TIMEOUT if a kernel of this plan abandoned a bounded wait since the last
 * check, or BSGEMV_ERR_CUDA if the synchronisation failed.  plan = NULL reads and clears the
 * error word of bsgemv_run_noalloc on the current device instead (kept across its calls until
 * read here).  Every wait of the kernels is bounded (4 s): a kernel that gives one up stops
 * reading its copies, waits (bounded again) for the copies it issued to land, completes its
 * partial sums so that the plan stays usable, and returns; its output is not valid.
 */
int bsgemv_device_status(bsgemv_plan_t plan, void* stream);

/*
 * Test hook of the failure path above (the method's pages have no counterpart; it exercises this
 * library's bounded waits without faulting the GPU).  skip_stage >= 0: in the plan's next calls
 * the copy warp of CTA 0 leaves out stage `skip_stage` of that CTA's range (nothing is copied
 * for it, so its consumer warps' wait on it runs out); -1: none.  wait_ns > 0: the calls' waits
 * give up after wait_ns nanoseconds instead of 4 s; 0: the default.  Host only, no CUDA call;
 * returns BSGEMV_ERR_INVALID_ARG for NULL, skip_stage < -1 or wait_ns < 0.
 * bsgemv_plan_set_test_fault(plan, -1, 0) restores normal calls.
 */
int bsgemv_plan_set_test_fault(bsgemv_plan_t plan, int skip_stage, int64_t wait_ns);

/*
 * The GEMV without any allocation, for callers that cannot call cudaMalloc: runtimes that own
 * all device memory up front, code running inside another framework's memory pool, paths where
 * an allocation could fail or synchronise at the wrong moment.  (The method's pages have no
 * counterpart; this is a property of this library's interface.)
 *
 * Arguments as bsgemv_plan plus bsgemv_run; no plan is created.  Every call runs the geometry of
 * a plan sized for 16 rows, whatever its M: a row's result is bit-identical for every M and
 * equal to bsgemv_plan(..., max_M = 16) + bsgemv_run.  Instead of a plan's cudaMalloc'd
 * workspace the cross-CTA reduction uses one fixed scratch area compiled into the library (a
 * file-scope device array of about 7.6 MiB that every GPU loading the library holds until the
 * process exits).  Limits: M <= 16 (BSGEMV_ERR_INVALID_ARG beyond), N <= 524288 output columns
 * and at most 480 persistent CTAs (a 152-SM GB300 uses 456); beyond them the call returns
 * BSGEMV_ERR_SCRATCH_LIMIT and does nothing.  The first call on a device looks up the scratch
 * area's device address (with that device current), and so does the first call after the
 * device's context changed (e.g. after cudaDeviceReset); make such a first call before any
 * stream capture.  Every call on a device shares the one scratch area: calls that overlap on
 * the GPU (other streams, other host threads) race on it and give wrong results, so serialise
 * them.  Each call clears the counters it uses with cudaMemsetAsync on `stream` before its
 * kernel; it calls no cudaMalloc, cudaFree or allocating routine.  A bounded wait that ran out
 * in one of these calls is reported by bsgemv_device_status(NULL, stream).  Enqueue only; no
 * synchronisation.
 */
int bsgemv_run_noalloc(int format, int block_size, int has_zp, int64_t N, int64_t K,
                       const void* A, const void* W, const void* scales, const void* zp, void* y,
                       int M, void* stream);

/*
 * Dense small-N GEMV ("[CUDA] MatMul: add an opt-in split-K GEMV for small-N fp16 shapes",
 * Description): y[M, N] = A[M, K] . B[K, N] with A, B and y fp16 (act_bf16 = 0) or bf16
 * (act_bf16 = 1), B row-major [K, N] (the MatMul right-hand side), 1 <= M <= max_M <= 8.
 * K is split over the CTAs of a thread-block cluster per 64-column tile and the partial sums
 * are added in a fixed order (results are deterministic and rows bit-identical across M).
 * N % 8 == 0, K % 8 == 0 and K >= 16 (16-byte row pitches) run the TMA / tensor-core kernel, with
 * A, B and y 16-byte aligned; any other N >= 1, K >= 1 (the page's tests include N = 1) runs a
 * CUDA-core kernel (8 columns per CTA, K split over a cluster, the same fixed-order reduction),
 * with A, B and y 2-byte aligned.  Device memory.  The plan allocates only an error word.  Same
 * status conventions as above.
 */
typedef struct bsgemv_dense_plan_s* bsgemv_dense_plan_t;

int bsgemv_dense_plan(bsgemv_dense_plan_t* out, int act_bf16, int64_t N, int64_t K, int max_M);

/* Enqueue y = A . B for the first M rows of A on `stream` (one kernel; no synchronisation). */
int bsgemv_dense_run(bsgemv_dense_plan_t plan, const void* A, const void* B, void* y, int M,
                     void* stream);

/* The plan's geometry: rows_per_tile = 64 columns, k_per_stage = 64, cluster = CTAs per tile. */
int bsgemv_dense_describe(bsgemv_dense_plan_t plan, bsgemv_geometry* g);

/* Pure host function: the geometry bsgemv_dense_plan would choose with `sm_count` SMs. */
int bsgemv_dense_geometry_for(int act_bf16, int64_t N, int64_t K, int max_M, int sm_count,
                              bsgemv_geometry* g);

/* Synchronise `stream`, then read and clear the plan's error word (as bsgemv_device_status). */
int bsgemv_dense_device_status(bsgemv_dense_plan_t plan, void* stream);

/* Free the plan (synchronises the device first).  NULL is a no-op. */
int bsgemv_dense_destroy(bsgemv_dense_plan_t plan);

/*
 * ---------------------------------------------------------------------------------------------
 * The rest of a decode step: the mixture-of-experts layer, attention over a paged cache and the
 * pages of that cache.  Same conventions as above (streams, statuses, caller-owned tensors, one
 * stream at a time per plan, enqueue only unless said otherwise).
 *
 * Mixture-of-experts layer for a few tokens.  For token t with router logits l[t, 0 .. E-1]:
 *
 *     e_1 .. e_k = the k largest logits (equal logits: the lowest expert first)
 *     p_j        = exp(l[e_j]) / sum of exp(l) over the chosen experts
 *                  (over all E without BSGEMV_MOE_RENORMALIZE)
 *     g, u       = W13[e_j] . x[t]    rows 0 .. I-1 and I .. 2I-1 of the [2I, H] weight
 *     y[t]       = sum over j of p_j * W2[e_j] . (g / (1 + exp(-g)) * u)       W2: [H, I]
 *
 * x, y and (unless BSGEMV_MOE_LOGITS_F32) the logits are in the activation dtype.  Sums, softmax
 * and the intermediate are fp32 (the intermediate enters the second product as two f16 parts with
 * a power of two for every 128 or 256 of a row: to 2^-22 of the largest of them); y is rounded
 * once.  An expert's weights are read once for all tokens that chose it, and other experts' weights
 * are not read.  A logit of -inf is
 * never chosen; a row with nothing to choose gives y = 0.  A row that holds a NaN or +inf logit
 * gives NaN, as the softmax has it.  What one token chose never reaches another token's row, NaN
 * weights included.
 *
 * Weights of all experts are stacked: W13 [E][2I][row bytes of H], W2 [E][H][row bytes of I],
 * scales and zero points likewise, each in the layout table's format.  zp13 / zp2: NULL without
 * zero points and for FP8; for NVFP4 the device pointers of E fp32 global scales, one per expert.
 */
typedef struct bsgemv_moe_plan_s* bsgemv_moe_plan_t;

enum bsgemv_moe_flags {
  BSGEMV_MOE_RENORMALIZE = 1, /* weights of the chosen experts sum to one */
  BSGEMV_MOE_LOGITS_F32 = 2   /* logits are fp32 whatever the activation dtype */
};

/*
 * format, block_size, has_zp as bsgemv_plan, except that integer block sizes are 16, 32, 64 or
 * 128.  H and I: multiples of 64 and of block_size, at least 64, below 2^24;
 * 2 I E and H E below 2^31.  1 <= E <= 1024, 1 <= top_k <= min(E, 16), 1 <= max_T <= 32, flags of bsgemv_moe_flags.
 */
int bsgemv_moe_plan(bsgemv_moe_plan_t* out, int format, int block_size, int has_zp, int64_t H,
                    int64_t I, int E, int top_k, int max_T, int flags);

/* Enqueue the layer for T (1 .. max_T) tokens.  x, W13, W2 and y 16-byte aligned; scales and
 * zero points 4-byte aligned, logits to their element.  Deterministic: repeated calls are
 * bit-identical. */
int bsgemv_moe_run(bsgemv_moe_plan_t plan, const void* x, const void* logits, const void* W13,
                   const void* scales13, const void* zp13, const void* W2, const void* scales2,
                   const void* zp2, void* y, int T, void* stream);

/* The same layer for a router of the caller's own: ids [T][top_k] int32 and weights [T][top_k]
 * fp32 (device) in place of the logits.  An id outside 0 .. E-1 is an unused place; an expert
 * named twice by a token counts with the sum of its weights. */
int bsgemv_moe_run_routed(bsgemv_moe_plan_t plan, const void* x, const int32_t* ids,
                          const float* weights, const void* W13, const void* scales13,
                          const void* zp13, const void* W2, const void* scales2, const void* zp2,
                          void* y, int T, void* stream);

/* Synchronise `stream`, then read and clear the plan's error word (as bsgemv_device_status).  After
 * BSGEMV_ERR_DEVICE_TIMEOUT the plan can be used again; calls between the failed one and this are
 * not to be relied on. */
int bsgemv_moe_device_status(bsgemv_moe_plan_t plan, void* stream);

/* Test hook, as bsgemv_plan_set_test_fault: in the plan's next calls block 0 of the first (product
 * 0: gate and up) or second (1: down) product leaves out the copies of stage `skip_stage` of its range
 * (-1: none), and all waits give up after wait_ns (0: the default).  (plan, 0, -1, 0) restores normal
 * calls. */
int bsgemv_moe_set_test_fault(bsgemv_moe_plan_t plan, int product, int skip_stage,
                              int64_t wait_ns);

/* Free the plan (synchronises the device first).  NULL is a no-op. */
int bsgemv_moe_destroy(bsgemv_moe_plan_t plan);

/*
 * Single-token attention of B sequences that share a prefix, over a paged cache: for sequence b
 * and query head h (kv head h / (Hq / Hkv)),
 *
 *     out[b, h] = sum over j < lens[b] of softmax_j(scale * q[b, h] . k_j) v_j
 *
 * Positions 0 .. prefix_len-1 are every sequence's (their K and V are read once for all), the
 * rest are a sequence's own.  Position j lies in row j % page_size of a page: of page
 * prefix_table[j / page_size] for the prefix, of page tables[b * table_stride + j / page_size]
 * for own positions (a page in which the prefix ends is read from prefix_table up to prefix_len
 * and from the sequence's table after it).  What pages hold outside these positions does not
 * matter, NaN included.  lens[b] is at most page_size times the entries of the sequence's row of
 * `tables`.  A slot with lens[b] < max(prefix_len, 1) holds no sequence: its
 * out rows are 0 and its lse -inf, and its row of `tables` is not read.
 *
 * q [B][Hq][D] with q_stride elements between sequences, out [B][Hq][D] contiguous, fp16 or bf16
 * like the cache.  k and v: element (page, head, row, d) of the cache at
 * page * page_stride + head * head_stride + row * row_stride + d elements, num_pages pages;
 * both layouts ([page][head][row][D] and [page][row][head][D]) are strides.  lse, if not NULL:
 * [B][Hq] fp32, log of the softmax's denominator with the maximum put back.  NaN among a row's
 * scores, or a score of +inf, gives NaN in its out and lse, NaN in a value its column (a weight of
 * 0 or not); a row all of whose scores are -inf gives NaN in out and -inf in lse.  Scores, softmax and
 * sums are fp32; the softmax numerators enter the second product in two parts of the cache's dtype, to
 * 2^-16 (bf16) or 2^-22 (fp16) of themselves.
 */
typedef struct bsgemv_attn_plan_s* bsgemv_attn_plan_t;

/* D one of 64, 128, 256; page_size a power of two from 8 to 1024; Hkv >= 1, Hq a multiple of Hkv
 * with Hq / Hkv <= 64 and Hq <= 1024; 1 <= max_B <= 1024.  act_bf16: 0 = fp16, 1 = bf16. */
int bsgemv_attn_plan(bsgemv_attn_plan_t* out, int act_bf16, int Hq, int Hkv, int D,
                     int page_size, int max_B);

/* Enqueue the attention of B (1 .. max_B) slots.  q, k, v, out 16-byte aligned, all strides
 * multiples of 8 elements; prefix_table, tables, lens int32 device memory (prefix_table may be
 * NULL when prefix_len == 0).  prefix_len is a host value: 0 <= prefix_len < 2^30.  Page ids
 * outside 0 .. num_pages-1 are read as zeros.  Strides that a TMA tensor map cannot describe (2^40
 * bytes or more): BSGEMV_ERR_UNSUPPORTED.  Deterministic: repeated calls are bit-identical. */
int bsgemv_attn_run(bsgemv_attn_plan_t plan, const void* q, int64_t q_stride, const void* k,
                    const void* v, int64_t page_stride, int64_t head_stride, int64_t row_stride,
                    int num_pages, const int32_t* prefix_table, int prefix_len,
                    const int32_t* tables, int64_t table_stride, const int32_t* lens, int B,
                    float scale, void* out, float* lse, void* stream);

/* Synchronise `stream`, then read and clear the plan's error word (as bsgemv_device_status).
 * BSGEMV_ERR_UNSUPPORTED: a call's lens are more than it can take.  Each is at most 2^30, and
 * Hkv * ceil(Hq / Hkv / 16) times the sum of (lens[b] - prefix_len) * D / 4096 + 4 over the slots has to
 * stay below 2^30 (16 TB of keys and values to read).  Beyond that a call may read none of them; the out
 * rows of its sequences are NaN then. */
int bsgemv_attn_device_status(bsgemv_attn_plan_t plan, void* stream);

/* Test hook, as bsgemv_plan_set_test_fault: in the plan's next calls the first warp of the streaming
 * kernel (kernel 0: a tile is 4096 / D positions, K and V) or the first block of the tensor-memory
 * prefix kernel (kernel 1: 64 positions, K and V in turn) leaves out the copy of tile `skip_tile` of its
 * range (-1: none), and all waits give up after wait_ns (0: the default).  (plan, 0, -1, 0) restores
 * normal calls. */
int bsgemv_attn_set_test_fault(bsgemv_attn_plan_t plan, int kernel, int skip_tile,
                               int64_t wait_ns);

/* Free the plan (synchronises the device first).  NULL is a no-op. */
int bsgemv_attn_destroy(bsgemv_attn_plan_t plan);

/*
 * Attention of new tokens over the paged cache: a chunk of a prompt, draft tokens to verify, single
 * tokens, in one ragged batch.  Rows starts[i] .. starts[i + 1] - 1 of q (starts: int32 [n + 1],
 * device, not decreasing) are the last tokens of sequence seqs[i], i < n, whose keys and values are
 * in the cache already: row r has position i_r = lens[seqs[i]] - (starts[i + 1] - r) and sees the
 * positions j of its sequence up to its own, the last `window` of them where window > 0:
 *
 *     t(r, h, j)  = scale * q[r, h] . k_j                  (kv head h / (Hq / Hkv))
 *     t           = cap * tanh(t / cap)                    where cap > 0
 *     t           = t + slopes[h] * (j - i_r)              where slopes is not NULL
 *     out[r, h]   = sum over j of softmax_j(t) v_j,        lse[r, h] = log of sum exp(t)
 *
 * Position j of sequence s lies in row j % page_size of page tables[s * table_stride + j /
 * page_size]; entries of tables past a sequence's last page are not read.  Rows of an entry whose
 * seqs is outside 0 .. num_seqs-1, and rows before a sequence's first position, get 0 in out and
 * -inf in lse; rows outside starts[0] .. starts[n] - 1 are left as they were.  A sequence counts with
 * max_pages * page_size tokens, and 2^30, at most.  What the cache holds in places that a row does not see does
 * not reach it, NaN and infinities included.
 *
 * q: head h of row r at q + r * q_stride + h * D elements, out [T][Hq][D] and lse [T][Hq] (fp32, or
 * NULL) contiguous, dtypes, cache layout and strides as bsgemv_attn_run.  NaN among a row's scores, or a
 * score of +inf, gives NaN in its out and lse; a row all of whose scores are -inf gets NaN in out and -inf
 * in lse.  Otherwise a column of out is infinite where an infinity is among the column's values that the
 * row sees, and NaN where infinities of both signs or NaN are (a weight of 0 or not).
 *
 * Scores, softmax and sums are fp32; numerators as in bsgemv_attn_run.  The tensor cores cut off what does
 * not fit when they add: a row that sees n positions is up to about 1.5e-9 n of itself too small.
 */
typedef struct bsgemv_chunk_plan_s* bsgemv_chunk_plan_t;

/* act_bf16, Hq, Hkv, D and page_size as bsgemv_attn_plan.  1 <= max_n <= 65536 entries and
 * 1 <= max_T < 2^24 rows a call, max_T * Hq below 2^28. */
int bsgemv_chunk_plan(bsgemv_chunk_plan_t* out, int act_bf16, int Hq, int Hkv, int D,
                      int page_size, int max_n, int max_T);

/* Enqueue the attention of T (1 .. max_T) rows in n (1 .. max_n) entries (a call without any is refused,
 * as bsgemv_attn_run's; bsgemv_cache_grow and _append return BSGEMV_OK).  cap: 0 for none, or > 0
 * with scale / cap and cap * log2(e) finite in fp32 (capped scores are right to 2^-20 of themselves
 * and the error of the scores); window: 0 for none, or >= 1; slopes: Hq fp32 (device) or NULL.
 * Alignment and strides as bsgemv_attn_run; table_stride >= max_pages.  Page ids outside 0 ..
 * num_pages-1 are read as zeros.  Deterministic: repeated calls are bit-identical (the bits of a row
 * may depend on the entries beside it: they decide where sums are cut). */
int bsgemv_chunk_run(bsgemv_chunk_plan_t plan, const void* q, int64_t q_stride, const void* k,
                     const void* v, int64_t page_stride, int64_t head_stride, int64_t row_stride,
                     int num_pages, const int32_t* tables, int64_t table_stride, int num_seqs,
                     int max_pages, const int32_t* lens, const int32_t* seqs,
                     const int32_t* starts, int n, int T, float scale, float cap, int window,
                     const float* slopes, void* out, float* lse, void* stream);

/* Synchronise `stream`, then read and clear the plan's error word (as bsgemv_device_status).
 * BSGEMV_ERR_UNSUPPORTED: a call's key tiles were more than it can count; its out rows are NaN. */
int bsgemv_chunk_device_status(bsgemv_chunk_plan_t plan, void* stream);

/* Test hook, as bsgemv_plan_set_test_fault: in the plan's next calls the first block of the
 * tensor-memory kernel (kernel 0: K and V tiles in turn) or the first warp of the streaming kernel
 * (kernel 1: a tile is 4096 / D positions, K and V) leaves out the copy of tile `skip_tile` of its
 * range (-1: none), and all waits give up after wait_ns (0: the default).  (plan, 0, -1, 0) restores
 * normal calls. */
int bsgemv_chunk_set_test_fault(bsgemv_chunk_plan_t plan, int kernel, int skip_tile,
                                int64_t wait_ns);

/* Free the plan (synchronises the device first).  NULL is a no-op. */
int bsgemv_chunk_destroy(bsgemv_chunk_plan_t plan);

/*
 * The pages of a cache.  The caller owns
 *
 *     pool    [planes][num_pages][page_bytes]   K and V of every layer, a plane each
 *     refs    [num_pages] int32                 sequences that hold the page; 0 = free
 *     tables  [max_seqs][max_pages] int32       pages of each sequence, -1 after the last
 *     lens    [max_seqs] int32                  tokens of each sequence
 *
 * in device memory; position j of sequence s lies in page tables[s][j / page_size].  All free
 * pages are alike: a page that is taken is always the free page with the lowest index, so the
 * state alone decides the result.  Lists of sequences and pages are int32 device arrays; an
 * entry outside its range is skipped.  No call synchronises.
 */
typedef struct bsgemv_cache_s* bsgemv_cache_t;

/* planes >= 1, num_pages >= 1 (below 2^24), page_bytes a positive multiple of 16, page_size >= 1,
 * 1 <= max_seqs <= 65536, max_pages >= 1 with max_seqs * max_pages below 2^31. */
int bsgemv_cache_plan(bsgemv_cache_t* out, int planes, int num_pages, int64_t page_bytes,
                      int page_size, int max_seqs, int max_pages);

/* Copy page src[i] to page dst[i] in every plane, i < n.  The pages of dst are distinct and none
 * is in src. */
int bsgemv_cache_copy(bsgemv_cache_t cache, void* pool, const int32_t* src, const int32_t* dst,
                      int n, void* stream);

/*
 * Slot children[i] becomes a copy of sequence parents[i], i < n <= max_seqs, all at once (a child
 * may be the parent of another entry): whole pages are shared, and a page that is only partly
 * filled is copied into a free page, so that both can grow.  What a child held before is released
 * first; children are distinct.  parents[i] == children[i] leaves the slot alone.
 * new_pages [n], if not NULL: the page taken for the copy, -1 where none was needed, -2 where the
 * pool had none left: that child becomes empty (earlier entries are served first).
 */
int bsgemv_cache_fork(bsgemv_cache_t cache, void* pool, int32_t* refs, int32_t* tables,
                      int32_t* lens, const int32_t* parents, const int32_t* children,
                      int32_t* new_pages, int n, void* stream);

/* Release sequences seqs[0 .. n-1] (distinct): their pages lose a reference, their rows become
 * -1 and their lengths 0. */
int bsgemv_cache_free(bsgemv_cache_t cache, int32_t* refs, int32_t* tables, int32_t* lens,
                      const int32_t* seqs, int n, void* stream);

/*
 * One more token for each of the sequences seqs[0 .. n-1] (distinct): lens grows by one, with a
 * page taken where the last one is full, and a copy of the last page where other sequences hold
 * it too.  A sequence that finds no free page (earlier entries are served first) or no room in
 * its row stays as it is; grown [n], if not NULL, is 1 or 0.
 */
int bsgemv_cache_extend(bsgemv_cache_t cache, void* pool, int32_t* refs, int32_t* tables,
                        int32_t* lens, const int32_t* seqs, int32_t* grown, int n, void* stream);

/*
 * Put one token's K and V of one layer at the last position (lens - 1) of each of the sequences
 * seqs[0 .. n-1]: for i < n, head h < heads and d: k[i * kv_stride + h * D + d] goes to element
 * h * head_stride + row * row_stride + d of its page in plane k_plane, and v likewise in v_plane.
 * 2-byte elements; D and the strides multiples of 8; k, v and pool 16-byte aligned.  Only for
 * sequences that the last bsgemv_cache_extend let grow: the last position of one that it left as it was
 * is a token already there, in a page that other sequences may hold, and is overwritten.
 */
int bsgemv_cache_write(bsgemv_cache_t cache, void* pool, const int32_t* tables,
                       const int32_t* lens, const int32_t* seqs, const void* k, const void* v,
                       int64_t kv_stride, int heads, int D, int64_t head_stride,
                       int64_t row_stride, int k_plane, int v_plane, int n, void* stream);

/*
 * counts[i] = starts[i + 1] - starts[i] more tokens for each of the sequences seqs[0 .. n-1]
 * (distinct), as bsgemv_cache_extend gives one: pages for all of them, and a copy of the last page
 * where it is partly filled and other sequences hold it too.  starts: int32 [n + 1] (device).
 * Entries are served in order, all of an entry's pages or none: one that finds too few pages left
 * stays as it is, and so does every entry after it that needs a page.  One with no room in its row
 * stays as it is and takes nothing; a count below 1 adds nothing.  grown [n], if not NULL, is 1
 * where the sequence has its tokens now, or 0.
 */
int bsgemv_cache_grow(bsgemv_cache_t cache, void* pool, int32_t* refs, int32_t* tables,
                      int32_t* lens, const int32_t* seqs, const int32_t* starts, int32_t* grown,
                      int n, void* stream);

/*
 * What is done to the queries and keys of new tokens before they are used: a norm over each head
 * (optional, with weights at the call) and the rotation of `rot` of its D elements by the token's
 * position,
 *
 *     y = x / sqrt(mean(x^2) + eps) * weight                 over the head's D elements
 *     (a, b) -> factor * (a cos f - b sin f, a sin f + b cos f),     f = position * freqs[p]
 *
 * for pair p < rot / 2: elements (p, p + rot / 2), or (2 p, 2 p + 1) with BSGEMV_ROPE_INTERLEAVED.
 * Elements from rot on are normalised only.  Angles are worked out modulo a turn in 64-bit fixed
 * point (to 2^-63 of a turn a position, with freqs as the doubles that they are) and rounded to fp32;
 * sines, norms and products are fp32, with one rounding at the end.
 */
typedef struct bsgemv_rope_s* bsgemv_rope_t;

enum bsgemv_rope_flags { BSGEMV_ROPE_INTERLEAVED = 1 };

/* act_bf16: 0 = fp16, 1 = bf16.  D a multiple of 16 up to 512; rot a multiple of 16, 0 <= rot <= D;
 * Hq, Hkv 1 .. 1024.  freqs: rot / 2 doubles in HOST memory, radians a position (finite, below 2^31;
 * NULL with rot == 0); factor: finite. */
int bsgemv_rope_plan(bsgemv_rope_t* out, int act_bf16, int Hq, int Hkv, int D, int rot, int flags,
                     const double* freqs, double factor);

/* Free the plan (synchronises the device first).  NULL is a no-op. */
int bsgemv_rope_destroy(bsgemv_rope_t rope);

/*
 * New tokens of one layer on their way into the cache: rows starts[i] .. starts[i + 1] - 1 of q, k
 * and v (starts: int32 [n + 1], device, not decreasing) are the last tokens of sequence seqs[i],
 * i < n: row r has position lens[seqs[i]] - (starts[i + 1] - r).  Queries, normalised and rotated
 * as `rope` says, go to q_out; keys likewise, and values as they are, to their places in the pages,
 * in planes k_plane and v_plane, as bsgemv_cache_write puts them: strides by which two heads or
 * rows of a page share an element, and one plane for both, are refused.  So a call follows
 * bsgemv_cache_grow (or _extend), for the entries that grew.
 *
 * q: head h of row r at q + r * q_stride + h * D elements (Hq heads), k and v likewise (Hkv heads),
 * q_out likewise; q_out may be q with the same stride.  q and q_out may be NULL together (keys and
 * values only), or k and v (queries only; pool, tables may be NULL then).  q_weight, k_weight: D
 * elements of the activation dtype, or NULL for no norm.  pos: int32 [T] positions for the rotation
 * (below zero allowed), or NULL for the positions in the sequences.  T: rows of the tensors.  Rows
 * outside starts[0] .. starts[n] - 1 or past T, rows of an entry whose seqs is outside 0 ..
 * max_seqs-1 and rows before a sequence's first position are left alone, in q_out and the pool; a
 * key whose page is not one of the pool's is not written.  q, k, v, q_out, weights and pool 16-byte
 * aligned, strides multiples of 8 elements; 0 <= n <= max_seqs, 0 <= T < 2^24.  The sequences are
 * distinct.
 */
int bsgemv_cache_append(bsgemv_cache_t cache, bsgemv_rope_t rope, void* pool,
                        const int32_t* tables, const int32_t* lens, const int32_t* seqs,
                        const int32_t* starts, int n, int T, const void* q, int64_t q_stride,
                        const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                        const void* q_weight, const void* k_weight, float eps,
                        const int32_t* pos, void* q_out, int64_t q_out_stride,
                        int64_t head_stride, int64_t row_stride, int k_plane, int v_plane,
                        void* stream);

/*
 * Move the live pages to the front: with L live pages, the i-th live page at or after L (in index
 * order) moves to the i-th free page before L, in every plane.  refs_out and tables_out (which
 * may be refs and tables themselves) get the new state, live_out [1] L; the moved pages' old
 * places keep their bytes, so tables that were read before stay readable until those pages are
 * taken again.  Entries of rows after a sequence's last page become -1.
 */
int bsgemv_cache_compact(bsgemv_cache_t cache, void* pool, const int32_t* refs,
                         const int32_t* tables, const int32_t* lens, int32_t* refs_out,
                         int32_t* tables_out, int32_t* live_out, void* stream);

/* Free the handle (synchronises the device first).  NULL is a no-op. */
int bsgemv_cache_destroy(bsgemv_cache_t cache);

/* Library version as MAJOR * 10000 + MINOR * 100 + PATCH. */
int bsgemv_version(void);

#ifdef __cplusplus
}
#endif

#endif /* BSGEMV_H_ */
