/*
 * migemm.h -- C ABI of a persistent, tile-scheduled, pipelined GEMM for
 * AMD Instinct MI355X (gfx950).
 *
 *   D = alpha * A * B + beta * C          (fp32 accumulation, bf16 D)
 *
 * A is M x K, B is K x N, C and D are M x N.  A and B are both bf16, or both
 * OCP fp8 e4m3 ("fn": largest finite 448, no infinities); C and D are bf16.
 * (The e4m3 instructions add eight products at a time, cut to the precision
 * that the scaled product's description below gives, before fp32 takes over.)
 *
 * The operation and its interface shape follow the CUTLASS SM90 "TMA warp-
 * specialized cooperative" GEMM kernel page: an MNK problem shape, separate
 * element types and strides for A, B, C and D, an epilogue that forms
 * alpha * accumulator + beta * C (the source C is loaded only when it is
 * needed), a feasibility check before launch (can_implement), a caller-owned
 * workspace with a size query, and a persistent grid sized from the device's
 * compute-unit count.  The tile hand-off of gemm_run_with_tile_consumer is the
 * producer acquire/commit and consumer wait/release protocol that CUTLASS
 * issue #2900 ("How to build a pipeline between epilogue and communication
 * warp groups?") asks for, so that a consumer stage can work on each finished
 * output tile; with MIGEMM_F_CONSUMER_OVERLAP it does so while the next
 * tile's main loop runs.
 *
 * Conventions shared by every entry point:
 *   - all sizes and strides are int64_t; strides are in ELEMENTS;
 *   - element (r, c) of an operand X is at X + r * x_rs + c * x_cs;
 *   - every device pointer is owned by the caller; the library never
 *     allocates device memory, never frees, and never synchronizes a stream;
 *   - a plan owns host memory only and is immutable after creation; one plan
 *     may be run concurrently on several streams; every entry point taking a
 *     plan first checks that it is live (created and not yet destroyed) and
 *     gives MIGEMM_ERR_INVALID_ARG otherwise, without reading it;
 *   - every call returns a migemm_status (0 = OK, negative = error) and never
 *     throws.  Argument, device and alignment errors are found before
 *     anything is launched; a launch failure reported by the HIP runtime gives
 *     MIGEMM_ERR_LAUNCH; a fault inside a kernel surfaces at the caller's next
 *     synchronization, as for any HIP kernel.
 */
#ifndef MIGEMM_H
#define MIGEMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element types (the pages keep ElementA/B/C/D separate). */
typedef enum migemm_dtype {
  MIGEMM_BF16 = 1,
  MIGEMM_FP8_E4M3 = 2,
  MIGEMM_INT8 = 3, /* where a description of an operator names it */
  MIGEMM_FP32 = 4  /* likewise */
} migemm_dtype;

typedef enum migemm_status {
  MIGEMM_OK = 0,
  MIGEMM_ERR_INVALID_ARG = -1, /* NULL pointer, negative size, bad stride, C NULL with beta != 0 */
  MIGEMM_ERR_UNSUPPORTED = -2, /* valid request this library does not implement (see below) */
  MIGEMM_ERR_MISALIGNED = -3,  /* a base pointer or leading stride is not 16-byte aligned */
  MIGEMM_ERR_DEVICE = -4,      /* no HIP device, wrong ordinal, or not gfx950 */
  MIGEMM_ERR_LAUNCH = -5,      /* the HIP runtime rejected the kernel launch */
  MIGEMM_ERR_TIMEOUT = -6,     /* a bounded hand-off wait expired (MIGEMM_F_HANDOFF_DEBUG) */
  MIGEMM_ERR_SCRATCH = -7      /* gemm_run_no_alloc: the plan needs more workspace than
                                  MIGEMM_NO_ALLOC_SCRATCH_BYTES */
} migemm_status;

/* Plan flags. */
#define MIGEMM_F_TILE_CONSUMER 0x1u /* plan may run gemm_run_with_tile_consumer */
/* Stream-K (the kernel page's stream-K scheduler and fixup): the tiles of the
 * last round are cut into K ranges shared by every workgroup, so that no
 * compute unit idles while others finish whole tiles; the partial sums of a
 * split tile are added through the workspace.  gemm_run only (UNSUPPORTED
 * with MIGEMM_F_TILE_CONSUMER).  MIGEMM_F_STREAM_K lets the plan choose it
 * where its cost model predicts a gain (moving the partials costs about as
 * much as 24 K stages of MFMA work); MIGEMM_F_STREAM_K_FORCE uses it whenever
 * K > 0.  gemm_plan_get_info reports the choice (stream_k_tiles). */
#define MIGEMM_F_STREAM_K 0x2u
#define MIGEMM_F_STREAM_K_FORCE 0x4u
/* With MIGEMM_F_TILE_CONSUMER (else INVALID_ARG): copy each tile to D_copy
 * inside the next tile's main loop, fetching it back from D, instead of right
 * after the tile's commit from the tile still staged in LDS (the row
 * statistics are folded right after the commit either way).  Same results
 * bit for bit.  The overlap is CUTLASS issue #2900's goal -- consumer work
 * running while the MMA waves start the next tile -- but here the consumer
 * work shares the MMA waves, and in the K loop it costs more than it does
 * on its own (about 2.5% of the 8192^3 bf16 kernel's time).  It is the form
 * for consumer work that waits on long transfers rather than computing. */
#define MIGEMM_F_CONSUMER_OVERLAP 0x8u
/* With MIGEMM_F_TILE_CONSUMER (else INVALID_ARG): debugging of the hand-off
 * ring.  gemm_plan_workspace_size then includes a debug area, which every
 * run (gemm_run too) needs and gemm_workspace_init zeroes:
 *   - each ring wait (acquire, wait) is bounded: after debug_wait_ticks of
 *     the device's 100 MHz real-time clock (0: 10^8, one second) it gives
 *     up, is counted, and the kernel goes on, so it always ends;
 *     gemm_debug_read then reports MIGEMM_ERR_TIMEOUT (results may be wrong);
 *   - every wave writes a trace record per tile of its workgroup: the clock
 *     at each step of the protocol and the ring's occupancy at its commit
 *     (migemm_debug_info describes the layout).
 * debug_force_wait > 0 adds that much to every acquire's target: a wait
 * that cannot pass, for testing the bounded wait itself. */
#define MIGEMM_F_HANDOFF_DEBUG 0x10u
/* Where gemm_run reads C (beta != 0).  With this flag: in the epilogue, after
 * the tile's K loop.  Without it, a plan whose workgroups each take one round
 * of whole tiles (tiles <= grid, not stream-K, K at least two stages) reads C
 * into LDS during the K loop's last two iterations, as the ring's slots fall
 * free -- the kernel page's separate C-load role, here taken by the MMA
 * waves -- so that half the read overlaps the last stages' MFMAs instead of
 * waiting in the epilogue; other plans read it in the epilogue.  The tile
 * consumer always reads C in the epilogue.  gemm_plan_get_info reports the
 * choice (c_in_k_loop).  Same results bit for bit either way. */
#define MIGEMM_F_C_IN_EPILOGUE 0x20u
/* Output tile height (the kernel page's tile shape, a compile-time choice
 * there; here two kernels).  Plans take 256 x 256 tiles, except that a
 * bf16 plan without MIGEMM_F_TILE_CONSUMER may take 192 x 256 tiles where
 * that gives each persistent workgroup less work: with T tiles on G
 * workgroups the work is ceil(T / G) tiles, and a 192-row tile takes about
 * 0.8 of a 256-row one's time (3/4 of the flops at a slightly lower rate),
 * so a problem whose 256-row tiles leave a poorly filled last round (8192 x
 * 1024: 128 tiles on 256 compute units) runs 4/3 as many smaller tiles in
 * one round.  With MIGEMM_F_STREAM_K the plan compares against stream-K too.  MIGEMM_F_TILE_M256 keeps 256 rows;
 * MIGEMM_F_TILE_M192 forces 192 (bf16 only, else UNSUPPORTED; INVALID_ARG
 * with MIGEMM_F_TILE_M256, MIGEMM_F_TILE_CONSUMER or a stream-K flag).  A
 * 192-row plan reads C (beta != 0) in the epilogue.  gemm_plan_get_info
 * reports the choice (tile_m, tiles_m).  Same results bit for bit either
 * way: each output's sum runs over K in the same order. */
#define MIGEMM_F_TILE_M256 0x40u
#define MIGEMM_F_TILE_M192 0x80u

/* Output tile of the persistent scheduler (and the hand-off unit); a plan
 * may report tile_m 192 instead (MIGEMM_F_TILE_M192). */
#define MIGEMM_TILE_M 256
#define MIGEMM_TILE_N 256

/*
 * Problem description (the pages' Arguments: problem shape, element types,
 * strides, hardware info).
 *
 * Layout rules checked by gemm_desc_validate:
 *   - M, N, K >= 0;
 *   - type pairs: (A, B, C, D) = (BF16, BF16, BF16, BF16) or
 *     (FP8_E4M3, FP8_E4M3, BF16, BF16);
 *   - each of A, B, C, D has exactly one unit stride, and its other stride
 *     is at least the extent of the contiguous dimension;
 *   - the non-unit stride times the element size is a multiple of 16 bytes
 *     (K itself may be anything, in every layout); a multiple of 128 bytes
 *     (64 bf16, 128 e4m3) runs faster: the kernels read 128-byte row
 *     segments, which then each fall in one cache line (4000 x 3000 x 5000
 *     bf16 with rows of 10000 and 6000 bytes: 9% slower than with 10112
 *     and 6144);
 *   - C and D have the same orientation (both row-major or both column-
 *     major); a column-major D is computed as D^T = B^T A^T;
 *   - the tile-consumer flag requires a row-major D;
 *   - the byte span of 256 rows (or K rows) of an operand fits in 2^31;
 *   - each operand, with all its batches, spans at most 2^47 bytes (else
 *     UNSUPPORTED; this also rejects strides whose products would wrap);
 *   - batches (the pages' rank-4 problem shape, L appended to MNK): L = 0 or
 *     1 is one product; for L > 1 matrix l of X starts x_bs * l elements
 *     after X, every x_bs >= 0 and x_bs times the element size a multiple of
 *     16 bytes; A, B and C may share a matrix between batches (x_bs = 0), D
 *     may not (d_bs is at least the extent of one D, so batches of D do not
 *     overlap).  The tile consumer's outputs are per batch too: row_sum and
 *     row_max are L x M x ceil(N/256), D_copy uses d_bs.
 * c_* fields are ignored when the caller will always pass beta == 0, but
 * must still describe a valid layout (use the same values as D).
 */
typedef struct migemm_desc {
  int64_t M, N, K;
  int32_t a_type, b_type, c_type, d_type; /* migemm_dtype */
  int64_t a_rs, a_cs;                     /* A: M x K */
  int64_t b_rs, b_cs;                     /* B: K x N */
  int64_t c_rs, c_cs;                     /* C: M x N */
  int64_t d_rs, d_cs;                     /* D: M x N */
  int32_t device;                         /* HIP device ordinal; must be gfx950 */
  uint32_t flags;                         /* MIGEMM_F_* */
  int32_t max_workgroups;                 /* 0: one persistent workgroup per CU;
                                             >0: cap on the persistent grid */
  int32_t reserved;                       /* must be 0 */
  int64_t L;                              /* batch count (0 or 1: one product) */
  int64_t a_bs, b_bs, c_bs, d_bs;         /* batch strides in elements (L > 1) */
  int64_t debug_wait_ticks;               /* MIGEMM_F_HANDOFF_DEBUG: wait budget (0: default) */
  int32_t debug_force_wait;               /* MIGEMM_F_HANDOFF_DEBUG: see there; else 0 */
  int32_t reserved2;                      /* must be 0 */
} migemm_desc;

/* What a plan chose (for tracing and tests). */
typedef struct migemm_plan_info {
  int64_t tiles_m, tiles_n, num_tiles;
  int32_t grid;            /* persistent workgroups launched */
  int32_t block_threads;   /* threads per workgroup (4 waves of 64) */
  int32_t lds_bytes;       /* LDS per workgroup (of the kernel gemm_run launches) */
  int32_t stages;          /* depth of the main-loop LDS ring */
  int32_t tile_m, tile_n, tile_k; /* output tile (tile_m 256, or 192: MIGEMM_F_TILE_M192) and
                                      K per pipeline stage (64 bf16, 128 e4m3) */
  int32_t swapped;         /* 1: column-major D, computed as D^T = B^T A^T */
  int32_t a_kmajor;        /* 1: A (after any swap) is K-contiguous */
  int32_t b_kmajor;        /* 1: B (after any swap) is K-contiguous */
  int32_t cu_count;        /* compute units of the device */
  int32_t handoff_slots;   /* depth of the tile hand-off ring */
  int64_t stream_k_tiles;  /* tiles cut into K ranges (0: every tile is taken whole) */
  int32_t stream_k_units_per_tile; /* K stages (tile_k each) per such tile */
  int32_t c_in_k_loop;     /* 1: with beta != 0, gemm_run reads C in the K loop's last two
                              iterations (else in the epilogue); see MIGEMM_F_C_IN_EPILOGUE */
  int64_t batches;         /* L (1 for one product) */
} migemm_plan_info;

typedef struct migemm_plan migemm_plan; /* opaque, host memory only */

/* Pure host check of a description; needs no device.  Returns MIGEMM_OK or
 * the error code gemm_plan_create would give before its device query.
 * Defined by: the kernel page (sm90_gemm_tma_warpspecialized_cooperative.hpp),
 * can_implement -- may this kernel run these arguments (problem rank,
 * tile-size and alignment rules), answered before any launch. */
int gemm_desc_validate(const migemm_desc* desc);

/* Validate, query the device (must be gfx950), choose the tile configuration
 * and the persistent grid, and return a plan in *out (set to NULL on error).
 * Errors: INVALID_ARG, UNSUPPORTED, MISALIGNED (strides), DEVICE.
 * Defined by: the kernel page (sm90_gemm_tma_warpspecialized_cooperative.hpp),
 * to_underlying_arguments (arguments -> kernel parameters, the persistent
 * grid's size from the device's SM count in hw_info) and get_grid_shape;
 * its device-side guard against the wrong architecture. */
int gemm_plan_create(const migemm_desc* desc, migemm_plan** out);

/* Free a plan (NULL is accepted and does nothing).  A pointer that is not a
 * live plan (destroyed already, or never created) gives INVALID_ARG and
 * frees nothing.  Destroying a plan while another thread is inside a call
 * on it is the caller's error (the liveness check catches stale handles,
 * not such races); runs already enqueued do not need the plan.  Host
 * memory only; the pages have no counterpart (their Params live in the
 * caller's object). */
int gemm_plan_destroy(migemm_plan* plan);

/* Copy the plan's choices into *out (grid, block, tiles, ring depths).
 * Defined by: the kernel page (sm90_gemm_tma_warpspecialized_cooperative.hpp),
 * get_grid_shape and get_block_shape, the launch geometry a caller queries. */
int gemm_plan_get_info(const migemm_plan* plan, migemm_plan_info* out);

/* Bytes of device workspace gemm_run needs.  Defined by: the kernel page
 * (sm90_gemm_tma_warpspecialized_cooperative.hpp), get_workspace_size -- the
 * epilogue's and the tile scheduler's workspace (stream-K partials) summed.
 * Plans without stream-K tiles need none: 0, and `workspace` arguments below
 * may then be NULL.  A stream-K plan needs grid x 512 KiB of fp32 partial
 * tiles (two per workgroup) plus one 32-bit arrival counter per stream-K tile
 * and wave (rounded up to 256 bytes). */
size_t gemm_plan_workspace_size(const migemm_plan* plan);

/* Make `workspace` (gemm_plan_workspace_size(plan) bytes of device memory,
 * 256-byte aligned, owned by the caller) ready for the plan's runs.  Defined
 * by: the kernel page (sm90_gemm_tma_warpspecialized_cooperative.hpp),
 * initialize_workspace on a stream.  Zeroes the arrival counters (and a
 * MIGEMM_F_HANDOFF_DEBUG plan's whole debug area), with a kernel
 * enqueued on `stream` (so it may be captured in a HIP graph).  Every run
 * that completes leaves the counters at zero again; call this before the
 * first run, after a run that did not complete, and before a workspace is
 * used with another plan.  A no-op returning OK when the size is 0.
 * Errors: INVALID_ARG (NULL plan, or NULL workspace with a nonzero size),
 * MISALIGNED, DEVICE (current device is not the plan's), LAUNCH. */
int gemm_workspace_init(const migemm_plan* plan, void* workspace, void* stream);

/* D = alpha*A*B + beta*C, enqueued on `stream` (a hipStream_t; NULL = the
 * null stream).  Defined by: the kernel page
 * (sm90_gemm_tma_warpspecialized_cooperative.hpp), the persistent kernel's
 * body -- each CTA takes output tiles from the tile scheduler, its producer
 * loads K stages into a multi-stage ring that its consumers drain into
 * accumulators, and the epilogue forms alpha * accumulator + beta * C (C
 * loaded only when needed) and stores D.  A, B, D must be non-NULL and 16-byte aligned; C may be NULL
 * only when beta == 0, in which case C is never read (it may hold NaN).
 * With K == 0, D = beta*C.  M == 0 or N == 0 is a no-op.  C may alias D only
 * with identical strides.  Asynchronous: returns once the kernel is queued.
 * `workspace`: NULL when gemm_plan_workspace_size(plan) is 0; otherwise that
 * many bytes, 256-byte aligned, prepared by gemm_workspace_init (else
 * INVALID_ARG / MISALIGNED).  Runs that share a workspace must not overlap
 * in time.  With stream-K the fp32 partial sums of a tile are added in the
 * order of their K ranges, so a plan gives the same D on every run; plans
 * with another grid size can round differently in the last bit. */
int gemm_run(const migemm_plan* plan, const void* A, const void* B, const void* C, void* D,
             float alpha, float beta, void* workspace, void* stream);

/* gemm_run, and in the same kernel a consumer stage fed through a 2-slot
 * tile hand-off ring.  Defined by: CUTLASS issue #2900 ("How to build a
 * pipeline between epilogue and communication warp groups?"), the requested
 * protocol -- producer acquire, store the tile, commit; consumer wait, work
 * on the tile, release -- with the producer's first acquires passing at once
 * (the kernel page starts producer pipeline states at the opposite phase;
 * the CuTe DSL task_scheduling.pipeline page names producer_acquire,
 * producer_commit and consumer_release): every finished 256 x 256 tile of D is committed by the
 * waves that stored it; the consumer work waits for the commit, reads the
 * tile as the epilogue staged it in LDS (with MIGEMM_F_CONSUMER_OVERLAP the
 * copy instead reads it back from D while the next tile's main loop runs),
 * and then releases the slot.  For
 * the tile at tile column t = n / 256 it writes, for each row r of the tile,
 * over the bf16 values x_j = D[r][256t + j] of the columns below N, widened
 * exactly to fp32:
 *   row_sum[r * ceil(N/256) + t] = s, the plain sequential fp32 sum in
 *       ascending column order: s = +0.0f, then s = s + x_j for j = 0, 1, ...
 *       (one rounding per addition),
 *   row_max[r * ceil(N/256) + t] = the largest x_j that is not a NaN, with
 *       -0 < +0 (IEEE 754-2019 maximumNumber); -inf if there is none,
 * and copies the tile bit for bit into D_copy (same strides as D).  Both
 * statistics therefore have exactly one correct value given D.  (The hand-off
 * issue leaves the consumer's work open -- "do something with the tile";
 * these are the statistics this library's consumer stage computes.)
 * row_sum and row_max are M x ceil(N/256) fp32, row-major, 4-byte aligned;
 * D_copy is 16-byte aligned and must not overlap D.  Requires a plan created
 * with MIGEMM_F_TILE_CONSUMER and a row-major D. */
int gemm_run_with_tile_consumer(const migemm_plan* plan, const void* A, const void* B,
                                const void* C, void* D, float alpha, float beta,
                                float* row_sum, float* row_max, void* D_copy,
                                void* workspace, void* stream);

/* What the hand-off debug area of a MIGEMM_F_HANDOFF_DEBUG plan holds.  The
 * trace starts trace_offset bytes into the workspace: for workgroup g
 * (0 .. grid-1), wave w (0 .. waves-1) and the workgroup's n-th tile (0 ..
 * trace_tiles-1), a record of trace_words uint64 at index
 * ((g * waves + w) * trace_tiles + n) * trace_words, holding the device
 * real-time clock (100 MHz) when the wave
 *   [0] began the tile's K loop, [1] ended it, [2] acquired the tile's ring
 *   slot, [3] committed the tile, [4] saw it committed by every wave (its
 *   consumer's wait), [5] stored the tile's first and [6] its last copy
 *   step, [7] released the slot,
 * then [8] the ring's occupancy right after this wave's commit (tiles
 * committed by every wave minus tiles released by every wave, over both
 * slots) and [9] the tile id (records of tiles a workgroup does not have
 * stay zero). */
typedef struct migemm_debug_info {
  uint32_t waits_given_up;     /* bounded waits that expired since the last init */
  uint32_t max_occupancy;      /* largest ring occupancy seen, in tiles */
  int64_t trace_offset;        /* bytes from the workspace to the first record */
  int32_t grid, waves, trace_tiles, trace_words;
} migemm_debug_info;

/* Synchronizes `stream`, then reads the debug header of a
 * MIGEMM_F_HANDOFF_DEBUG plan's workspace into *out.  The waits it reports
 * on are those of the hand-off protocol of CUTLASS issue #2900 (producer
 * acquire, consumer wait), bounded here so that a protocol fault ends as a
 * status rather than a hang.  Returns
 * MIGEMM_ERR_TIMEOUT if a bounded ring wait has given up since the last
 * gemm_workspace_init, else MIGEMM_OK (or INVALID_ARG for a plan without
 * the flag, a NULL argument; DEVICE if the copy fails). */
int gemm_debug_read(const migemm_plan* plan, const void* workspace, void* stream,
                    migemm_debug_info* out);

/* Size of the fixed device scratch of gemm_run_no_alloc: 64 MiB per device. */
#define MIGEMM_NO_ALLOC_SCRATCH_BYTES (64ll << 20)

/* gemm_run for callers that cannot allocate device memory (code under HIP
 * graph capture, tight serving loops, harnesses that forbid hipMalloc): the
 * same computation with the same plan, but a plan that needs a workspace
 * (stream-K) gets it from a fixed array inside the library instead of from
 * the caller.  The array is MIGEMM_NO_ALLOC_SCRATCH_BYTES of device memory
 * on every device the library runs on, held until the process ends; this
 * call allocates and frees nothing.  A plan whose gemm_plan_workspace_size
 * exceeds it gets MIGEMM_ERR_SCRATCH, with nothing launched (a stream-K plan
 * fits with up to about 120 workgroups; cap it with max_workgroups).  Each
 * call that uses the array first clears its arrival counters with a fill
 * kernel on `stream`.  Every call on one device shares that device's array:
 * calls whose executions overlap in time on one device race (use one stream,
 * or order them), and the array keeps the last call's contents.  Arguments,
 * results and the other errors are those of gemm_run. */
int gemm_run_no_alloc(const migemm_plan* plan, const void* A, const void* B, const void* C,
                      void* D, float alpha, float beta, void* stream);

/*
 * Operators around the product
 * ============================
 * What stands on either side of a GEMM in a large language model: the norm
 * that makes its input, the product of 8-bit rows, and the loss over a large
 * vocabulary.  Each has a description, a plan and runs, under the conventions
 * at the top of this file; a plan of one kind is refused by the calls of
 * another.  All matrices are row-major with a row stride *_rs in elements:
 * at least the columns (else INVALID_ARG), a multiple of 16 bytes (else
 * MISALIGNED), the matrix within 2^47 bytes (else UNSUPPORTED).  Base
 * pointers are 16-byte aligned (vectors of fp32: 4-byte, where not said
 * otherwise).  What lies between a row's columns and its stride is never
 * written, and its contents do not matter.  Every run is a number of kernel
 * launches on `stream`: it can be captured in a graph, gives the same bits on
 * every call (no atomics decide an order of additions), and keeps nothing
 * from one call for the next.  Workspaces need no initialization; calls that
 * share one must not overlap in time.
 */

/* Norm: the residual's addition and the root-mean-square norm of each row.
 *   h = bf16(x + r)                      (without a residual, h = x)
 *   rstd = 1 / sqrt(mean of h^2 + eps)   (fp32)
 *   y = bf16(h * rstd * weight), or, with y_type MIGEMM_FP8_E4M3,
 *   scale = max |h * rstd * weight| / 448 and y = e4m3(h * rstd * weight /
 *   scale), saturating at 448: the rows that gemm_scaled_run takes.  A row
 *   of zeros gets scale 0 and codes 0; a NaN in a row makes its scale NaN.
 * Gradients, with n = h * rstd and g = dy:
 *   dx = bf16(rstd * (g * weight - n * mean(g * weight * n)) + dh)
 *   dweight = sum over the rows of g * n  (fp32)
 * (dx is the gradient of h: of both x and r.)  Sums are fp32: rows whose sum
 * of squares passes 3e38 overflow.  cols is 1 .. 32768 (above: UNSUPPORTED);
 * rows may be 0. */
typedef struct migemm_norm_desc {
  int64_t rows, cols;
  int64_t x_rs, y_rs;        /* x: bf16; y: y_type */
  int64_t r_rs, h_rs;        /* the residual in and out (bf16); both 0: none */
  int64_t dy_rs, dx_rs;      /* backward pass (bf16); both 0: none */
  int64_t dh_rs;             /* the residual's gradient (bf16); 0: none added */
  float eps;                 /* > 0 and finite */
  int32_t y_type;            /* MIGEMM_BF16 or MIGEMM_FP8_E4M3 */
  int32_t device;            /* HIP device ordinal; must be gfx950 */
  int32_t reserved;          /* must be 0 */
} migemm_norm_desc;

typedef struct migemm_norm_plan migemm_norm_plan; /* opaque, host memory only */

int gemm_norm_desc_validate(const migemm_norm_desc* desc);
int gemm_norm_plan_create(const migemm_norm_desc* desc, migemm_norm_plan** out);
int gemm_norm_plan_destroy(migemm_norm_plan* plan);
/* Bytes of workspace the backward pass needs (256-byte aligned): one row of
 * fp32 column sums for each of the workgroups that walk the rows.  0 for a
 * plan without a backward pass. */
size_t gemm_norm_workspace_size(const migemm_norm_plan* plan);

/* The kernels a plan has chosen (for tuning and tests): the waves that share a
 * row and the 16-byte vectors of it that each lane holds, and the workgroups
 * that walk the rows backward (0 without a backward pass). */
typedef struct migemm_norm_info {
  int32_t forward_waves, forward_vectors;
  int32_t backward_waves, backward_vectors;
  int32_t backward_workgroups;
  int32_t cu_count;
} migemm_norm_info;
int gemm_norm_plan_get_info(const migemm_norm_plan* plan, migemm_norm_info* info);

/* r and h are given exactly when the plan has a residual, scale (fp32 [rows])
 * exactly when y is e4m3; rstd is fp32 [rows], weight bf16 [cols], 16-byte
 * aligned.  h may be x or r itself (same strides), and a bf16 y may be x. */
int gemm_norm_run(const migemm_norm_plan* plan, const void* x, const void* r, const void* weight,
                  void* h, void* y, float* scale, float* rstd, void* stream);

/* h is what the forward pass normed (stride h_rs with a residual, else x
 * with stride x_rs), rstd what it wrote.  dh is given exactly when the plan
 * has dh_rs.  dx may be dy or dh itself (same strides).  dweight is fp32
 * [cols], written whole (zeros for no rows). */
int gemm_norm_run_backward(const migemm_norm_plan* plan, const void* dy, const void* h,
                           const void* weight, const float* rstd, const void* dh, void* dx,
                           float* dweight, void* workspace, void* stream);

/* The product of 8-bit rows, each with its scale, and 8-bit weights with a
 * scale per output channel:
 *   d[m][n] = bf16(a_scale[m] * b_scale[n] * sum over k of a[m][k] b[n][k])
 * a is M x K and b N x K e4m3 (both K-contiguous: b_cs is the stride between
 * the columns of the K x N operand), d M x N bf16, rounded once from an fp32
 * sum.  Up to K = 256 that sum takes the exact products.  Above, the e4m3
 * matrix instructions first add the products of eight consecutive k (8 i to
 * 8 i + 7), each cut toward zero to a multiple of 2^-13 of the power of two of
 * the largest of the eight (a subnormal code counts as 2^-6 there): normally
 * distributed codes lose about 1e-5 of the sum of magnitudes by it, and beside
 * an outlier, products below 2^-13 of it among its eight are lost.  From one row to many: the plan chooses among kernels by the sizes,
 * and where it splits K a run needs a workspace for the parts' sums.
 * M, N and K may be 0 (K = 0: d is zero); 256 rows of a, b and d each span
 * less than 2^31 bytes (else UNSUPPORTED).  Strides of whole 128 bytes load
 * fastest, padded if need be (4000 x 3000 x 5000: 67 us with strides of 5008,
 * 54 with 5120). */
typedef struct migemm_scaled_desc {
  int64_t M, N, K;
  int64_t a_rs, b_cs, d_rs;
  int32_t device;
  int32_t reserved; /* must be 0 */
} migemm_scaled_desc;

typedef struct migemm_scaled_plan migemm_scaled_plan; /* opaque, host memory only */

int gemm_scaled_desc_validate(const migemm_scaled_desc* desc);
int gemm_scaled_plan_create(const migemm_scaled_desc* desc, migemm_scaled_plan** out);
int gemm_scaled_plan_destroy(migemm_scaled_plan* plan);
/* Bytes of workspace a run needs (256-byte aligned); 0: it may be NULL. */
size_t gemm_scaled_workspace_size(const migemm_scaled_plan* plan);

/* The kernel a plan has chosen (for tuning and tests). */
typedef struct migemm_scaled_info {
  int32_t tile_m, tile_n; /* rows and columns of D a workgroup takes at a time */
  int32_t lds_stages;     /* 128-byte stages of K in LDS at once; 0: straight to registers */
  int32_t splits;         /* ranges of K, added up by a second launch if more than 1 */
  int32_t exact;          /* 1: the codes are multiplied as bf16 */
  int32_t cu_count;
} migemm_scaled_info;
int gemm_scaled_plan_get_info(const migemm_scaled_plan* plan, migemm_scaled_info* info);

/* a_scale is fp32 [M], b_scale fp32 [N], both 16-byte aligned. */
int gemm_scaled_run(const migemm_scaled_plan* plan, const void* a, const float* a_scale,
                    const void* b, const float* b_scale, void* d, void* workspace, void* stream);

/* Softmax cross entropy over a vocabulary, from the hidden states x (rows x
 * hidden) and the output projection's weights w (vocab x hidden), both bf16,
 * without the logits in memory:
 *   logits = x w^T (fp32);   lse = log of the sum of exp(logits) of a row
 *   loss = lse - logits[target], 0 where target < 0 (a row that does not
 *   count: a prompt's token, padding), NaN where target >= vocab
 * and with g = (exp(logits - lse) - onehot(target)) * dloss
 *   dx = bf16(g w),   dw = bf16(g^T x)
 * where a row whose target is not in [0, vocab) has g = 0 exactly, whatever
 * x and dloss hold there: its dx is 0, and it adds nothing to dw.  lse is
 * written for every row.  Logits, sums and exponentials are fp32.  g, over the
 * significand of the largest |dloss| of the rows that count, is rounded to bf16
 * on its way into the two products, whose sums are fp32: one rounding of each
 * entry of g, 2^-8 at most, beside that of dx and dw themselves (with one dloss
 * for every row, as for a mean, the one-hot part is exact before the target's
 * probability is added to it).  rows may be 0, vocab and hidden are at
 * least 1; rows and vocab below 2^28, and 256 rows of each matrix span less
 * than 2^31 bytes (else UNSUPPORTED).  Strides of whole 128 bytes load fastest
 * here too (1001 x 32001 x 2000 forward: 150 us with strides of 2000 elements,
 * 125 with 2048). */
typedef struct migemm_vocab_loss_desc {
  int64_t rows, vocab, hidden;
  int64_t x_rs, w_rs;
  int64_t dx_rs, dw_rs; /* backward pass; both 0: none */
  int32_t device;
  int32_t reserved; /* must be 0 */
} migemm_vocab_loss_desc;

typedef struct migemm_vocab_loss_plan migemm_vocab_loss_plan; /* opaque, host memory only */

int gemm_vocab_loss_desc_validate(const migemm_vocab_loss_desc* desc);
int gemm_vocab_loss_plan_create(const migemm_vocab_loss_desc* desc, migemm_vocab_loss_plan** out);
int gemm_vocab_loss_plan_destroy(migemm_vocab_loss_plan* plan);
/* Bytes of workspace either run needs (256-byte aligned).  Forward: 8 bytes a
 * row (of up to 16384) and 16 to 128 vocabulary entries.  Backward: the rows
 * that count, copied together; one piece of g, 2 bytes a row and entry of as
 * many entries as fit 512 MiB, but 1024 at least, and 64 more a row; fp32 sums
 * of dx, 4 bytes a row and hidden unit, unless one workgroup finishes each of
 * its tiles; and where K is split, that many of dx or of the piece's dw, up to
 * 512 MiB each (all of them in whole tiles). */
size_t gemm_vocab_loss_workspace_size(const migemm_vocab_loss_plan* plan);

/* The kernels a plan has chosen (for tuning and tests): the tiles (rows x
 * columns) of the logits forward and backward and of the backward pass's two
 * products, the ranges of K that those split into, and the vocabulary entries
 * that the backward pass takes at a time.  0 without a backward pass. */
typedef struct migemm_vocab_loss_info {
  int32_t forward_tile_m, forward_tile_n;
  int32_t gradient_tile_m, gradient_tile_n;
  int32_t dx_tile_m, dx_tile_n, dx_splits;
  int32_t dw_tile_m, dw_tile_n, dw_splits;
  int32_t cu_count;
  int32_t pieces;
  int64_t piece;
} migemm_vocab_loss_info;
int gemm_vocab_loss_plan_get_info(const migemm_vocab_loss_plan* plan, migemm_vocab_loss_info* info);

/* target is int64 [rows]; loss and lse are fp32 [rows]. */
int gemm_vocab_loss_run(const migemm_vocab_loss_plan* plan, const void* x, const void* w,
                        const int64_t* target, float* loss, float* lse, void* workspace,
                        void* stream);

/* lse is what the forward run wrote, dloss fp32 [rows] the gradient of each
 * row's loss.  dx and dw are written whole. */
int gemm_vocab_loss_run_backward(const migemm_vocab_loss_plan* plan, const void* x, const void* w,
                                 const int64_t* target, const float* lse, const float* dloss,
                                 void* dx, void* dw, void* workspace, void* stream);

/* The product of int8 rows, each with its scale, and int8 weights with a scale
 * per output channel, with a bias per channel or none:
 *   d[m][n] = bf16(a_scale[m] * b_scale[n] * sum over k of a[m][k] b[n][k] + bias[n])
 * a is M x K and b N x K int8 (both K-contiguous, as the scaled product's), any
 * codes from -128 to 127; d is M x N bf16.  The sum is int32 and exact, then
 * rounded to fp32 (2^-24 of it); scales and bias are fp32, and the result is
 * rounded to bf16 once.  K is at most 131071 (more: UNSUPPORTED), so that no
 * sum leaves int32.  The factors are taken in the order sum, a_scale, b_scale,
 * each product in fp32: one that passes 3e38 on the way is infinite, whatever
 * stands behind it.  Otherwise sizes, strides and the workspace are as the
 * scaled product's. */
typedef struct migemm_int8_desc {
  int64_t M, N, K;
  int64_t a_rs, b_cs, d_rs;
  int32_t device;
  int32_t reserved; /* must be 0 */
} migemm_int8_desc;

typedef struct migemm_int8_plan migemm_int8_plan; /* opaque, host memory only */

int gemm_int8_desc_validate(const migemm_int8_desc* desc);
int gemm_int8_plan_create(const migemm_int8_desc* desc, migemm_int8_plan** out);
int gemm_int8_plan_destroy(migemm_int8_plan* plan);
/* Bytes of workspace a run needs (256-byte aligned); 0: it may be NULL. */
size_t gemm_int8_workspace_size(const migemm_int8_plan* plan);

/* The kernel a plan has chosen (for tuning and tests). */
typedef struct migemm_int8_info {
  int32_t tile_m, tile_n; /* rows and columns of D a workgroup takes at a time */
  int32_t lds_stages;     /* 128-byte stages of K in LDS at once; 0: straight to registers */
  int32_t splits;         /* ranges of K, added up by a second launch if more than 1 */
  int32_t cu_count;
} migemm_int8_info;
int gemm_int8_plan_get_info(const migemm_int8_plan* plan, migemm_int8_info* info);

/* a_scale is fp32 [M], b_scale and bias fp32 [N], all 16-byte aligned; bias may
 * be NULL. */
int gemm_int8_run(const migemm_int8_plan* plan, const void* a, const float* a_scale, const void* b,
                  const float* b_scale, const float* bias, void* d, void* workspace, void* stream);

/* bf16 rows to 8 bits with a scale each: the rows that gemm_int8_run (q_type
 * MIGEMM_INT8, top = 127) and gemm_scaled_run (MIGEMM_FP8_E4M3, top = 448) take.
 *   scale = max |x| / top  (fp32),   q = x * top / max |x|
 * q rounded to the nearest code, ties to even, as if from the exact quotient.
 * A row of zeros gets scale 0 and codes 0; a row with an infinity or a NaN gets
 * scale NaN and codes 0, so that its products are NaN.  cols is 1 .. 32768
 * (above: UNSUPPORTED); rows may be 0. */
typedef struct migemm_quantize_desc {
  int64_t rows, cols;
  int64_t x_rs, q_rs; /* x: bf16; q: q_type */
  int32_t q_type;     /* MIGEMM_INT8 or MIGEMM_FP8_E4M3 */
  int32_t device;
  int64_t reserved;   /* must be 0 */
} migemm_quantize_desc;

typedef struct migemm_quantize_plan migemm_quantize_plan; /* opaque, host memory only */

int gemm_quantize_desc_validate(const migemm_quantize_desc* desc);
int gemm_quantize_plan_create(const migemm_quantize_desc* desc, migemm_quantize_plan** out);
int gemm_quantize_plan_destroy(migemm_quantize_plan* plan);
/* 0: no run needs a workspace. */
size_t gemm_quantize_workspace_size(const migemm_quantize_plan* plan);

/* The kernel a plan has chosen (for tuning and tests): the waves that share a
 * row and the 16-byte vectors of it that each lane holds. */
typedef struct migemm_quantize_info {
  int32_t waves, vectors;
  int32_t cu_count;
} migemm_quantize_info;
int gemm_quantize_plan_get_info(const migemm_quantize_plan* plan, migemm_quantize_info* info);

/* scale is fp32 [rows]. */
int gemm_quantize_run(const migemm_quantize_plan* plan, const void* x, void* q, float* scale, void* stream);

/* Block norm: what stands between two blocks of a model, in one pass.  x is a
 * block's output, z its gate's input, r the residual:
 *   post_rstd = 1 / sqrt(mean of x^2 + eps),  u = x * post_rstd * post_weight
 *     (post_norm 0: u = x)
 *   h = residual_scale * r + branch_scale * sigmoid(z) * u    (z_rs 0: no gate,
 *     the sigmoid's place is 1)
 *   rstd = 1 / sqrt(mean of h^2 + eps),  y = h * rstd * weight
 * y is bf16, or e4m3 or int8 codes with a scale per row, max |y| / 448 or / 127
 * (the rows that gemm_scaled_run and gemm_int8_run take).  h is rounded to bf16
 * where it is stored; rstd, y and scale come from it before that.  A row of
 * zeros gets scale 0 and codes 0.  A row of h with an infinity or a NaN has a
 * NaN or infinite scale with e4m3, and with int8 a NaN scale and codes 0: its
 * products hold no number.  8-bit rows are made of h * weight in fp32: a row
 * where that passes 3e38 counts as one with an infinity.
 * Gradients, with h as it was stored, n = h * rstd, s = sigmoid(z), p = x *
 * post_rstd, g = dy:
 *   d = dh + rstd * (g * weight - n * mean(g * weight * n))
 *   dr = bf16(residual_scale * d);  dweight = sum over the rows of g * n (fp32)
 *   v = branch_scale * d;  dz = bf16(v * u * s * (1 - s))
 *   dx = bf16(post_rstd * (v * s * post_weight - p * mean(v * s * post_weight * p)))
 *     (post_norm 0: bf16(v * s));  dpost_weight = sum over the rows of v * s * p
 * Sums are fp32: rows whose sum of squares passes 3e38 overflow.  cols is
 * 1 .. 16384 (above: UNSUPPORTED); rows may be 0. */
typedef struct migemm_block_norm_desc {
  int64_t rows, cols;
  int64_t x_rs, r_rs, h_rs;    /* bf16 */
  int64_t y_rs;                /* y_type */
  int64_t z_rs;                /* the gate's input (bf16); 0: no gate */
  int64_t dy_rs, dx_rs, dr_rs; /* backward pass (bf16); all 0: none */
  int64_t dz_rs;               /* with a gate and a backward pass; else 0 */
  int64_t dh_rs;               /* the residual's gradient (bf16); 0: none added */
  float eps;                   /* > 0 and finite */
  float branch_scale, residual_scale; /* finite */
  int32_t post_norm;           /* 1: x is normed first; 0: it is not */
  int32_t y_type;              /* MIGEMM_BF16, MIGEMM_FP8_E4M3 or MIGEMM_INT8 */
  int32_t device;              /* HIP device ordinal; must be gfx950 */
} migemm_block_norm_desc;

typedef struct migemm_block_norm_plan migemm_block_norm_plan; /* opaque, host memory only */

int gemm_block_norm_desc_validate(const migemm_block_norm_desc* desc);
int gemm_block_norm_plan_create(const migemm_block_norm_desc* desc, migemm_block_norm_plan** out);
int gemm_block_norm_plan_destroy(migemm_block_norm_plan* plan);
/* Bytes of workspace the backward pass needs (256-byte aligned): for each of the
 * workgroups that walk the rows, a row of fp32 column sums, with post_norm two.
 * 0 for a plan without a backward pass. */
size_t gemm_block_norm_workspace_size(const migemm_block_norm_plan* plan);

/* The kernels a plan has chosen, as migemm_norm_info. */
typedef struct migemm_block_norm_info {
  int32_t forward_waves, forward_vectors;
  int32_t backward_waves, backward_vectors;
  int32_t backward_workgroups;
  int32_t cu_count;
} migemm_block_norm_info;
int gemm_block_norm_plan_get_info(const migemm_block_norm_plan* plan, migemm_block_norm_info* info);

/* z is given exactly when the plan has a gate, post_weight and post_rstd exactly
 * with post_norm, scale (fp32 [rows]) exactly when y is 8-bit.  post_weight and
 * weight are bf16 [cols], 16-byte aligned; post_rstd and rstd fp32 [rows].  h
 * may be x, z or r itself (same strides), and a bf16 y another of them. */
int gemm_block_norm_run(const migemm_block_norm_plan* plan, const void* x, const void* z, const void* r,
                        const void* post_weight, const void* weight, void* h, void* y, float* scale,
                        float* post_rstd, float* rstd, void* stream);

/* h, post_rstd and rstd are what the forward pass wrote.  dh is given exactly
 * when the plan has dh_rs; x may be NULL in a plan with neither a gate nor
 * post_norm.  dx, dr and dz may each be one of the bf16 matrices that come in
 * (same strides).  dweight and dpost_weight are fp32 [cols], written whole
 * (zeros for no rows); dpost_weight is given exactly with post_norm. */
int gemm_block_norm_run_backward(const migemm_block_norm_plan* plan, const void* dy, const void* dh,
                                 const void* x, const void* z, const void* h, const void* post_weight,
                                 const void* weight, const float* post_rstd, const float* rstd, void* dx,
                                 void* dz, void* dr, float* dpost_weight, float* dweight, void* workspace,
                                 void* stream);

/* Checkpoint: activations x (tokens x cols, bf16) kept in 8 bits for the
 * backward pass, and the gradient of the weights (out_cols x cols) of the
 * product that took them, from the kept form.
 * The kept form is e4m3 codes with a power of two for each 32 tokens of a
 * column (the last group may have fewer), the least that brings the group's
 * largest magnitude to 448 or below, but from 2^-109 to 2^119:
 *   e = that power's exponent + 127 (18 .. 246),  code = e4m3(x * 2^(127 - e))
 * rounded to nearest, ties to even; past 448 (x past 1.75 * 2^127) the code is
 * 448's.  An infinity or a NaN becomes the code NaN and does not count for the
 * power.  In memory: the codes [tokens / 16][ld][16 tokens], tokens rounded up
 * to 32 and ld = cols rounded up to 16, then the bytes e [tokens / 32][ld];
 * codes of tokens and columns past the last are 0 (e of such columns 18).
 *   weight_gradient: dw = sum over the tokens of dy[t][n] * code * 2^(e - 127)
 * dy is tokens x out_cols bf16; the products are exact and the sums fp32; dw is
 * out_cols x cols, bf16 (rounded once), or fp32, to which with accumulate the
 * sum is added.  tokens may be 0 (the gradient is then 0, or unchanged).
 * tokens below 2^31 - 64; 256 rows of dy and dw span less than 2^31 bytes,
 * and dw has fewer than 2^38 elements (else UNSUPPORTED). */
typedef struct migemm_checkpoint_desc {
  int64_t tokens, cols;
  int64_t x_rs;               /* bf16 */
  int64_t out_cols;           /* the weights' gradient; these three 0: none */
  int64_t dy_rs, dw_rs;       /* dy: bf16; dw: dw_type */
  int32_t dw_type;            /* MIGEMM_BF16 or MIGEMM_FP32 */
  int32_t accumulate;         /* 1: dw is added to (fp32 only); 0: written */
  int32_t device;
  int32_t reserved;           /* must be 0 */
} migemm_checkpoint_desc;

typedef struct migemm_checkpoint_plan migemm_checkpoint_plan; /* opaque, host memory only */

int gemm_checkpoint_desc_validate(const migemm_checkpoint_desc* desc);
int gemm_checkpoint_plan_create(const migemm_checkpoint_desc* desc, migemm_checkpoint_plan** out);
int gemm_checkpoint_plan_destroy(migemm_checkpoint_plan* plan);
/* Bytes of the kept form (16-byte aligned): one a token and column, and 1 / 32. */
size_t gemm_checkpoint_size(const migemm_checkpoint_plan* plan);
/* Bytes of workspace that weight_gradient needs (256-byte aligned); 0: it may
 * be NULL. */
size_t gemm_checkpoint_workspace_size(const migemm_checkpoint_plan* plan);

/* Where the kept form's parts lie, and the gradient's kernel (for tuning and
 * tests; its fields are 0 without one). */
typedef struct migemm_checkpoint_info {
  int64_t code_bytes, scale_bytes;
  int32_t tile_m, tile_n; /* rows and columns of dw a workgroup takes at a time */
  int32_t lds_stages;     /* stages of 64 tokens in LDS at once */
  int32_t splits;         /* ranges of the tokens, added up by a second launch if more than 1 */
  int32_t cu_count;
  int32_t reserved;
} migemm_checkpoint_info;
int gemm_checkpoint_plan_get_info(const migemm_checkpoint_plan* plan, migemm_checkpoint_info* info);

int gemm_checkpoint_pack(const migemm_checkpoint_plan* plan, const void* x, void* kept, void* stream);
/* x = bf16(code * 2^(e - 127)), exactly. */
int gemm_checkpoint_unpack(const migemm_checkpoint_plan* plan, const void* kept, void* x, void* stream);
int gemm_checkpoint_weight_gradient(const migemm_checkpoint_plan* plan, const void* dy, const void* kept,
                                    void* dw, void* workspace, void* stream);

/* Static text for a status code (never NULL).  No counterpart on the pages. */
const char* gemm_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* MIGEMM_H */
