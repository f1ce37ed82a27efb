/*
 * sdt.h -- C ABI of the shape-driven-tile library (libsdt.so) for GB300 (sm_103a).
 *
 * Two products with the tile-selection calls around them, the attention of a decode step
 * between them, and a layer's products in 8 bits with what makes their operands:
 *
 *   gemm_f16   C = A . B, fp16 in, fp32 accumulate, fp16 out, with the CTA tile
 *              chosen from the problem shape.
 *   gemv_m1    y = W . x for a single activation row (M = 1 decode), streaming a
 *              K-major weight matrix, bf16 or q8 (int8 + one fp16 scale per 32).
 *   paged_attn_m1  attention of one new token per request over a paged key-value
 *              cache (paged_tables, paged_append around it).
 *   gemm_fp8   C = A . W^T, fp8 values with a scale per 128 of k, fp32 sums
 *              (rms_norm_fp8, quant_fp8 before it, rope_qk after it).
 *
 * Conventions for every call in this header:
 *  - Pointers named A, B, C, x, W, scales, y are DEVICE pointers owned by the
 *    caller (typically PyTorch-allocated).  The library never frees, keeps or
 *    allocates device memory for them; it allocates no device memory at all.
 *  - `stream` is a cudaStream_t (NULL = the legacy default stream) owned by the
 *    caller.  Work is enqueued on it asynchronously; the library never
 *    synchronises on the hot path.  Kernel faults surface on the caller's next
 *    synchronising CUDA call, as with any CUDA kernel.
 *  - Layouts are tight row-major: A is MxK (row stride K), B is KxN (row stride
 *    N), C is MxN (row stride N).  W is [N][K] ("K-major": each output's K
 *    weights are contiguous), scales are [N][K/32].
 *  - Return value: SDT_OK (0) or a negative sdt_status.  Argument errors are
 *    detected on the host before anything is enqueued; the message of the last
 *    failure on the calling thread is available from sdt_last_error().
 *
 * Sources (the pages this library restates; cited by title and section):
 *  [P1] "Beating hipBLASLt on a Gaming GPU" -- sections "The result" (the
 *       pipelined fp16 GEMM) and "The part that actually mattered" (tile
 *       geometry chosen from how many blocks the grid yields).
 *  [P2] "mojo-baro" -- "Four rounds on the decode shape" (M=1, K=4096,
 *       N=12288 decode; K-major weights; q8 with a scale per 32 weights;
 *       several contiguous columns per thread with wide loads; an
 *       M=1-specialised kernel).
 *  [P3] FlyDSL pull request "Speed up the RDNA3 GEMM up to 1.85x by choosing
 *       the tile from the shape" -- "Changes" (pick_tile over feasible_tiles,
 *       opt-in measured sweep frozen into an artefact, k-loop start stagger with
 *       mask wraparound for power-of-two k-tile counts) and the third commit
 *       message (the K-scan that isolates power-of-two row strides).
 *  [P4] "Iteratively Tuning hipBLASLt TensileLite Kernels" -- "The Six Rounds"
 *       (split-K with a choice of reduction algorithm; workgroup mapping).
 */
#ifndef SDT_H
#define SDT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same object as cudaStream_t / CUstream; declared here so this header needs no CUDA headers. */
typedef struct CUstream_st *sdt_stream_t;

typedef enum sdt_status {
    SDT_OK = 0,
    SDT_ERR_NULL = -1,               /* a required pointer is NULL */
    SDT_ERR_ALIGN = -2,              /* a pointer is not 16-byte aligned */
    SDT_ERR_SHAPE = -3,              /* negative dims, no feasible tile, N or K not a multiple of 8,
                                        q8 with K not a multiple of 32 */
    SDT_ERR_UNSUPPORTED_DEVICE = -4, /* current device is not compute capability 10.3 (sm_103) */
    SDT_ERR_LAUNCH = -5,             /* the kernel launch was rejected by the CUDA runtime */
    SDT_ERR_TIMEOUT = -6,            /* a kernel gave up a bounded wait (read by sdt_check_device_status) */
    SDT_ERR_TILE = -7,               /* unknown tile id, or the forced tile is infeasible for the shape */
    SDT_ERR_TABLE = -8,              /* tune table could not be read or parsed */
    SDT_ERR_CUDA = -9,               /* another CUDA runtime / driver call failed */
    SDT_ERR_ARG = -10                /* another invalid argument (e.g. stagger value) */
} sdt_status;

/* ------------------------------------------------------------------------ */
/* Core calls                                                                */
/* ------------------------------------------------------------------------ */

/*
 * gemm_f16 -- C[M][N] = A[M][K] . B[K][N]; fp16 (IEEE binary16) operands,
 * fp32 accumulation on the tensor cores, C rounded to fp16 (nearest even).
 * [P1 "The result"; P3 "Changes"].
 *
 * The tile is the tune-table entry for (M,N,K) when one is loaded and
 * feasible, otherwise sdt_pick_tile(M,N,K).  With SDT_AUTOTUNE=1 in the
 * environment, the first call for a shape times every feasible tile on
 * `stream` (synchronising it) and remembers the fastest for later calls.
 * The k-loop stagger follows SDT_STAGGER: "auto" (default) staggers the
 * one-CTA tiles when the k-tile count is a power of two and leaves the
 * persistent and two-CTA tiles unstaggered (measured faster on GB300); "0" and
 * "1" force it off or on.
 *
 * Requirements: A, B, C 16-byte aligned; M, N, K >= 0.  M == 0 or N == 0 is a
 * no-op; K == 0 writes C = 0.  Otherwise some tile must divide the shape
 * (M % 64, N % 64, K % 64 == 0 and K >= 128 at the least) or SDT_ERR_SHAPE is
 * returned; shapes with ragged edges are not handled.
 */
int gemm_f16(int64_t M, int64_t N, int64_t K,
             const void *A, const void *B, void *C, sdt_stream_t stream);

/*
 * gemv_m1 -- y[n] = sum_k x[k] * W[n][k] for n < N  (M = 1 decode).
 * [P2 "Four rounds on the decode shape", rounds v1-v4].
 *
 *   x       bf16 [K]
 *   W       scales == NULL: bf16 [N][K];  scales != NULL: int8 [N][K] (q8)
 *   scales  NULL, or fp16 [N][K/32]: weight k of row n is
 *           q[n][k] * scales[n][k/32]; the scale multiplies each group sum.
 *   y       fp32 [N] (written, not accumulated into)
 *
 * Requirements: x, W, y 16-byte aligned (scales 2-byte aligned); K a
 * multiple of 8 (bf16) or 32 (q8); K, N <= 2^30.  N == 0 is a no-op; K == 0
 * writes y = 0.
 *
 * Launched with programmatic dependent launch, the kernel may start while the
 * previous kernel in `stream` is still running; before it waits for that
 * kernel it only asks L2 for the first rows of W (a prefetch, which cannot
 * observe stale data: L2 is where device memory is coherent), so results still
 * reflect everything the previous kernel wrote to x, W and scales.  q8 sums
 * each group exactly in int32 after scaling the group's activations to int16
 * by a power of two (exact for activations within a factor 2^7 of the group's
 * largest; otherwise off by at most 2^-15 of it).
 */
int gemv_m1(int64_t K, int64_t N, const void *x, const void *W,
            const void *scales, float *y, sdt_stream_t stream);

/* The two arms of gemv_m1 called explicitly (same contract; the q8 arm requires scales). */
int gemv_m1_bf16(int64_t K, int64_t N, const void *x, const void *W, float *y,
                 sdt_stream_t stream);
int gemv_m1_q8(int64_t K, int64_t N, const void *x, const void *W,
               const void *scales, float *y, sdt_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Tile ladder, feasibility and selection  [P3 "Changes"; P1 tile rule]      */
/* ------------------------------------------------------------------------ */

/* Static description of one tile of the ladder. */
typedef struct sdt_tile_desc {
    int id;           /* index into the ladder, 0 .. sdt_num_tiles()-1 */
    int BM, BN, BK;   /* output rows x columns covered (by the CTA pair when cta_group == 2), k-depth */
    int cta_group;    /* 1, or 2 for a two-CTA (cluster pair) tile */
    int stages;       /* depth of the shared-memory TMA/MMA ring */
    int threads;      /* threads per CTA */
    int smem_bytes;   /* dynamic shared memory per CTA, including alignment slack */
    int tmem_cols;    /* tensor-memory columns allocated per CTA */
    char name[24];    /* e.g. "128x256", "2cta_256x128" */
} sdt_tile_desc;

/* The ladder also holds "skinny" tiles, named s<BM>x<BN> (s128x16, s128x32), for
 * problems with few rows (M up to a few tens): gemm_ex and gemm_ex_splitk run
 * them on C^T = op(B)^T . op(A)^T so that the many output columns fill the MMA's
 * 128 rows, and write C back transposed.  They need A stored M x K (K
 * contiguous); sdt_feasible_tiles, pick_tile, gemm_f16, gemm_f16_splitk and the
 * tune table never use them. */
int sdt_num_tiles(void);
/* Fills *out for tile `tile_id`; SDT_ERR_TILE for an unknown id, SDT_ERR_NULL for out == NULL. */
int sdt_tile_info(int tile_id, sdt_tile_desc *out);
/* Static name of a tile, or NULL for an unknown id. */
const char *sdt_tile_name(int tile_id);

/*
 * Feasible tiles for (M,N,K) [P3 "Changes"]: a tile is feasible when it
 * (i) divides the shape (BM | M, BN | N, BK | K), (ii) can fill the pipeline
 * (at least two k-tiles), (iii) fits on chip (its shared memory within
 * `smem_limit` bytes per block, its accumulator within 512 TMEM columns).
 * Writes up to `cap` tile ids in ladder order to `ids` (may be NULL when
 * cap == 0) and returns how many tiles are feasible (which may exceed cap),
 * or a negative status.  The `_for` form needs no GPU; the plain form uses
 * the current device's opt-in shared-memory limit.
 */
int sdt_feasible_tiles_for(int64_t M, int64_t N, int64_t K, int smem_limit,
                           int *ids, int cap);
int sdt_feasible_tiles(int64_t M, int64_t N, int64_t K, int *ids, int cap);

/*
 * pick_tile [P3 "Changes"; P1 "The part that actually mattered"]: the
 * heuristic tile for (M,N,K) on a GPU with `sm_count` SMs, chosen among the
 * feasible tiles by an estimate of each one's run time: the waves (or, for
 * the persistent and two-CTA tiles, the rounds per worker) its grid makes on
 * `sm_count` SMs, priced by per-tile launch, k-tile, per-round, operand
 * streaming and co-residency costs fitted to a measured sweep.  Needs no GPU
 * and measures nothing.  Returns a tile id, or SDT_ERR_SHAPE when no tile is
 * feasible.
 * The plain form reads the current device's SM count and shared-memory limit.
 */
int sdt_pick_tile_for(int64_t M, int64_t N, int64_t K, int sm_count, int smem_limit);
int sdt_pick_tile(int64_t M, int64_t N, int64_t K);

/*
 * The launcher rule of [P1 "The part that actually mattered"] as printed for
 * a 96-unit card and scaled to `units`: count the 128x128-equivalent blocks
 * (M/128)*(N/128); >= units -> the 128x128 tile, >= 2*units/3 -> 64x128,
 * else 64x64.  Returns that tile's id (the seed the fitted heuristic grew
 * from; kept for comparison).
 */
int sdt_seed_tile(int64_t M, int64_t N, int units);

/*
 * gemm_f16 with a forced tile (for sweeps).  `stagger`: -1 = as gemm_f16
 * (SDT_STAGGER / auto), 0 = off, 1 = on when the k-tile count is a power of
 * two (otherwise silently off) [P3 "Changes", third commit message].
 * SDT_ERR_TILE if the tile is unknown or infeasible for the shape.
 */
int gemm_f16_with_tile(int64_t M, int64_t N, int64_t K,
                       const void *A, const void *B, void *C, sdt_stream_t stream,
                       int tile_id, int stagger);

/*
 * gemm_ex -- the general form: caller row strides, transposed operands, bf16,
 * and shapes no tile divides [P3 "Changes": the row strides are taken from the
 * caller's tensors; the measured layouts are TN and NN; P3 "Performance" runs
 * bf16].  C[M][N] (row stride ldc) = op(A) . op(B) with fp32 accumulation:
 *   op(A): layout without SDT_LAYOUT_A_T: A is M x K row-major (lda >= K);
 *          with it, A is stored K x M (lda >= M), i.e. A^T is given.
 *   op(B): without SDT_LAYOUT_B_T: B is K x N row-major (ldb >= N);
 *          with it, B is stored N x K (ldb >= K), i.e. B^T is given ("TN" is
 *          SDT_LAYOUT_B_T: C = A . (B^T)^T).
 *   dtype: SDT_DTYPE_F16 or SDT_DTYPE_BF16 for A, B and C alike.
 * Any M, K >= 0; N a multiple of 8; lda, ldb, ldc multiples of 8 (16-byte
 * rows) at least the row lengths above; pointers 16-byte aligned.  Tiles
 * overhang ragged edges: the TMA reads zeros outside the operands and the
 * epilogue writes only inside C.  tile_id -1 picks with sdt_pick_tile_any_for's
 * model; a forced tile needs only to fit on chip.  The k-loop stagger follows
 * SDT_STAGGER as in gemm_f16.  Errors: SDT_ERR_SHAPE (N % 8, dims > 2^30),
 * SDT_ERR_ARG (strides, dtype, layout), SDT_ERR_ALIGN, SDT_ERR_NULL,
 * SDT_ERR_TILE.
 */
#define SDT_DTYPE_F16 0
#define SDT_DTYPE_BF16 1
#define SDT_LAYOUT_A_T 1
#define SDT_LAYOUT_B_T 2
int gemm_ex(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, const void *B, int64_t ldb,
            void *C, int64_t ldc, int dtype, int layout, int tile_id, sdt_stream_t stream);
/*
 * gemm_f16_ws / gemm_ex_ws -- gemm_f16 / gemm_ex with a caller workspace that lets
 * the two-CTA tiles split the contraction of their last round [P3, third commit
 * message: persistent workgroups and the grid tail when the tile count is not a
 * multiple of the slot count; P4 "The Six Rounds": splitting the contraction, and
 * Stream-K's decomposition of the iteration space, of which this is the special case
 * "whole tiles, then the last partial wave split in K"].
 *
 * A two-CTA launch runs T output tiles on P = SMs/2 pairs.  When L = T mod P tiles
 * are left for a last round (P - L pairs idle), each of them may run as S full-width
 * items over consecutive k-ranges (L*S <= P, 2 <= S <= nK) instead of gemm_f16's form
 * (whole, or two half-width items).  Split 0 takes the first k-tiles and is made
 * longer than the others (sdt_pair_tail_plan's split0_ktiles) so that it normally
 * finishes last.  An item that finishes while another split is still running writes
 * its fp32 partial to the workspace and counts its arrival; the last to finish adds
 * the S partials in split order (so the result does not depend on the order of
 * arrival) and writes C.  The form is chosen per launch by a cost estimate (on GB300
 * it splits at 4096^3 and above and keeps the half-width items at 2560^3, where 40
 * k-tiles leave too little to hide the sum); gemm_ex_ws's tail_splits forces it: -1
 * estimate, 0 never split, 2..8
 * that count (lowered to what L*S <= P, nK and the shared memory for the partials'
 * copies allow: at most 7 with the current tiles; below 2 it is not split).
 * Every other tile, and a launch with no partial last round, runs exactly as
 * gemm_f16 / gemm_ex would.  Results may differ from gemm_f16's in the last bits
 * (the split tiles add their k-ranges in another order); integer-valued products
 * are identical.
 *
 * Workspace: NULL runs exactly gemm_f16 / gemm_ex.  Otherwise device memory owned
 * by the caller, 256-byte aligned, at least sdt_gemm_workspace_bytes() bytes (the
 * 1 MiB counter region of the split-K workspaces, then one 256 x 256 fp32 slot per
 * SM pair: 20 MiB on a 152-SM GPU, for any shape).  Its counters must be zero before
 * the first call (sdt_splitk_workspace_init); every completed call leaves them zero,
 * so a workspace zeroed once serves any sequence of calls, and it may be shared with
 * the split-K calls.  Calls that share a workspace must not overlap on the GPU.
 * After a call that reported a device error (sdt_check_device_status), zero it again.
 * Arguments and errors otherwise as gemm_f16 / gemm_ex, plus SDT_ERR_ALIGN and
 * SDT_ERR_ARG for the workspace and SDT_ERR_ARG for tail_splits outside -1, 0, 2..8.
 */
int gemm_f16_ws(int64_t M, int64_t N, int64_t K, const void *A, const void *B, void *C, void *workspace,
                size_t workspace_bytes, sdt_stream_t stream);
int gemm_ex_ws(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, const void *B, int64_t ldb,
               void *C, int64_t ldc, int dtype, int layout, int tile_id, int tail_splits, void *workspace,
               size_t workspace_bytes, sdt_stream_t stream);
/* Workspace bytes gemm_f16_ws / gemm_ex_ws accept on the current device (0 on error),
 * and on a GPU with sm_count SMs (needs no GPU). */
size_t sdt_gemm_workspace_bytes(void);
size_t sdt_gemm_workspace_bytes_for(int sm_count);
/*
 * The last-round plan of two-CTA tile `tile_id` on M x N x K with sm_count SMs and
 * smem_limit bytes of shared memory per block (needs no GPU): items [0, *tail_start)
 * are whole tiles, items [*tail_start, *num_items) the last round's, as *splits
 * k-ranges per tile (*splits >= 2; split 0 has *split0_ktiles k-tiles, the others
 * share the rest evenly) or two half-width items per tile (*splits == 0,
 * *num_items > *tail_start); *tail_start == *num_items means whole tiles throughout.
 * with_workspace != 0 plans as gemm_ex_ws with `tail_splits`, 0 as gemm_ex.
 * SDT_ERR_TILE for a tile that is not two-CTA, SDT_ERR_ARG for bad sizes.
 */
int sdt_pair_tail_plan(int64_t M, int64_t N, int64_t K, int tile_id, int sm_count, int smem_limit,
                       int with_workspace, int tail_splits, int *tail_start, int *num_items, int *splits,
                       int *split0_ktiles);
/* pick_tile's cost model over every tile for any shape (tiles may overhang); needs no GPU. */
int sdt_pick_tile_any_for(int64_t M, int64_t N, int64_t K, int sm_count, int smem_limit);
/*
 * The run-time estimate (microseconds) pick_tile gives tile `tile_id` on an M x N x K
 * problem with `sm_count` SMs (228 KiB of shared memory per SM), whether or not the
 * tile divides the shape or is a candidate; a negative status (SDT_ERR_TILE, SDT_ERR_ARG)
 * for an unknown tile or a dimension outside 1..2^30.  Needs no GPU.
 */
double sdt_tile_estimate_us(int tile_id, int64_t M, int64_t N, int64_t K, int sm_count);

/*
 * Split-K [P4 "The Six Rounds", the "Split-K" step: the contraction is split
 * across CTAs and the partial results are reduced; the page distinguishes a
 * reduction in a separate pass from one inside the single kernel].
 *
 * Output tile t of a one-CTA-per-tile ladder rung (64x64, 64x128, 128x64,
 * 128x128, 128x256) is computed by `splits` CTAs, CTA s accumulating k-tiles
 * [s*ceil(nK/splits), ...) (nK = K/64) and writing an fp32 partial tile to the
 * caller's workspace; the partials are summed in split order (independent of
 * arrival order) and rounded once to fp16:
 *   SDT_SPLITK_REDUCE_KERNEL  a second kernel sums the partials;
 *   SDT_SPLITK_IN_KERNEL      the last CTA of each tile to finish (per-tile
 *                             arrival counter in the workspace) sums them and
 *                             resets its counter to zero.
 * `splits` is rounded down to the count that leaves no split empty.
 * tile_id < 0 picks tile and splits with sdt_pick_splitk_for (then splits <= 0
 * takes the picked count).  The k-loop stagger is not applied.
 *
 * Workspace: device memory owned by the caller, 256-byte aligned, at least
 * sdt_splitk_workspace_bytes(M,N,K,tile_id,splits) bytes: a fixed 1 MiB region
 * of u32 counters (the in-kernel reduction uses one per output tile, at most
 * 262144 tiles; stream-K one per tile and TMEM lane quarter), then fp32
 * partials [splits][M][N].  The counter region has the same place and size in
 * every configuration.  The counters must be zero before the first SDT_SPLITK_IN_KERNEL call on a
 * workspace (sdt_splitk_workspace_init zeroes a workspace on `stream`); every
 * completed call leaves them zero again and writes partials only after the
 * counter region, so a workspace zeroed once serves any sequence of split-K
 * calls (any shape, tile, split count or algorithm) that fit in it.  Calls that
 * share a workspace must not overlap on the GPU.  Same operand requirements as gemm_f16 (tight row-major,
 * 16-byte aligned; tile dims divide M, N; K % 64 == 0).
 * Errors: SDT_ERR_TILE (tile without split-K form or not dividing the shape),
 * SDT_ERR_ARG (splits out of 1..nK, unknown algo, workspace too small),
 * SDT_ERR_ALIGN, SDT_ERR_NULL, as well as gemm_f16's.
 */
#define SDT_SPLITK_REDUCE_KERNEL 0
#define SDT_SPLITK_IN_KERNEL 1
#define SDT_SPLITK_STREAM 2        /* stream-K, fix-up by the last CTA to arrive; see sdt_streamk_workspace_bytes */
#define SDT_SPLITK_STREAM_REDUCE 3 /* stream-K, fix-up by a second kernel over the whole GPU */
int gemm_f16_splitk(int64_t M, int64_t N, int64_t K, const void *A, const void *B, void *C,
                    void *workspace, size_t workspace_bytes, int tile_id, int splits, int algo,
                    sdt_stream_t stream);
/* Bytes of workspace gemm_f16_splitk needs (0 for an invalid combination, including a
 * dimension above 2^30 or more than 2^30 - 1 output tiles, which the launch refuses). */
size_t sdt_splitk_workspace_bytes(int64_t M, int64_t N, int64_t K, int tile_id, int splits);
/* Zero a split-K workspace on `stream` (its counters must start at zero). */
int sdt_splitk_workspace_init(void *workspace, size_t workspace_bytes, sdt_stream_t stream);
/*
 * Heuristic (tile, splits) for split-K on a GPU with `sm_count` SMs: the
 * pick_tile cost model with K shared among the splits plus the reduction's
 * fp32 traffic, minimised over the split-K tiles and 1..32 splits.  splits == 1
 * means splitting does not pay.  Needs no GPU.
 */
int sdt_pick_splitk_for(int64_t M, int64_t N, int64_t K, int sm_count, int smem_limit,
                        int *tile_id, int *splits);

/*
 * gemm_ex_splitk -- split-K in gemm_ex's general form [P4 "The Six Rounds",
 * the split-K step, with the operands of P3 "Changes"]: caller row strides, either
 * transposed operand, fp16 or bf16, and shapes no tile divides.  Arguments and
 * requirements as gemm_ex, plus the split-K arguments of gemm_f16_splitk.
 * The partial planes cover whole tiles: the 1 MiB counter region, then [splits][ceil(M/BM)*BM][ceil(N/BN)*BN] fp32; the
 * workspace (shareable with gemm_f16_splitk calls) must hold
 * sdt_splitk_ex_workspace_bytes(M,N,K,tile_id,splits) bytes (256-byte
 * aligned; counters zero before the first SDT_SPLITK_IN_KERNEL call, as for
 * gemm_f16_splitk).  The reduction writes only inside C (row stride ldc), in
 * the operands' type.  tile_id < 0 picks with sdt_pick_splitk_any_for (then
 * splits <= 0 takes the picked count).  Errors as gemm_ex and gemm_f16_splitk.
 */
int gemm_ex_splitk(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, const void *B, int64_t ldb,
                   void *C, int64_t ldc, int dtype, int layout, void *workspace, size_t workspace_bytes,
                   int tile_id, int splits, int algo, sdt_stream_t stream);
/* Bytes of workspace gemm_ex_splitk needs for any shape (0 for a tile without split-K form,
 * splits outside 1..ceil(K/64), a dimension outside 1..2^30, or more than 2^30 - 1 output
 * tiles: the shapes the launch refuses). */
size_t sdt_splitk_ex_workspace_bytes(int64_t M, int64_t N, int64_t K, int tile_id, int splits);
/*
 * Stream-K [P4 "The Six Rounds", the last round "Stream-K": a fixed grid of
 * workgroups shares the whole iteration space instead of the contraction being
 * split per tile; a workgroup's share may end inside an output tile, and the
 * partial tiles are fixed up afterwards].  algo = SDT_SPLITK_STREAM in
 * gemm_f16_splitk / gemm_ex_splitk, with `splits` read as the CTA count G
 * (<= 0: one CTA per SM slot, sdt_streamk_ctas; lowered to the unit count when
 * larger).  The units are (output tile, 64-deep k-tile) pairs, tiles in banded
 * raster order and k-tiles in order; CTA g takes units
 * [floor(g*U/G), floor((g+1)*U/G)).  Whole tiles are stored directly; a CTA's
 * first and last tile may be partial: it writes an fp32 partial tile to its
 * slots (2g, 2g+1) and counts its arrival on per-(tile, TMEM lane quarter)
 * counters; the last CTA to arrive sums the tile's partials in CTA order,
 * writes C and zeroes the counter (SDT_SPLITK_STREAM), or a second kernel sums
 * every shared tile's partials in the same order (SDT_SPLITK_STREAM_REDUCE; the
 * counters are not used).  Same tiles as split-K (the one-CTA rungs
 * and the skinny tiles), any shape and layout gemm_ex takes.
 * Workspace: the 1 MiB counter region shared with split-K (zero before the
 * first call, left zero by every completed call), then 2*G fp32 tiles of
 * BM x BN: sdt_streamk_workspace_bytes(M,N,K,tile_id,G) bytes (G >= 1, taken
 * as at most the unit count; 0 for
 * a tile without stream-K form, a dimension outside 1..2^30, more than 65536
 * output tiles or more than 2^20 CTAs).
 */
size_t sdt_streamk_workspace_bytes(int64_t M, int64_t N, int64_t K, int tile_id, int ctas);
/* Default stream-K CTA count of a tile: SMs x CTAs of its kernel per SM (needs no GPU). */
int sdt_streamk_ctas_for(int tile_id, int sm_count, int smem_limit);
/* The same on the current device. */
int sdt_streamk_ctas(int tile_id);
/* sdt_pick_splitk_for's model over the split-K tiles for any shape (tiles may overhang). */
int sdt_pick_splitk_any_for(int64_t M, int64_t N, int64_t K, int sm_count, int smem_limit,
                            int *tile_id, int *splits);

/*
 * gemm_f16_splitk_noalloc -- gemm_f16_splitk (SDT_SPLITK_REDUCE_KERNEL) with its
 * workspace in a fixed 16 MiB array that the library holds in device memory,
 * so the call allocates nothing.  The pages have no counterpart; this is an
 * interface for callers that cannot allocate device memory where they
 * multiply: code that must not synchronise the device (cudaMalloc and
 * cudaFree can), plugin hosts that give a kernel library a fixed memory
 * budget and no allocator, latency-critical loops that forbid allocator calls.
 *
 * Arguments as gemm_f16_splitk, minus the workspace and the algorithm
 * (tile_id < 0 picks tile and splits).  The array holds the workspace layout
 * of gemm_f16_splitk: the 1 MiB counter region, then the fp32 partials, so
 * the partials get 15 MiB (sdt_splitk_workspace_bytes must be at most 16 MiB:
 * e.g. 1024x1024 with 3 splits, 512x512 with 15).  A given split count whose
 * workspace exceeds that is rejected with SDT_ERR_ARG and a message naming
 * the sizes; a split count the call picks itself (tile_id < 0, splits <= 0)
 * is lowered until it fits, and only a shape that does not fit unsplit is
 * rejected.  K == 0 writes C = 0 whatever tile and splits say.  The first
 * call on each device looks up the array's device address
 * (cudaGetSymbolAddress) with that device current; make that first call
 * before any stream capture.  Every GPU on which the library's module holding
 * the array is loaded keeps the 16 MiB until the process exits.  All calls
 * share the array: nothing in it has to start at zero (each call overwrites
 * the partials it reads), but calls that overlap on the GPU race on it and
 * corrupt each other's results.
 */
int gemm_f16_splitk_noalloc(int64_t M, int64_t N, int64_t K, const void *A, const void *B, void *C,
                            int tile_id, int splits, sdt_stream_t stream);

/*
 * Frozen tune table [P3 "Changes": the measured sweep can be frozen into an
 * offline artefact].  Text file, one entry per line: "M N K tile_name
 * [stagger]"; '#' starts a comment.  Loading replaces the current table.
 * Entries whose tile is infeasible for their shape are rejected
 * (SDT_ERR_TABLE, table left unchanged).  The table named by the environment
 * variable SDT_TUNE_TABLE is loaded on the first gemm_f16 call.
 * sdt_tune_table_lookup returns the tile id for a shape or -1.
 */
int sdt_load_tune_table(const char *path);
void sdt_clear_tune_table(void);
int sdt_tune_table_size(void);
int sdt_tune_table_lookup(int64_t M, int64_t N, int64_t K);

/* ------------------------------------------------------------------------ */
/* Paged key-value cache: one decode step's attention                        */
/* ------------------------------------------------------------------------ */

/*
 * A cache of num_pages pages of page_size tokens.  Token t of page p holds, for each of
 * kv_heads heads, head_dim contiguous keys and values, at element
 * p * k_page + t * k_token + h * k_head of k (v likewise), so pages may lie token by token
 * or head by head.  dtype SDT_DTYPE_F16 or SDT_DTYPE_BF16: 16-bit elements, head_dim a
 * multiple of 8 up to 256, base and strides multiples of 16 bytes.  SDT_DTYPE_Q8: int8
 * elements with one fp16 scale per 32 (element e of a head is q[e] * scale[e / 32], as in
 * gemv_m1_q8); head_dim a multiple of 64 up to 256; the scales have strides of their own,
 * head_dim / 32 contiguous, base and strides multiples of 4 bytes (8 with head_dim 128).
 * num_pages * page_size < 2^31; strides up to 16 GiB, offsets of any size.
 */
#define SDT_DTYPE_Q8 2
typedef struct sdt_paged_cache {
    void *k, *v;
    void *k_scales, *v_scales; /* NULL unless q8 */
    int64_t num_pages, page_size, kv_heads, head_dim;
    int64_t k_page, k_token, k_head; /* strides in elements */
    int64_t v_page, v_token, v_head;
    int64_t ks_page, ks_token, ks_head;
    int64_t vs_page, vs_token, vs_head;
    int dtype;
} sdt_paged_cache;

/*
 * paged_tables -- block tables and slot maps of a step, from the requests' lengths.
 * (The calls with many arguments take them in a struct, which they read before they return.)
 * Request b of `batch` (1 .. 16384) holds lens[b] tokens and adds new_tokens[b] (0 or
 * more).  Its row table + b * table_stride holds its ceil(lens[b] / page_size) pages; the
 * call appends the pages that the new tokens need, taken in request order from the front
 * of free_pages, and leaves every other entry as it is.  Written besides: kv_lens[b] =
 * lens[b] + new_tokens[b]; starts[0 .. batch], the exclusive prefix sums of new_tokens;
 * slots[starts[b] + i] = page * page_size + offset of request b's i-th new token, and -1
 * for entries from starts[batch] to num_slots; used[0], the number of pages taken.
 * A table entry or slot for which free_pages has no page is -1 (used[0] > num_free then
 * says how many were needed), and so is a slot past max_pages; tokens past num_slots get
 * no slot.  The same call on the same inputs writes the same values.
 * Negative lengths count as 0, lengths past max_pages * page_size as that; the sum of
 * new_tokens must be below 2^31.
 * No output may overlap an input or another output (SDT_ERR_ARG): lengths are updated in
 * place by paged_tables_taken only.
 */
typedef struct sdt_paged_step {
    const int32_t *lens, *new_tokens, *free_pages;
    int32_t *table, *kv_lens, *starts, *used;
    int64_t *slots;
    int64_t batch, page_size, max_pages, table_stride, num_free, num_slots;
} sdt_paged_step;
int paged_tables(const sdt_paged_step *step, sdt_stream_t stream);

/*
 * paged_tables_taken -- paged_tables for a step that is captured once and replayed: the place
 * in the free list is on the device.  taken: int32 [2], zeros before the first call; taken[0]
 * is the number of entries of free_pages that earlier calls have used.  The call takes its
 * pages from there on (num_free counts the whole list) and adds how many it took, at most up
 * to num_free; taken[1] is zero between calls.  kv_lens may be lens itself here.  Calls that
 * share `taken` must not overlap on the GPU.
 */
int paged_tables_taken(const sdt_paged_step *step, int32_t *taken, sdt_stream_t stream);

/*
 * paged_append -- the keys and values of `tokens` tokens into the cache at their slots
 * (slot = page * page_size + offset).  k and v: fp16 or bf16 (dtype; a 16-bit cache's own
 * type), head h of token t at t * k_token + h * k_head elements, head_dim contiguous;
 * bases 16-byte aligned, strides multiples of 8 (of a single token or head: anything).  A
 * negative slot's token is left out; a slot past the cache is left out too and reported by
 * sdt_check_device_status.  Slots that are not negative must differ: tokens with one slot may
 * leave a row mixed from both, in q8 under the scale of either.  k and v must not lie at slots
 * that the call writes.  q8: scale = fp16(max|x| * fl32(1/127)), at most 65504, q = x / scale
 * rounded to the nearest integer (ties to even) within +-127, 0 where the scale is 0 or x is
 * NaN.
 */
int paged_append(int64_t tokens, const void *k, int64_t k_token, int64_t k_head, const void *v, int64_t v_token,
                 int64_t v_head, int dtype, const int64_t *slots, const sdt_paged_cache *cache,
                 sdt_stream_t stream);

/*
 * paged_attn_m1 -- attention of one new token per request:
 *   out[b][i] = sum_n softmax_n(scale * q[b][i] . k[n][h]) v[n][h],  h = i / (q_heads / kv_heads),
 * over the tokens n of request b that its table row names: max(0, lens[b] - window) <= n <
 * lens[b] with window > 0, all lens[b] with window == 0.  q, out: [batch][q_heads][head_dim]
 * fp16 or bf16 (dtype; a 16-bit cache's own type) with strides in elements (q multiples of
 * 8 and 16-byte aligned, out multiples of 4 and 8-byte aligned).  lse, if not NULL, gets
 * log(sum exp(scores)) as fp32 [batch][q_heads].  A request without keys, or whose scores
 * are all -inf, gets zeros and lse -inf.  A NaN or an infinity among a request's values (or
 * q8 value scales) makes the outputs of its column (or group) NaN or infinite, and no others.
 * What lies in the cache outside the named tokens is not read.  A page id outside the cache
 * is not followed and reported by sdt_check_device_status; the request's out and lse are NaN.
 * A length past max_pages * page_size is reported and taken as that.  Results do not depend
 * on the order in which the CTAs run.
 *
 * Workspace: device memory owned by the caller, 256-byte aligned, at least
 * sdt_paged_attn_workspace_bytes() bytes: the 1 MiB counter region of the split-K
 * workspaces (zero before the first call, left zero by every completed call; it may be
 * shared with those), then a list of the requests that are split over CTAs and their
 * pieces.  Calls that share a workspace must not overlap on the GPU.
 */
typedef struct sdt_paged_attn {
    const void *q;
    void *out;
    float *lse;                /* NULL: not wanted */
    const int32_t *table, *lens;
    const sdt_paged_cache *cache;
    void *workspace;
    int64_t batch, q_heads;
    int64_t q_batch, q_head, out_batch, out_head; /* strides in elements */
    int64_t table_stride, max_pages, window, workspace_bytes;
    float scale;
    int dtype;
} sdt_paged_attn;
int paged_attn_m1(const sdt_paged_attn *call, sdt_stream_t stream);
/* Workspace bytes of paged_attn_m1 on the current device, for any batch and lengths (0 on error). */
size_t sdt_paged_attn_workspace_bytes(int64_t q_heads, int64_t kv_heads, int64_t head_dim);

/* ------------------------------------------------------------------------ */
/* A layer in 8 bits: fp8 products, their operands, rotary positions          */
/* ------------------------------------------------------------------------ */

#define SDT_DTYPE_F32 3
#define SDT_DTYPE_E4M3 4
#define SDT_DTYPE_E5M2 5

/*
 * gemm_fp8 -- product of fp8 activations and fp8 weights with a scale per 128 values of k:
 *   C[m][n] = sum_b a_scales[m][b] * w_scales[n / 128][b] * sum_{k in block b} A[m][k] * W[n][k],
 * blocks b of 128 consecutive k (the last one may be shorter).  A: M x K, W: N x K ("K-major",
 * as gemv_m1's), e4m3 or e5m2 each (SDT_DTYPE_E4M3 / _E5M2); scales fp32 of any strides; C:
 * M x N fp16, bf16 or fp32.  Block sums are formed on the tensor cores, multiplied by the product
 * of both scales and added in fp32, and rounded once to C's type.  (That product is an fp32 number
 * of its own: past fp32's range it is infinite, and below 2^-126 it has fewer bits.)  Results depend
 * on the shape and on whether rows of A and W start at multiples of 32 bytes (which decide the tile
 * and how k is shared out) but not on timing.  A NaN among a row's values or scales makes that row
 * (of W: that column, of W's scales their 128 columns) of C NaN; memory outside the operands is not
 * read.  C must not overlap them or the scales (slices of the same rows do not).
 *
 * Any M, K >= 0 (M == 0 or N == 0: no-op; K == 0 writes zeros); N a multiple of 8; dimensions
 * up to 2^30.  A, W and C 16-byte aligned, lda and ldw (elements) multiples of 16 at least K,
 * ldc a multiple of 8 at least N; a stride of a single row may be anything.  Scales 4-byte
 * aligned, strides not negative.
 * tile: 0 picks; 16, 32, 64 or 128 tokens per tile of 128 weight rows, whose blocks `splits`
 * (0 picks, 1 .. 8; no more than blocks) CTAs share; 192 or 256: two-CTA tiles of 256 tokens by
 * that many outputs, which are never split: `splits` counts for nothing there.
 * Errors: SDT_ERR_NULL, SDT_ERR_ALIGN, SDT_ERR_SHAPE (N, dimensions), SDT_ERR_ARG (types,
 * strides, splits), SDT_ERR_TILE.
 */
typedef struct sdt_gemm_fp8 {
    const void *a;
    const float *a_scales;
    const void *w;
    const float *w_scales;
    void *c;
    int64_t M, N, K, lda, ldw, ldc;
    int64_t as_row, as_block, ws_row, ws_block; /* scale strides in elements */
    int a_dtype, w_dtype, c_dtype, tile, splits;
} sdt_gemm_fp8;
int gemm_fp8(const sdt_gemm_fp8 *call, sdt_stream_t stream);
/* The tile and splits that gemm_fp8 takes for a call on a GPU with sm_count SMs (M, N and K at least 1;
 * nothing is followed or enqueued, and no GPU is needed). */
int sdt_gemm_fp8_plan_call(const sdt_gemm_fp8 *call, int sm_count, int *tile, int *splits);
/* The same for sizes alone: rows of K rounded up to 16, from bases at multiples of 32 bytes. */
int sdt_gemm_fp8_plan_for(int64_t M, int64_t N, int64_t K, int sm_count, int *tile, int *splits);

/*
 * quant_fp8 -- gemm_fp8's operand from 16-bit rows: q[t][i] = e4m3(y[t][i] * 448 / top), scale
 * top / 448 (fp32), top = max(max|y|, 2^-100) of the block of 128, with y = x, or act(gate) * x
 * (activation 1: silu, g / (1 + exp(-g)); 2: gelu's tanh form,
 * 0.5 g (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3)))), computed in fp32.  q is the nearest e4m3
 * number and the even one of a tie, at most 448: without a gate exact ties of x are ties here.
 * With one, y is known to some fp32 steps, and a value as near to a border between two e4m3 numbers
 * may fall on its other side.  A NaN
 * stays a NaN of its own; a block that holds an infinity gets an infinite scale and stands for
 * NaN.  Width a multiple of 8 up to 65536; tokens times the width in whole blocks of 128 below 2^34 - 2^12.
 * x and gate: fp16 or bf16 (dtype), 16-byte aligned, row strides multiples of 8 (they may be
 * slices of one row, as a product writes them side by side); q: e4m3, 8-byte aligned, row
 * stride a multiple of 8; scales: fp32 of any strides.  The outputs must not overlap the inputs
 * or each other (SDT_ERR_ARG; slices of the same rows do not).
 */
typedef struct sdt_quant_fp8 {
    const void *x, *gate; /* gate: NULL with activation 0 */
    void *q;
    float *scales;
    int64_t tokens, width, x_row, gate_row, q_row, s_row, s_block; /* strides in elements */
    int dtype, activation;
} sdt_quant_fp8;
int quant_fp8(const sdt_quant_fp8 *call, sdt_stream_t stream);

/*
 * rms_norm_fp8 -- the residual's addition, root-mean-square norm, and fp8 output:
 *   r = x + residual, rounded to their type and written back to residual (without one: r = x);
 *   y[t][i] = r[t][i] * weight[i] / sqrt(mean_j r[t][j]^2 + eps)      (fp32)
 * (squares are summed in fp32: a row with values past 1e18 may overflow, and is zeros or NaN then)
 * and q, scales of y as quant_fp8 makes them with a gate.  out, if not NULL, receives y rounded to
 * x's type.
 * x, residual, out: fp16 or bf16 (dtype), 16-byte aligned, row strides multiples of 8; weight:
 * x's type or fp32 (weight_dtype), 16-byte aligned; width up to 32768; sizes and outputs
 * otherwise as quant_fp8.
 * The outputs must not overlap the inputs or each other (residual is updated in place and must not
 * overlap x; SDT_ERR_ARG).  The order of a row's sum follows from width and tokens, not from timing.
 */
typedef struct sdt_rms_norm_fp8 {
    const void *x, *weight;
    void *residual, *out; /* NULL: none */
    void *q;
    float *scales;
    int64_t tokens, width, x_row, r_row, o_row, q_row, s_row, s_block;
    float eps;
    int dtype, weight_dtype;
} sdt_rms_norm_fp8;
int rms_norm_fp8(const sdt_rms_norm_fp8 *call, sdt_stream_t stream);

/*
 * rope_qk -- rotary positions of queries and keys.  Pair i of a head is (x, y) = elements
 * (i, rotary / 2 + i), or (2 i, 2 i + 1) with interleaved; with t = positions[token] *
 * turns[i] / 2^64 turns (modulo 1, exactly, negative positions too),
 *   x' = magnitude * (x cos t - y sin t),  y' = magnitude * (y cos t + x sin t)
 * in fp32, rounded once; inverse turns the other way (with it the call takes gradients of the
 * outputs to gradients of the inputs).  Elements from rotary on are copied.
 * q, k, q_out, k_out: [tokens][heads][head_dim] fp16 or bf16 (dtype), head_dim contiguous, any
 * other strides in elements up to 2^32 (16-byte aligned heads are fastest); heads may be 0 (no
 * such side).
 * An output is its input itself or lies apart from both inputs, the other output, positions and turns
 * (SDT_ERR_ARG; slices of the same rows lie apart).  positions: int32 or int64
 * (position_bytes 4 or 8); turns: uint64 [rotary / 2].  head_dim even, rotary even, at most
 * head_dim; tokens * heads * head_dim below 2^31.
 */
typedef struct sdt_rope_qk {
    const void *q, *k;
    void *q_out, *k_out;
    const void *positions;
    const uint64_t *turns;
    int64_t tokens, q_heads, k_heads, head_dim, rotary;
    int64_t q_token, q_head, k_token, k_head, qo_token, qo_head, ko_token, ko_head;
    float magnitude;
    int dtype, position_bytes, interleaved, inverse;
} sdt_rope_qk;
int rope_qk(const sdt_rope_qk *call, sdt_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Diagnostics                                                               */
/* ------------------------------------------------------------------------ */

/* Message of the last failed call on this thread ("" if none).  Valid until the next call. */
const char *sdt_last_error(void);

/*
 * Every mbarrier wait in the kernels is bounded (by default 2 s).  A kernel
 * that gives up records a code in a device status word and returns without
 * trapping.  This call synchronises `stream`, reads and clears the word for
 * the current device, and returns SDT_OK or SDT_ERR_TIMEOUT (SDT_ERR_CUDA if
 * the stream itself reports an error).  `where` (may be NULL) receives the
 * recorded code: its low 4 bits are the site (1 producer, 2 MMA issuer,
 * 3 epilogue, 4 drain, 5 probe); 8, 9 and 10 stand for a page id, slot or length outside
 * the cache or table that a paged operator met and left out (SDT_ERR_ARG is returned
 * then); the two-CTA kernels add the CTA's rank in the
 * pair at bit 4 and the loop position from bit 8.
 */
int sdt_check_device_status(sdt_stream_t stream, int *where);

/*
 * Test hook for the bounded waits: launches one CTA of the GEMM kernel's
 * wait routine on an mbarrier nothing ever arrives at, with the given limit
 * in microseconds (1 .. 10,000,000).  The kernel gives up, records code 5 and
 * returns; read it with sdt_check_device_status.
 */
int sdt_debug_timeout_probe(sdt_stream_t stream, int64_t limit_us);

/*
 * Number of TMA tensor maps encoded so far by this process (misses of the
 * tensor-map cache, whose key holds the base pointer, both extents, the row
 * stride and the box).  For tests of the cache key.
 */
int64_t sdt_debug_tensor_map_encodes(void);

/* SM count and opt-in shared memory per block of the current device. */
int sdt_device_sm_count(void);
int sdt_device_smem_optin(void);

/* ABI version of this header (bumped on incompatible changes). */
#define SDT_ABI_VERSION 1
int sdt_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SDT_H */
