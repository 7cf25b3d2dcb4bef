/*
 * dp_gemm.h -- C ABI of the GB300 (sm_103a) dense projection GEMM library.
 *
 * The library computes the projection GEMMs of one training step of a linear
 * layer Y = X W^T, as described on the FlashInfer pull-request pages about the
 * "Cake" dense projection GEMM packages:
 *
 *   forward          Y[T,N]  = X[T,K] . W[N,K]^T           (K-major B)
 *   input gradient   dX[T,K] = dY[T,N] . W[N,K]            (MN-major B)
 *   weight gradient  dW[N,K] = dY[T,N]^T . X[T,K]          (contraction over the
 *                                                           T tokens, 64-token blocks)
 *   router           the same three contractions on FP32 operands (hidden H -> 256
 *                    experts) computed through BF16x3 emulation.
 *
 * Page references used below:
 *   [det-dgrad]  "perf(cake_dense_projection_det_gemm): plan the 4096 -> 12288
 *                input gradient with the row-half-release program at T-exact keys",
 *                PR body: forward (K-major B) and input-gradient (MN-major B) forms;
 *                whole K per output tile keeps outputs bitwise identical.
 *   [k1-wgrad]   "perf(cake_dense_projection_gemm): restore the K1 weight-gradient
 *                routes that meet the deterministic package's absolute FP64 budgets",
 *                PR body: K1 has BF16 or FP32 output; wgrad contracts over 64-token
 *                K blocks with one or two K splits; the FP64 error budgets.
 *   [router]     "perf(cake_dense_projection_gemm): cache the router entry points'
 *                calls by their own tensors", summary: FP32 router [T,H] x [256,H]^T,
 *                BF16x3 emulation, router_forward / router_dgrad / router_wgrad,
 *                deterministic=True is the default.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Memory.  All matrix pointers are DEVICE pointers on the current CUDA device,
 *   row-major, 16-byte aligned.  BF16 operands are passed as raw 16-bit patterns
 *   (`const void*`).  Leading dimensions (`ld*`, in elements) give the distance
 *   between consecutive rows; 0 means "contiguous" (the row length).  Every
 *   leading dimension times the element size must be a multiple of 16 bytes, and
 *   the row lengths N and K must be multiples of 8 (16-byte rows).  An output
 *   with a padded leading dimension is written only in its first N (or K) columns.
 * Ownership.  The caller owns every buffer, the workspace and the stream.  The
 *   library never allocates device memory, never synchronises and never frees.
 * Workspace.  `workspace` is caller-provided device memory of at least
 *   dp_workspace_size(...) bytes (may be NULL when that size is 0).  It is
 *   scratch: FP32 partial tiles of split contractions and the router's bf16
 *   hi/lo operand copies, written before they are read within the call, so it
 *   needs no initial value.  One workspace must not be used by two calls that may
 *   run concurrently.
 * Launches.  Each call enqueues one GEMM kernel; a plan that splits contractions
 *   adds the kernel that sums the partials, and a router call adds the kernel
 *   that splits its reused FP32 operand into bf16 hi/lo before the GEMM (a router
 *   call on the small-T SIMT program is that one kernel alone; a non-deterministic
 *   plan adds a memset of its FP32 output instead of the reduction).  The GEMM
 *   and the reduction launch as programmatic dependents of the kernel before them
 *   on the stream: their setup overlaps that kernel's tail, and they wait for its
 *   completion before touching global memory, so stream order between calls (one
 *   call reading what the previous one wrote, or overwriting what it read) holds
 *   as for ordinary launches.
 * Stream.  `stream` is a cudaStream_t (NULL = legacy default stream).  All work
 *   is enqueued on it; calls return before the GPU finishes.  Calls are legal
 *   inside CUDA stream capture after the first call on the device (which sets
 *   kernel attributes; dp_init() does it explicitly).
 * Determinism.  With deterministic != 0 (the default of the pages' entry points)
 *   every output is bitwise reproducible for the same inputs, shapes, strides and
 *   SM count: each output tile's contraction is split into a fixed partition
 *   chosen by a pure planner, and split partials are summed in split order.
 *   deterministic = 0 (the pages' non-deterministic package) admits, for FP32
 *   outputs of single-problem calls, plans whose split units add their FP32
 *   partials into the output with atomic adds after a zero fill of the output
 *   (a memset node, or a job of the router's split kernel): no partial workspace
 *   and no reduction kernel, at the cost of run-to-run variation in the last bits
 *   (the adds' order).  The planner takes it only where its model finds it
 *   faster; BF16 outputs, batched calls and plans without split tiles stay
 *   deterministic either way.
 * Errors.  Arguments are checked before anything is enqueued; a non-DP_OK status
 *   means nothing was launched (except DP_ERR_LAUNCH, reported by CUDA after the
 *   attempt).  No exception crosses the ABI.
 * Empty input.  T == 0 is legal: forward and input gradient enqueue nothing; the
 *   weight gradient writes zeros (the sum over an empty token set).
 */
#ifndef DP_GEMM_H
#define DP_GEMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum dp_status {
    DP_OK = 0,
    DP_ERR_INVALID_ARG = 1,   /* null pointer, negative size, ld smaller than the row */
    DP_ERR_ALIGNMENT = 2,     /* pointer or row stride not 16-byte aligned */
    DP_ERR_UNSUPPORTED = 3,   /* N or K not a multiple of 8, or a size beyond 2^31-1 */
    DP_ERR_WORKSPACE = 4,     /* workspace NULL or smaller than dp_workspace_size() */
    DP_ERR_ARCH = 5,          /* current device is not compute capability 10.3 (sm_103a) */
    DP_ERR_LAUNCH = 6,        /* a CUDA call failed while enqueueing */
    DP_ERR_TIMEOUT = 7        /* a kernel gave up waiting on one of its barriers (debug read-out) */
} dp_status;

typedef enum dp_out_dtype {
    DP_OUT_BF16 = 0,          /* FP32 accumulator rounded once to bf16, nearest-even */
    DP_OUT_F32 = 1            /* FP32 accumulator stored as is */
} dp_out_dtype;

typedef enum dp_op {
    DP_OP_FWD = 0,
    DP_OP_DGRAD = 1,
    DP_OP_WGRAD = 2,
    DP_OP_ROUTER_FWD = 3,
    DP_OP_ROUTER_DGRAD = 4,
    DP_OP_ROUTER_WGRAD = 5
} dp_op;

/* A cudaStream_t, passed as a plain pointer. */
typedef void* dp_stream;

/* ------------------------------------------------------------------ BF16 ops */

/* Forward, [det-dgrad] "forward (K-major B) form":
 *   Y[t][n] = sum_k X[t][k] * W[n][k]
 * X: T x K bf16 (ldx), W: N x K bf16 (ldw), Y: T x N (ldy) in `out` precision.
 * FP32 accumulation; rows t >= T are never written. */
dp_status dp_gemm_fwd(const void* X, const void* W, void* Y,
                      int64_t T, int64_t N, int64_t K, dp_out_dtype out, int deterministic,
                      void* workspace, size_t workspace_bytes, dp_stream stream);
dp_status dp_gemm_fwd_ex(const void* X, int64_t ldx, const void* W, int64_t ldw,
                         void* Y, int64_t ldy,
                         int64_t T, int64_t N, int64_t K, dp_out_dtype out, int deterministic,
                         void* workspace, size_t workspace_bytes, dp_stream stream);

/* Input gradient, [det-dgrad] "input-gradient (MN-major B) form":
 *   dX[t][k] = sum_n dY[t][n] * W[n][k]
 * dY: T x N bf16 (ldg), W: N x K bf16 (ldw; read with the contraction N as its
 * outer, MN-major dimension), dX: T x K (ldx) in `out` precision. */
dp_status dp_gemm_dgrad(const void* dY, const void* W, void* dX,
                        int64_t T, int64_t N, int64_t K, dp_out_dtype out, int deterministic,
                        void* workspace, size_t workspace_bytes, dp_stream stream);
dp_status dp_gemm_dgrad_ex(const void* dY, int64_t ldg, const void* W, int64_t ldw,
                           void* dX, int64_t ldx,
                           int64_t T, int64_t N, int64_t K, dp_out_dtype out, int deterministic,
                           void* workspace, size_t workspace_bytes, dp_stream stream);

/* Weight gradient, [k1-wgrad] (contraction over the tokens in 64-token K blocks):
 *   dW[n][k] = sum_t dY[t][n] * X[t][k]
 * dY: T x N bf16 (ldg), X: T x K bf16 (ldx), dW: N x K (ldw) in `out` precision.
 * The token blocks of one output tile are summed by one CTA in order, or, for
 * thin outputs, split into S contiguous block ranges whose FP32 partials are
 * added in ascending split order before the single output rounding. */
dp_status dp_gemm_wgrad(const void* dY, const void* X, void* dW,
                        int64_t T, int64_t N, int64_t K, dp_out_dtype out, int deterministic,
                        void* workspace, size_t workspace_bytes, dp_stream stream);
dp_status dp_gemm_wgrad_ex(const void* dY, int64_t ldg, const void* X, int64_t ldx,
                           void* dW, int64_t ldw,
                           int64_t T, int64_t N, int64_t K, dp_out_dtype out, int deterministic,
                           void* workspace, size_t workspace_bytes, dp_stream stream);

/* Weight gradient for callers that cannot allocate device memory.  The pages have
 * no counterpart of this entry point; it exists for this library's users.
 * Some callers cannot pass a workspace: a serving runtime that reserves all device
 * memory at start-up, or a plugin whose host forbids cudaMalloc on its hot path
 * because it can synchronise the device.  This call computes exactly what
 * dp_gemm_wgrad_ex computes (same plan, same kernels, same bits) but keeps its
 * split partials in a 64 MiB scratch array built into the library,
 * which every GPU that loads the library holds until the process exits.  The
 * caller still passes dY, X and dW.  Arguments and errors as dp_gemm_wgrad_ex;
 * a shape whose plan needs more than 64 MiB of scratch returns DP_ERR_WORKSPACE
 * (dp_workspace_size(DP_OP_WGRAD, ...) tells beforehand).  The first call on each
 * device looks up the array's device address (with that device current).  Every
 * call shares the one array; calls that overlap on the GPU
 * (different streams or threads) race on it and must be serialised by the caller.  No cudaMalloc,
 * cudaFree or allocating library routine is called. */
dp_status dp_gemm_wgrad_noalloc(const void* dY, int64_t ldg, const void* X, int64_t ldx,
                                void* dW, int64_t ldw,
                                int64_t T, int64_t N, int64_t K, dp_out_dtype out, int deterministic,
                                dp_stream stream);

/* ------------------------------------------------------------ batched BF16 ops */
/* Batched projection GEMMs: B independent problems of one shape in one launch,
 * as the pages' integration runs its per-head projections ("one batched BF16 GEMM
 * over strided views, forward and both gradients", with a weight layout option).
 * Problem b reads X_b = X + b*bsx (and so on for every operand and output, in
 * elements; a batch stride of 0 means packed, rows * ld).  Batch strides may be
 * smaller than a row (per-head slices of a [T][H][D] tensor: ld = H*D, bs = D);
 * they must keep 16-byte alignment.  weight_kn = 0: W_b and dW_b are [N][K]
 * matrices as in the single-problem calls; 1: they are [K][N].  One plan covers
 * the B * tiles_m * tiles_n tiles in one persistent launch (its tile shape and
 * splits are chosen for the whole batch, so they can differ from a single
 * problem's); every problem's tiles use the same fixed contraction partition and
 * summation order, so the outputs are deterministic (whatever `deterministic`). */
dp_status dp_gemm_fwd_batched(const void* X, int64_t ldx, int64_t bsx, const void* W, int64_t ldw, int64_t bsw,
                              int weight_kn, void* Y, int64_t ldy, int64_t bsy,
                              int64_t B, int64_t T, int64_t N, int64_t K, dp_out_dtype out, int deterministic,
                              void* workspace, size_t workspace_bytes, dp_stream stream);
dp_status dp_gemm_dgrad_batched(const void* dY, int64_t ldg, int64_t bsg, const void* W, int64_t ldw, int64_t bsw,
                                int weight_kn, void* dX, int64_t ldx, int64_t bsx,
                                int64_t B, int64_t T, int64_t N, int64_t K, dp_out_dtype out, int deterministic,
                                void* workspace, size_t workspace_bytes, dp_stream stream);
dp_status dp_gemm_wgrad_batched(const void* dY, int64_t ldg, int64_t bsg, const void* X, int64_t ldx, int64_t bsx,
                                void* dW, int64_t ldw, int64_t bsw, int weight_kn,
                                int64_t B, int64_t T, int64_t N, int64_t K, dp_out_dtype out, int deterministic,
                                void* workspace, size_t workspace_bytes, dp_stream stream);

/* -------------------------------------------------------- backward pass (BF16) */
/* Input gradient and weight gradient of one layer from the same dY (the pages'
 * "bwd" op is dgrad + wgrad, [router] benchmark rows):
 *   dX[t][k] = sum_n dY[t][n] * W[n][k]      (as dp_gemm_dgrad_ex)
 *   dW[n][k] = sum_t dY[t][n] * X[t][k]      (as dp_gemm_wgrad_ex)
 * with their own output precisions and leading dimensions.  The planner picks one
 * of two forms (dp_plan_query_bwd reports which):
 *   - the two single-op calls, one after the other on `stream`, sharing the
 *     workspace (bitwise the same as calling dp_gemm_dgrad_ex, dp_gemm_wgrad_ex);
 *   - one co-scheduled launch: both problems tiled alike (one tile shape) with
 *     whole K per tile, their tiles in one list dealt to one persistent grid, so
 *     the SMs left idle by one problem's last wave run the other's tiles.  Needs
 *     no workspace.  Every output element is the same whole-K sum a whole-K
 *     single-op plan computes.
 * Chosen when the cost model expects the co-scheduled launch to be at least 3%
 * faster (small and mid-size T, where each single-op launch leaves SMs idle);
 * DP_FORCE_FUSE (with DP_TUNING, see below) overrides (0: two calls; 1:
 * co-scheduled; 2 / 3: co-scheduled with the weight / input gradient's tiles
 * first).  dX and dW must not overlap
 * dY, X or W.
 * Arguments and errors as the single-op calls; workspace: dp_workspace_size_bwd. */
dp_status dp_gemm_bwd(const void* dY, int64_t ldg, const void* X, int64_t ldx, const void* W, int64_t ldw,
                      void* dX, int64_t ld_dx, dp_out_dtype out_dx, void* dW, int64_t ld_dw, dp_out_dtype out_dw,
                      int64_t T, int64_t N, int64_t K, int deterministic,
                      void* workspace, size_t workspace_bytes, dp_stream stream);

/* ----------------------------------------------------------------- router ops */
/* [router]: FP32 operands and FP32 output; N is the expert count (256 on the
 * pages) and K the hidden size.  Each FP32 operand value x is split into bf16
 * hi = RNE(x) and lo = RNE(x - hi); every product a*b is formed as
 * hi_a*hi_b + hi_a*lo_b + lo_a*hi_b on the BF16 tensor cores with FP32
 * accumulation (lo_a*lo_b is dropped).  The operand the whole output reuses (W,
 * or dY for the weight gradient; both for the input gradient) is split once per
 * call into bf16 copies in the workspace; the streamed FP32 operand is split
 * inside the GEMM.  The weight gradient is computed as dW^T = X^T dY and stored
 * transposed.
 * Small T (a few hundred tokens or fewer, as the planner's cost model decides;
 * dp_plan_info.program reports it): a SIMT FP32 program instead -- the plain
 * FP32 contraction with FP32 fused multiply-adds on the CUDA cores, in one launch
 * and without workspace, each output tile's contraction split over the CTAs of a
 * thread-block cluster whose partials are summed in a fixed order (so the output
 * is bitwise repeatable; its error is the FP32 rounding of the sum, below the
 * BF16x3 program's).  DP_FORCE_FFMA=0 / 1 (with DP_TUNING, see below) forces
 * either program (1: where the forced tile width and split count, if any, fit the
 * shape). */

/* Router forward: Y[t][n] = sum_k X[t][k] * W[n][k];  X: T x K, W: N x K, Y: T x N. */
dp_status router_fwd(const float* X, const float* W, float* Y,
                     int64_t T, int64_t N, int64_t K, int deterministic,
                     void* workspace, size_t workspace_bytes, dp_stream stream);
dp_status router_fwd_ex(const float* X, int64_t ldx, const float* W, int64_t ldw,
                        float* Y, int64_t ldy, int64_t T, int64_t N, int64_t K, int deterministic,
                        void* workspace, size_t workspace_bytes, dp_stream stream);

/* Router input gradient: dX[t][k] = sum_n dY[t][n] * W[n][k];  dY: T x N, dX: T x K. */
dp_status router_dgrad(const float* dY, const float* W, float* dX,
                       int64_t T, int64_t N, int64_t K, int deterministic,
                       void* workspace, size_t workspace_bytes, dp_stream stream);
dp_status router_dgrad_ex(const float* dY, int64_t ldg, const float* W, int64_t ldw,
                          float* dX, int64_t ldx, int64_t T, int64_t N, int64_t K, int deterministic,
                          void* workspace, size_t workspace_bytes, dp_stream stream);

/* Router weight gradient: dW[n][k] = sum_t dY[t][n] * X[t][k];  dW: N x K. */
dp_status router_wgrad(const float* dY, const float* X, float* dW,
                       int64_t T, int64_t N, int64_t K, int deterministic,
                       void* workspace, size_t workspace_bytes, dp_stream stream);
dp_status router_wgrad_ex(const float* dY, int64_t ldg, const float* X, int64_t ldx,
                          float* dW, int64_t ldw, int64_t T, int64_t N, int64_t K, int deterministic,
                          void* workspace, size_t workspace_bytes, dp_stream stream);

/* ------------------------------------------- products grouped by expert (BF16) */
/* The projections of a layer of experts: the T rows of X (or dY) are sorted by expert,
 * expert e owns the rows [offsets[e], offsets[e + 1]), and each row meets its expert's
 * weights:
 *   forward          Y[t]  = X[t] W_e^T          W_e: N x K
 *   input gradient   dX[t] = dY[t] W_e
 *   weight gradient  dW_e  = sum over the expert's rows of dY[t]^T X[t]
 * No counterpart on the pages; operands, outputs and errors as the calls above.
 * offsets: E + 1 values in DEVICE memory, int32 or int64 (offset_bits), never read by the
 *   host: the call needs no synchronisation and can be captured before the router's choice
 *   is known.  They should not decrease and lie in [0, T].  Values that do not are clamped
 *   (to [0, T] and to the running maximum) and reported as DP_ERR_INVALID_ARG by
 *   dp_device_error().
 * Rows before offsets[0] and from offsets[E] on (padding of a buffer with room to spare)
 *   belong to no expert: their output rows are zero and no weight gradient sees them.
 *   Infinities and NaN there, or in another expert's rows, reach no other output.
 * Experts without rows: dW_e = 0.
 * weight_kn: W_e and dW_e are [N][K] (0) or [K][N] (1) matrices, ldw apart by rows and bsw
 *   apart by experts (elements; 0 = packed).
 * FP32 accumulation in pieces of 512 contraction elements that are added in FP32 with
 * round-to-nearest, whatever the group's size; every output is deterministic.  One launch,
 * no workspace.  At most 1024 experts.
 * One SM (or a pair) contracts an output tile's whole length: a few experts with a few tiles
 * leave SMs idle however long the contraction (one expert of 256 x 256, weight gradient: 8
 * tiles); dp_gemm_wgrad shares a contraction among SMs. */
dp_status dp_gemm_fwd_grouped(const void* X, int64_t ldx, const void* W, int64_t ldw, int64_t bsw, int weight_kn,
                              const void* offsets, int offset_bits, void* Y, int64_t ldy,
                              int64_t E, int64_t T, int64_t N, int64_t K, dp_out_dtype out, dp_stream stream);
dp_status dp_gemm_dgrad_grouped(const void* dY, int64_t ldg, const void* W, int64_t ldw, int64_t bsw, int weight_kn,
                                const void* offsets, int offset_bits, void* dX, int64_t ldx,
                                int64_t E, int64_t T, int64_t N, int64_t K, dp_out_dtype out, dp_stream stream);
dp_status dp_gemm_wgrad_grouped(const void* dY, int64_t ldg, const void* X, int64_t ldx,
                                const void* offsets, int offset_bits, void* dW, int64_t ldw, int64_t bsw,
                                int weight_kn, int64_t E, int64_t T, int64_t N, int64_t K, dp_out_dtype out,
                                dp_stream stream);

/* ------------------------------- 8-bit floating point, a scale per 128 elements */
typedef enum dp_fp8_format {
    DP_FP8_E4M3 = 0,          /* largest value 448 */
    DP_FP8_E5M2 = 1           /* largest value 57344 */
} dp_fp8_format;

typedef enum dp_fp8_scaling {
    DP_FP8_ROW = 0,           /* blocks of 128 elements of a row */
    DP_FP8_COL = 1,           /* blocks of 128 elements of a column */
    DP_FP8_BLOCK = 2,         /* blocks of 128 x 128 */
    DP_FP8_BOTH = 3           /* row blocks into q, s and column blocks into q_col, s_colwise */
} dp_fp8_scaling;

/* Quantise x [rows][cols] (BF16, or FP32 with x_f32):
 *   a = max(max |x| over the block, 1e-30), s = a / top, q = rn(x * (top / a))
 * with top the format's largest value; the last blocks may be partial.  A block that holds a
 * NaN gets a NaN scale, one that holds an infinity an infinite scale.
 *   q, s          row or 128 x 128 blocks: the scale of row (or row block) r and column block
 *                 c goes to s[r * s_row + c * s_col]
 *   q_col, s_colwise  column blocks: row block r, column c at s_colwise[r * sc_row + c]
 *                 (16-byte aligned rows)
 * The unused pair may be null.  cols a multiple of 16. */
dp_status dp_fp8_quantize(const void* x, int64_t ldx, int x_f32, int64_t rows, int64_t cols, dp_fp8_scaling scaling,
                          dp_fp8_format format, void* q, int64_t ldq, float* s, int64_t s_row, int64_t s_col,
                          void* q_col, int64_t ldq_col, float* s_colwise, int64_t sc_row, dp_stream stream);

/* Products of quantised operands, x = q * s.  The 128-element blocks run along the
 * contraction; each block's sum is scaled and added in FP32:
 *   forward          Y  = X W^T   X: row blocks, W: 128 x 128 blocks
 *   input gradient   dX = dY W    dY: row blocks (along N), W as in the forward pass (the
 *                                 same bytes: no transposed copy)
 *   weight gradient  dW = dY^T X  dY and X: column blocks (along T)
 * Scales lie at any non-negative strides: row blocks at s[t * row + block * blk], 128 x 128
 * blocks at s[row block * row + column block * col], column blocks at
 * s[block * blk + column * col].  A block's two scales meet in FP32: the products of row and
 * 128 x 128 scales are rounded to FP32 before they multiply the block's sum, column scales
 * multiply it one after the other.  Scales from 2^-60 to 2^60 lose nothing by that which an FP32
 * output could hold; two scales whose product leaves FP32's range give zeros, infinities
 * or NaN even where the sum times both would not.  N, K and leading dimensions multiples of 16.  T == 0 as
 * for the BF16 calls.  Deterministic; one launch, no workspace. */
dp_status dp_gemm_fwd_fp8(const void* Xq, int64_t ldx, dp_fp8_format x_format, const float* Xs, int64_t xs_row,
                          int64_t xs_blk, const void* Wq, int64_t ldw, dp_fp8_format w_format, const float* Ws,
                          int64_t ws_row, int64_t ws_col, void* Y, int64_t ldy,
                          int64_t T, int64_t N, int64_t K, dp_out_dtype out, dp_stream stream);
dp_status dp_gemm_dgrad_fp8(const void* dYq, int64_t ldg, dp_fp8_format dy_format, const float* dYs, int64_t gs_row,
                            int64_t gs_blk, const void* Wq, int64_t ldw, dp_fp8_format w_format, const float* Ws,
                            int64_t ws_row, int64_t ws_col, void* dX, int64_t ldx,
                            int64_t T, int64_t N, int64_t K, dp_out_dtype out, dp_stream stream);
dp_status dp_gemm_wgrad_fp8(const void* dYq, int64_t ldg, dp_fp8_format dy_format, const float* dYs, int64_t gs_blk,
                            int64_t gs_col, const void* Xq, int64_t ldx, dp_fp8_format x_format, const float* Xs,
                            int64_t xs_blk, int64_t xs_col, void* dW, int64_t ldw,
                            int64_t T, int64_t N, int64_t K, dp_out_dtype out, dp_stream stream);

/* ------------------------------------------------------- AdamW over many tensors */
typedef struct dp_adamw_tensor {
    void* param;              /* FP32, or BF16 with param_bf16; updated in place */
    const void* grad;         /* FP32, or BF16 with grad_bf16; null: the tensor is skipped */
    void* exp_avg;            /* FP32, or E4M3 codes (state_bits = 8); updated in place */
    void* exp_avg_sq;         /* FP32, or E4M3 codes of the square root */
    float* exp_avg_scale;     /* state_bits = 8: one scale per 128 elements */
    float* exp_avg_sq_scale;
    void* copy;               /* BF16 copy of the updated parameter, or null */
    int64_t numel;
    int32_t param_bf16;
    int32_t grad_bf16;
} dp_adamw_tensor;

typedef struct dp_adamw_hyper {
    double lr, beta1, beta2, eps, weight_decay;
    double grad_scale;            /* gradients are multiplied by this */
    const float* grad_scale_ptr;  /* and, if not null, by this DEVICE value */
    int64_t step;                 /* 1 for the first update (bias corrections) of these tensors */
} dp_adamw_hyper;

/* One AdamW update of `count` dense tensors (the table is read on the host during the call):
 *   g' = g * scale;  m = beta1 m + (1 - beta1) g';  v = beta2 v + (1 - beta2) g'^2
 *   p  = p (1 - lr wd) - lr / (1 - beta1^step) * m / (sqrt(v) / sqrt(1 - beta2^step) + eps)
 * in FP32: the moments' operations rounded one by one, the parameter's update to 6e-7 of
 * itself; p is rounded once to its type.
 * state_bits = 8: m is held as E4M3 codes with a scale max|m| / 448 for each 128 consecutive
 * elements, and sqrt(v) likewise; a v above zero is never held as zero.  Codes are rounded to
 * nearest up to beta1 = 0.98 (m) and beta2 = 0.95 (sqrt(v)); above, where a step moves the moment by
 * less than a nearest code would show, stochastically, by a hash of the element's index in its
 * tensor and `step`: the same call gives the same bits.  sqrt(v) then follows its 32-bit value
 * with a standard deviation of 12 to 20%.  A non-finite gradient makes its element (32 bits)
 * or its 128 elements' state (8 bits) non-finite.
 * 16-byte aligned tensors are faster; any element alignment works.  One launch per 256
 * tensors, no workspace.  Rate, step and the table are arguments of the launch: a captured
 * call repeats that one step, so a graph's replays do not continue it. */
dp_status dp_adamw_step(const dp_adamw_tensor* tensors, int64_t count, int state_bits, const dp_adamw_hyper* hyper,
                        dp_stream stream);

/* ------------------------------------------------------------------- layer norm */
/* Over each row of x [T][C] (BF16, or FP32 with x_f32):
 *   mu = mean(x), rs = 1 / sqrt(mean((x - mu)^2) + eps), h = (x - mu) rs, y = h weight + bias
 * weight, bias: [C], both FP32 (weight_f32) or both BF16; null: 1 and 0.  mean and rstd [T] receive mu
 * and rs, which the backward pass reads.  FP32 arithmetic, y rounded once.
 * Backward, with g = dy weight (dy BF16, or FP32 with dy_f32):
 *   dx = rs (g - mean(g) - h mean(g h)),  dw = sum_t dy h,  db = sum_t dy   (dw, db FP32 [C])
 * dw and db may both be null (then no workspace is needed either); T == 0 makes them zero.  Their
 * sums are deterministic.  C a multiple of 8, at most 16384.  An infinity or a NaN in a row of x
 * reaches that row's outputs, and dw and db, only.  Outputs must not overlap inputs. */
dp_status dp_layer_norm_fwd(const void* x, int64_t ldx, int x_f32, const void* weight, const void* bias, int weight_f32,
                            double eps, void* y, int64_t ldy, dp_out_dtype out, float* mean, float* rstd,
                            int64_t T, int64_t C, dp_stream stream);
dp_status dp_layer_norm_bwd(const void* dy, int64_t ldg, int dy_f32, const void* x, int64_t ldx, int x_f32,
                            const float* mean, const float* rstd, const void* weight, int weight_f32, void* dx,
                            int64_t ld_dx, dp_out_dtype out, float* dw, float* db, int64_t T, int64_t C,
                            void* workspace, size_t workspace_bytes, dp_stream stream);
/* Workspace of the backward pass, for one call at a time (sm_count <= 0: the current device's). */
dp_status dp_layer_norm_workspace_size(int64_t T, int64_t C, int sm_count, size_t* bytes);

/* ---------------------------------------------------- the router's choice of experts */
/* The k largest of each token's E logits (FP32, router_fwd's output), by value and then by the
 * lowest index, and their gates (both [T][k]):
 *   gate_j = exp(l_j - m) / sum exp(l - m)   over the k chosen (renormalize) or over all E
 * A logit of -infinity is a closed expert: it is never chosen, and where fewer than k are open the
 * rest of the row has choice -1 and gate 0.  A NaN counts as the largest value; a row with NaN or
 * +infinity has NaN gates.  E at most 1024, k at most 32 (and E).
 * Gradient of the logits [T][E] from that of the gates, with s = sum_j dgate_j gate_j:
 *   over the chosen: gate_e (dgate_e - s), 0 elsewhere; over all: p_e ([e chosen] dgate_e - s)
 * Choices outside [0, E) take no part, whatever their dgates.  logits are read only without
 * renormalize and may be null with it. */
dp_status dp_route_topk(const float* logits, int64_t ld, float* gates, int32_t* choice, int64_t T, int64_t E, int64_t k,
                        int renormalize, dp_stream stream);
dp_status dp_route_topk_bwd(const float* dgates, const float* logits, int64_t ld, const float* gates, const int32_t* choice,
                            float* dlogits, int64_t ld_d, int64_t T, int64_t E, int64_t k, int renormalize, dp_stream stream);

/* ------------------------------------------------ tokens to their experts and back */
/* Pair p = t k + j is token t's j-th choice.  The sorted buffer has T k rows.
 * Sort: offsets [E + 1] as the grouped products read them, row_of [pairs] the row of each pair,
 *   order [pairs] the pair of each row; pairs of one expert keep their order.  Pairs whose choice
 *   is outside [0, E) have no expert: they follow the last group (which the products leave out),
 *   and their row r is held as ~r, below zero.  choice: int32 or int64 (choice_bits).  At most 1024
 *   experts.
 * Gather: rows[row_of[t][j]] = x[t], zeros for pairs without an expert.
 * Combine: out[t] = add[t] + sum_j gate[t][j] y[row_of[t][j]] over the pairs that have an expert, in
 *   FP32 in the order of j, rounded once.  gates [T][k] FP32 or null (1: the gradient of gather); add of
 *   out's type, or null.
 * Its gradient: dy[row_of[t][j]] = gate[t][j] dout[t] (zeros without an expert), dgates[t][j] =
 *   dout[t] . y[row_of[t][j]] (0 without).
 * An entry of row_of that names no row of the buffer is left out and reported as
 * DP_ERR_INVALID_ARG by dp_device_error(); two pairs must not name one row.  C a multiple of 8, at most 2^31 - 2048.
 * Outputs must not overlap inputs.  Deterministic. */
dp_status dp_expert_sort(const void* choice, int choice_bits, int64_t pairs, int64_t E, int32_t* offsets, int32_t* row_of,
                         int32_t* order, void* workspace, size_t workspace_bytes, dp_stream stream);
dp_status dp_expert_sort_workspace_size(int64_t pairs, int64_t E, size_t* bytes);
dp_status dp_expert_gather(const void* x, int64_t ldx, int x_f32, const int32_t* row_of, void* rows, int64_t ld_rows,
                           int64_t T, int64_t k, int64_t C, dp_stream stream);
dp_status dp_expert_combine(const void* y, int64_t ldy, int y_f32, const int32_t* row_of, const float* gates,
                            const void* add, int64_t ld_add, void* out, int64_t ldo, dp_out_dtype out_dtype,
                            int64_t T, int64_t k, int64_t C, dp_stream stream);
dp_status dp_expert_combine_bwd(const void* dout, int64_t ldd, int dout_f32, const void* y, int64_t ldy, int y_f32,
                                const int32_t* row_of, const float* gates, void* dy, int64_t ld_dy, dp_out_dtype dy_dtype,
                                float* dgates, int64_t T, int64_t k, int64_t C, dp_stream stream);

/* -------------------------------------------- 4-bit weights, a scale per group of a row */
/* w[n][k] = (q - z) s for groups of 32, 64 or 128 elements along k (K a multiple of the group):
 *   q  [rows][K / 2] bytes, two codes 0..15 each, the even k in the low half
 *   s  [rows][K / group], FP32 (s_f32) or BF16
 *   z  [rows][K / group] bytes (their low four bits), or null: 8
 * all packed; experts follow one another as rows.
 * Quantise (BF16, or FP32 with w_f32): without z, s = max(max|w| / 7, 1e-30); with z, over the range
 *   [lo, hi] of the group and 0, s = max((hi - lo) / 15, 1e-30) and z = rn(-lo / s); s is rounded to its type
 *   first, then q = min(max(rn(w / s) + z, 0), 15).  A group that holds a NaN gets a NaN scale.
 * Dequantise: w = (q - z) s, rounded once.
 * Products of few rows (decoding), X [T][K] BF16: Y[t][n] = sum_k X[t][k] w[n][k], the whole or by
 *   expert with offsets as in dp_gemm_fwd_grouped (rows outside all groups are zero).  Each group's
 *   sum meets its scale in FP32.  Right for any T and fast while the weights' bytes bound it (a few
 *   dozen rows, or as many per expert); more rows want dp_int4_dequantize and dp_gemm_fwd.  N a
 *   multiple of 8, K at most 32768.  Deterministic; one launch, no workspace. */
dp_status dp_int4_quantize(const void* w, int64_t ldw, int w_f32, int64_t rows, int64_t K, int64_t group, void* q, void* s,
                           int s_f32, void* z, dp_stream stream);
dp_status dp_int4_dequantize(const void* q, const void* s, int s_f32, const void* z, int64_t rows, int64_t K, int64_t group,
                             void* w, int64_t ldw, dp_out_dtype out, dp_stream stream);
dp_status dp_gemm_fwd_int4(const void* X, int64_t ldx, const void* Wq, const void* Ws, int s_f32, const void* Wz,
                           int64_t group, void* Y, int64_t ldy, int64_t T, int64_t N, int64_t K, dp_out_dtype out,
                           dp_stream stream);
dp_status dp_gemm_fwd_int4_grouped(const void* X, int64_t ldx, const void* Wq, const void* Ws, int s_f32, const void* Wz,
                                   int64_t group, const void* offsets, int offset_bits, void* Y, int64_t ldy,
                                   int64_t E, int64_t T, int64_t N, int64_t K, dp_out_dtype out, dp_stream stream);

/* ------------------------------------------------------------ planning, misc */
/* Tuning and test overrides.  They are read from the environment only in a
 * process that has DP_TUNING set when the library first plans a call; such a
 * process reads them again on every call (so a test can change them between
 * calls).  Without DP_TUNING no call reads the environment.  The variables:
 * DP_FORCE_BN (64 / 128 / 256), DP_FORCE_SPLITS (uniform split count),
 * DP_FORCE_TAIL_SPLITS (split only the last partial wave, this many ways),
 * DP_FORCE_SWAP (0 / 1: BF16 weight-gradient orientation), DP_FORCE_PAIR (0 / 1:
 * single-CTA or CTA-pair tiles), DP_FORCE_CLUSTER_SUM=0 (sum split partials in
 * the reduction kernel instead of inside the GEMM's clusters; the two give the
 * same bits), DP_FORCE_TMA_STORE (0 / 1: the epilogue's whole-tile TMA stores off
 * / on for every non-transposed output; both store paths give the same bits),
 * DP_FORCE_STORE2=0 (FP32 whole tiles store one 32 x 32 block per TMA store
 * instead of two; the same bits), DP_FORCE_EPI_SINGLE=1 (one TMA-store staging
 * block per epilogue warp instead of two; the same bits), DP_FORCE_EVICT_FIRST=0
 * (no L2 evict-first policy on the operand a launch reads once; the same bits),
 * DP_FORCE_FUSE (0 / 1 / 2 / 3: dp_gemm_bwd as two calls or as one co-scheduled
 * launch, see dp_gemm_bwd), DP_FORCE_STREAM_K (0: never; 1: a stream-K plan where
 * the shape admits one), DP_FORCE_ATOMIC (calls with deterministic = 0: 0 ordered
 * split sums, 1 atomic ones wherever admitted), DP_FORCE_KPS (1 / 2 contraction
 * blocks per ring stage; BF16x3 plans keep 1), DP_FORCE_FFMA (0 / 1: the router's
 * BF16x3 or SIMT program), DP_FORCE_GROUP (raster group width in tiles) and
 * DP_FORCE_RASTER_M (1: groups of row tiles, 0: of column tiles).
 * The 8-bit products read DP_FORCE_BN (128 / 256), DP_FORCE_PAIR and DP_FORCE_SPLITS (1: no
 * split; 2 to 8: clusters of that many CTAs share a tile's contraction); a call that
 * has no such form is refused with DP_ERR_UNSUPPORTED.  The products with 4-bit weights read
 * DP_FORCE_INT4_TEAMS (1 / 4: how an SM's warps share its work) and DP_FORCE_INT4_TOKENS (1 to 16
 * tokens a pass, fewer where shared memory does not hold them), their quantisation and expansion
 * DP_FORCE_INT4_ROWS (rows a launch, at most as many as are counted in 31 bits); dp_expert_sort
 * reads DP_FORCE_SORT_CLUSTER (0: two launches, 1: one of a cluster).
 * A forced plan is still deterministic and keeps the accumulation-length bound. */

/* The plan the library uses for one call.  The planner is a pure function of
 * (op, T, N, K, out, sm_count), so a workspace sized here fits the call. */
typedef struct dp_plan_info {
    int32_t block_m;          /* output tile rows (128, or 256 for a CTA pair) */
    int32_t block_n;          /* output tile columns (64, 128 or 256) */
    int32_t block_k;          /* contraction block (64 elements = 64 tokens for wgrad; 32 for
                                 the router's forward and weight gradient) */
    int32_t stages;           /* shared-memory pipeline depth */
    int32_t splits;           /* contraction splits per output tile (1 = whole K per tile) */
    int32_t raster_group;     /* tiles per raster group (columns, or rows if raster_rows) */
    int32_t grid;             /* persistent CTAs launched (<= sm_count; even for a pair) */
    int32_t a_mn_major;       /* A operand read MN-major (1) or K-major (0) */
    int32_t b_mn_major;       /* B operand read MN-major (1) or K-major (0) */
    int32_t swap_ab;          /* weight gradient as dW^T = X^T dY (thin N as the MMA's N),
                                 stored transposed into dW */
    int32_t cta_pair;         /* 1: tiles of 256 rows shared by a cluster of two CTAs */
    int32_t raster_rows;      /* 1: raster groups of row tiles, rows fastest (B is the larger
                                 operand, or more than half the L2) */
    int32_t stream_k;         /* 1: the grid's slots share all tiles' contraction blocks evenly
                                 (slot c takes blocks [c W / grid_slots, (c + 1) W / grid_slots)
                                 of the tile-major order, W = tiles * k_blocks); a tile cut by
                                 slot boundaries is summed from up to `splits` pieces in block
                                 order; units counts the pieces */
    int64_t gemm_m;           /* output rows of the contraction */
    int64_t gemm_n;           /* output columns */
    int64_t gemm_k;           /* contraction length (3N for the router's input gradient,
                                 which contracts concatenated [lo|hi|hi] x [hi;lo;hi] copies) */
    int64_t tiles_m;
    int64_t tiles_n;
    int64_t k_blocks;         /* ceil(gemm_k / block_k) */
    int64_t units;            /* full_units + (tiles_m * tiles_n - full_units) * splits */
    int64_t full_units;       /* leading whole-K units; the remaining tiles are split */
    uint64_t workspace_bytes; /* == dp_workspace_size() */
    double model_us;          /* the planner's modelled duration of the call (diagnostic) */
    int64_t batch;            /* independent problems in the launch (1 except batched calls) */
    int64_t tiles;            /* batch * tiles_m * tiles_n */
    int32_t weight_kn;        /* batched calls: W / dW stored [K][N] */
    int32_t program;          /* router: 0 tensor-core BF16x3 program, 1 SIMT FP32 program
                                 (64 x block_n tiles, `splits` CTAs per tile, block_k
                                 contraction elements per stage); BF16 ops: 0 */
    int32_t atomic;           /* 1: split units add into the zero-filled FP32 output with
                                 atomic adds (deterministic = 0 only) */
    int32_t blocks_per_stage; /* contraction blocks per stage of the operand ring (1 or 2: a
                                 stage's loads complete on one barrier, so streaming plans
                                 carry two blocks per stage in half as many stages) */
    int32_t cluster_sum;      /* split plans with one unit per CTA: the tile's `splits` CTAs
                                 run as one thread-block cluster and sum their partials
                                 themselves after the main loop, with no reduction kernel
                                 (the cluster size, 2..8).  0: the reduction kernel sums the
                                 split partials, or the plan has none.  It depends on how
                                 many such clusters the device runs at once, so it is known
                                 only for the current device (sm_count <= 0); -1 otherwise */
} dp_plan_info;

/* Fill `info` with the plan for a call on a GPU with `sm_count` SMs
 * (sm_count <= 0: query the current device).  Pure host function. */
dp_status dp_plan_query(dp_op op, int64_t T, int64_t N, int64_t K, dp_out_dtype out,
                        int sm_count, dp_plan_info* info);
/* The same for a call with the given `deterministic` flag (dp_plan_query is
 * deterministic = 1).  A non-deterministic plan needs no more workspace than the
 * deterministic one of the same call. */
dp_status dp_plan_query_ex(dp_op op, int64_t T, int64_t N, int64_t K, dp_out_dtype out, int deterministic,
                           int sm_count, dp_plan_info* info);
/* The same for a batched BF16 call (op DP_OP_FWD / DGRAD / WGRAD, B >= 1). */
dp_status dp_plan_query_batched(dp_op op, int64_t B, int64_t T, int64_t N, int64_t K, dp_out_dtype out,
                                int weight_kn, int sm_count, dp_plan_info* info);

/* The backward pass's plan: the form chosen and the plan of each problem (for the
 * co-scheduled launch, whole-K plans of one tile shape; grid is the launch's). */
typedef struct dp_bwd_plan_info {
    int32_t fused;            /* 1: one co-scheduled launch; 0: two single-op calls */
    int32_t wgrad_first;      /* co-scheduled: the weight gradient's tiles are dealt first */
    int32_t grid;             /* co-scheduled: persistent CTAs of the launch (else 0) */
    int32_t blocks_per_stage; /* co-scheduled: contraction blocks per ring stage, for both
                                 problems (else 0; each call's own is in dgrad / wgrad) */
    double model_us;          /* modelled duration of the chosen form */
    double separate_us;       /* modelled duration of the two single-op calls */
    uint64_t workspace_bytes; /* == dp_workspace_size_bwd() */
    dp_plan_info dgrad;       /* input-gradient problem */
    dp_plan_info wgrad;       /* weight-gradient problem */
} dp_bwd_plan_info;
dp_status dp_plan_query_bwd(int64_t T, int64_t N, int64_t K, dp_out_dtype out_dx, dp_out_dtype out_dw,
                            int sm_count, dp_bwd_plan_info* info);

/* Workspace bytes a call needs (see dp_plan_query for sm_count). */
dp_status dp_workspace_size(dp_op op, int64_t T, int64_t N, int64_t K, dp_out_dtype out,
                            int sm_count, size_t* bytes);
dp_status dp_workspace_size_batched(dp_op op, int64_t B, int64_t T, int64_t N, int64_t K, dp_out_dtype out,
                                    int weight_kn, int sm_count, size_t* bytes);
dp_status dp_workspace_size_bwd(int64_t T, int64_t N, int64_t K, dp_out_dtype out_dx, dp_out_dtype out_dw,
                                int sm_count, size_t* bytes);

/* Check the device's architecture and set kernel attributes on `device`
 * (the current device if < 0).  Optional: the first call on a device does it. */
dp_status dp_init(int device);

/* Debug read-out: synchronise the current device and report whether any kernel
 * of this library gave up waiting (DP_ERR_TIMEOUT), or else was given group offsets
 * that decrease or leave [0, T], or rows of pairs outside their buffer (DP_ERR_INVALID_ARG), since
 * the last clear.
 * `clear` != 0 resets the flag.  Not for use inside stream capture. */
dp_status dp_device_error(int clear);

/* Test entry for the kernels' bounded waits (the failure-detection path).  Every
 * barrier wait in this library's kernels gives up after a time limit that is a
 * launch argument (2 s in the calls above), records the fault in the device status
 * word that dp_device_error() reports as DP_ERR_TIMEOUT, and lets the kernel
 * unwind and return instead of hanging the GPU.  This call enqueues on `stream` one
 * CTA that waits through that same bounded wait, with limit `limit_ns`
 * (1e3 .. 2e9 ns, else DP_ERR_INVALID_ARG), on a shared-memory barrier that nothing
 * arrives on (arrive = 0: the wait runs out and the kernel records the timeout) or
 * that the waiting thread arrived on first (arrive != 0: it returns at once and
 * records nothing).  The kernel holds no TMEM and issues no copies, so it ends
 * either way and the stream stays usable.  No counterpart on the pages: it exists
 * so the timeout path can be tested on a GPU without faulting or hanging one. */
dp_status dp_wait_probe(uint64_t limit_ns, int arrive, dp_stream stream);

/* Static description of a status code. */
const char* dp_status_string(dp_status status);

/* Library ABI version (major * 10000 + minor * 100 + patch). */
int dp_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DP_GEMM_H */
