/*
 * ns_hip.h - C ABI of the MI355X (gfx950) Newton–Schulz orthogonalization
 * library, libns_hip.so.
 *
 * The operation is Muon's quintic Newton–Schulz iteration applied to one
 * matrix or to a stack of independent matrices [batch, rows, cols]:
 *
 *   X  <- X / (||X||_F + 1e-7)            per matrix (slice)
 *   work on Xᵀ if rows > cols              (result returned untransposed)
 *   repeat ns_steps times:
 *     A = X Xᵀ,   B = b A + c A A,   X = a X + B X
 *
 * Sources (page title, section):
 *   - prime-rl PR #3873 (Muon optimizer-step speedups), "Summary" item 1:
 *     X Xᵀ and b A + c A A on a symmetric GEMM that computes one triangle and
 *     mirrors it; a X + B X as one GEMM with the scalar folded in; fp32
 *     alpha/beta epilogue (microbenchmark note under the NS table).
 *   - same page, "Summary" item 2: a 3-D stack is a batch along its leading
 *     axis; each slice is orthogonalized on its own.
 *   - param-decomp PR #978 "stacked-NS Muon", section "What": same-shape
 *     leaves batched into one NS; ns_steps (default 5); ns_dtype float32 or
 *     bfloat16.
 *   - Megatron-LM PR #6381 "Add --muon-use-syrk option ...", "Summary": the
 *     Gram product is symmetric, so a SYRK needs about half a GEMM's FLOPs;
 *     "Version compatibility": a requested fast path that cannot run must be
 *     a hard error, never a silent fallback (hence the status codes below).
 *
 * Conventions for every entry point:
 *   - Pointers named in/out/x/... are DEVICE pointers on the calling thread's
 *     current HIP device, 16-byte aligned, to contiguous row-major data.
 *     The caller owns them; the library never frees or retains them.
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream).
 *     All work is enqueued on it; calls return after enqueueing, without a
 *     host synchronisation.
 *   - Argument errors are detected on the host before anything is enqueued;
 *     no partial work is left behind.  Every call returns an ns_status.
 *   - No entry point falls back to another implementation.
 *   - Calls that share a device AND a stream share one library-owned
 *     workspace and are ordered by that stream, also calls of several host
 *     threads: one enqueues all its work before the other's begins.  Calls
 *     on different streams get different workspaces.
 *     A captured call keeps the workspace of the stream it was captured on:
 *     its replays must not overlap in time with calls on that stream, nor
 *     with replays of other graphs that were captured on it.
 */
#ifndef NS_HIP_H
#define NS_HIP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ------------------------------------------------------ */
typedef enum {
  NS_OK = 0,
  NS_ERR_INVALID_ARG = 1, /* null pointer, non-positive size, ns_steps < 0,
                             rows*cols >= 2^31, partial overlap in/out    */
  NS_ERR_DTYPE = 2,       /* dtype is not NS_DTYPE_F32 / NS_DTYPE_BF16    */
  NS_ERR_ALIGNMENT = 3,   /* a pointer not 16-byte aligned; for the stage
                             exports also rows or cols not a multiple of 8 */
  NS_ERR_ARCH = 4,        /* current device is not gfx950                 */
  NS_ERR_OOM = 5,         /* workspace allocation failed                  */
  NS_ERR_HIP = 6,         /* a HIP runtime call or launch failed;
                             details in ns_last_error()                   */
  NS_ERR_SCRATCH = 7      /* ns_orthogonalize_noalloc: the call needs more
                             than NS_NOALLOC_SCRATCH_BYTES of workspace    */
} ns_status;

/* Storage and compute dtype of every matrix of one call. */
enum {
  NS_DTYPE_F32 = 0,  /* fp32 storage, fp32 MFMA, fp32 epilogues           */
  NS_DTYPE_BF16 = 1  /* bf16 storage, bf16 MFMA with fp32 accumulation,
                        fp32 epilogues, fp32 diagonals (see below)        */
};

/*
 * ns_orthogonalize - the whole method on a stack of matrices.
 *
 *   in, out   device pointers to [batch, rows, cols] row-major, `dtype`.
 *             out may be the same pointer as in (in-place); any other
 *             overlap is NS_ERR_INVALID_ARG.  out always has the input's
 *             orientation (tall inputs are NOT returned transposed).
 *   batch     number of independent slices (0..65535; 0 enqueues nothing).
 *   rows,cols slice shape, each > 0.  When rows or cols is not a multiple
 *             of 8 the call zero-pads each slice to multiples of 8 in the
 *             workspace, runs on the padded copy and copies the caller's
 *             block back (zero rows and columns add only zero singular
 *             values, so the result is NS of the caller's matrix); the pad
 *             and unpad passes cost two extra copies of the stack.
 *   dtype     NS_DTYPE_F32 or NS_DTYPE_BF16.
 *   ns_steps  number of quintic steps (>= 0; 0 returns X / (||X||_F + eps)).
 *   a, b, c   quintic coefficients (Muon's usual: 3.4445, -4.7750, 2.0315).
 *   stream    hipStream_t as void*.
 *
 * Each slice is normalised by its own Frobenius norm.  An all-zero slice
 * yields zeros.  NaN/Inf inputs propagate; they are not checked.  The sum
 * of squares and the first Gram product accumulate the raw input in fp32
 * (the 1/||X|| scaling is applied in their epilogues), so a slice whose
 * ||X||_F exceeds about 1.8e19 (its sum of squares past the fp32 range)
 * gives no meaningful result (NaN or zeros).
 * Internally the Gram matrix A and the polynomial C = aI + bA + cAA are held
 * as an off-diagonal matrix (zero diagonal) in `dtype` plus an fp32 diagonal
 * vector; only lower-triangle tiles of both are computed.  C is mirrored;
 * A is mirrored too, except on large bf16 stacks, where it is kept as its
 * lower block triangle and the polynomial reads the rest transposed.
 * The workspace (ns_workspace_bytes) is allocated on first use per
 * (device, stream) and grown when needed.  Growing allocates a new buffer of
 * at least twice the old one's size (of the call's own, where there is no room
 * for that) without synchronising; the replaced one stays allocated (work queued
 * earlier may still use it) until ns_release_workspace.  Where there is room, a
 * stream thus holds at most four times what its largest call needs.  Once the workspace
 * of (device, stream) is at least this call's size, a call makes no
 * allocation and no synchronisation: it enqueues only kernels (and, in place
 * with an odd step count, one device copy), so it can be captured into a
 * HIP graph, provided the capture runs on that same stream and workspace
 * poisoning is off.
 */
int ns_orthogonalize(const void* in, void* out, int64_t batch, int64_t rows,
                     int64_t cols, int dtype, int ns_steps, float a, float b,
                     float c, void* stream);

/* Bytes of library workspace one ns_orthogonalize call of this shape needs. */
size_t ns_workspace_bytes(int64_t batch, int64_t rows, int64_t cols, int dtype);

/*
 * ns_orthogonalize_noalloc - ns_orthogonalize for callers that cannot
 * allocate device memory: code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc.
 *
 * Same arguments, checks, kernels and results as ns_orthogonalize (bitwise),
 * but the workspace is a fixed device array inside the library, one copy
 * per GPU, of NS_NOALLOC_SCRATCH_BYTES (256 MiB), held from the moment the
 * library's code is loaded on that GPU until the process ends.  The call
 * makes no device allocation (no hipMalloc, no hipFree, no allocating
 * library routine) and no synchronisation; the caller still provides in and
 * out.  A shape whose ns_workspace_bytes() exceeds NS_NOALLOC_SCRATCH_BYTES
 * is rejected with NS_ERR_SCRATCH before anything is enqueued (256 MiB
 * covers, e.g., bf16 4096 x 4096, 4096 x 14336 and 16 x 1536 x 2048).
 *
 * Every call on a GPU uses that GPU's one array and leaves its last contents
 * there; nothing in it has to start at zero (every kernel writes what a later
 * one reads).  Calls that overlap in time on one GPU - on different streams,
 * or from different threads without ordering - race on the array; order
 * them on one stream.  Kernel timing (ns_timing_*) does not apply to this
 * entry point.  Workspace poisoning (ns_set_workspace_poison) does, with
 * a memset of the array.
 */
#define NS_NOALLOC_SCRATCH_BYTES ((size_t)256 << 20)
int ns_orthogonalize_noalloc(const void* in, void* out, int64_t batch,
                             int64_t rows, int64_t cols, int dtype,
                             int ns_steps, float a, float b, float c,
                             void* stream);

/*
 * ns_orthogonalize_grouped - the same method on several stacks of different
 * shapes in one call (param-decomp PR #978, "What": same-shape leaves are
 * batched into one NS; here leaves of different shapes share the launches
 * too, and prime-rl PR #3873, "Summary" item 2: each slice on its own).
 *
 *   n_groups  number of stacks, 0..NS_MAX_GROUPS (0 enqueues nothing).
 *   in, out   HOST arrays of n_groups DEVICE pointers; stack g is
 *             [batch[g], rows[g], cols[g]] row-major at in[g], result at
 *             out[g], with ns_orthogonalize's rules for each pair
 *             (out[g] == in[g] allowed, any other overlap is an error).
 *             No out[g] may overlap another stack's in or out.
 *   batch, rows, cols
 *             HOST arrays of n_groups sizes, each checked as in
 *             ns_orthogonalize (batch[g] == 0: stack g is skipped and
 *             its pointers are not read, so they may be NULL).
 *   dtype, ns_steps, a, b, c, stream
 *             as in ns_orthogonalize, shared by every stack.
 *
 * The host arrays are read during the call only.  Each step runs at most
 * five launches whatever the number of stacks (Gram of the wide stacks,
 * Gram of the tall ones, one poly over all, update of the wide, update of
 * the tall; each split per 16 stacks), so many small leaves fill the GPU
 * together.  Every slice's result is bitwise the one ns_orthogonalize gives
 * for it.  ns_steps == 0 runs the stacks one after another.  Errors in any
 * stack are reported before anything is enqueued, with the stack's index in
 * ns_last_error().
 */
#define NS_MAX_GROUPS 4096
int ns_orthogonalize_grouped(int n_groups, const void* const* in, void* const* out,
                             const int64_t* batch, const int64_t* rows,
                             const int64_t* cols, int dtype, int ns_steps,
                             float a, float b, float c, void* stream);

/* Bytes of library workspace one ns_orthogonalize_grouped call needs (0 for
 * invalid arguments). */
size_t ns_workspace_bytes_grouped(int n_groups, const int64_t* batch,
                                  const int64_t* rows, const int64_t* cols,
                                  int dtype);

/* Free every cached workspace (all devices and streams), replaced ones
 * included.  Synchronises each device that held one.  Must not run while
 * another thread is inside a call; graphs that were captured before hold
 * what it frees and must not be replayed after.  Returns NS_OK or NS_ERR_HIP. */
int ns_release_workspace(void);

/* Number of workspace allocations (hipMalloc) the library has made since it
 * was loaded.  A call whose workspace is warm leaves it unchanged. */
int64_t ns_workspace_allocations(void);

/* ---- diagnostics --------------------------------------------------------- */

/* Static description of a status code. */
const char* ns_status_string(int status);

/* Text of the last error raised on the calling thread ("" if none). */
const char* ns_last_error(void);

/* Writes (NUL-terminated, truncated to n) a description of the kernels and
 * tile shapes the last successful call on this thread enqueued, so that a
 * caller can tell which path ran.  Returns the full length. */
int ns_query_last_config(char* buf, size_t n);

/*
 * Per-kernel timing with HIP events on the launch stream.
 * ns_timing_enable(mask): from now on, every launch of a kernel whose kind
 * bit is set in `mask` (1 << NS_KIND_*) records two hipEvents in its own
 * dispatch packet (hipExtLaunchKernel: the kernel's start and end), so no
 * packet goes between the kernels of a call; 0 disables.  The events are
 * timing-only (no system-scope fence); the stream must be synchronised
 * before their results are read on the host.  A timed dispatch still
 * releases its events at its end, which delays the next kernel by a few
 * microseconds: time a sample of the launches (ns_timing_sample) where the
 * call's own duration matters.
 * ns_timing_sample(every, offset): time only launch i of each kind (counted
 * from the last reset) with i % every == offset; every = 1, offset = 0 (the
 * default) times them all.  NS_ERR_INVALID_ARG unless 0 <= offset < every.
 * ns_timing_reset() drops the records and restarts the launch counts.
 * ns_timing_query(kind, &total_ms, &launches) waits for the recorded events
 * and returns the summed kernel time and the number of launches recorded.
 */
enum {
  NS_KIND_SUMSQ = 0,   /* per-slice sum of squares (norm, pass 1)        */
  NS_KIND_SCALE = 1,   /* scale and cast (norm, pass 2)                   */
  NS_KIND_GRAM = 2,    /* lower-triangle X Xᵀ (mirrored or lower-only)    */
  NS_KIND_POLY = 3,    /* lower-triangle C = aI + bA + cAA with mirror     */
  NS_KIND_UPDATE = 4,  /* X' = C X (or X C for tall), diagonal folded     */
  NS_KIND_LAYER_NORM = 5,  /* layer norm, forward and backward            */
  NS_KIND_ROUTE = 6,       /* routing with its plan, forward and backward */
  NS_KIND_EXPERTS = 7,     /* the experts' products and their gradients   */
  NS_KIND_COMBINE = 8,     /* weighted sum per token, and its gradient    */
  NS_KIND_RMS_NORM = 9,    /* RMS norm, forward and backward              */
  NS_KIND_QUANTIZE = 10,   /* values to 8 bits with scales, and back      */
  NS_KIND_COUNT = 11
};
int ns_timing_enable(int mask);
int ns_timing_sample(int every, int offset);
int ns_timing_reset(void);
int ns_timing_query(int kind, double* total_ms, int64_t* launches);

/*
 * Diagnostic: with on != 0, every later ns_orthogonalize and
 * ns_orthogonalize_grouped call first fills its whole workspace with 0xFF
 * bytes (NaN in bf16 and in fp32) on its stream, so that any kernel reading
 * a workspace element that no earlier kernel of the call wrote turns the
 * result into NaN.  0 turns it off (the default).  For tests: it costs one
 * fill of the workspace per call, enqueued as a memset, so keep it off
 * while a stream is being captured into a graph.  Returns NS_OK.
 */
int ns_set_workspace_poison(int on);

/*
 * Roofline calibration on the current device (a measurement helper; no step
 * of the method): every wave of two workgroups per CU runs `iters` (a
 * multiple of 4, at most 2^30) rounds of four back-to-back MFMAs on
 * registers only, v_mfma_f32_32x32x16_bf16 (dtype 1) or
 * v_mfma_f32_32x32x2_f32 (dtype 0), with operands that change from one
 * instruction to the next.  Writes the achieved dense rate in TFLOP/s (HIP
 * events on `stream`) and the average shader clock in MHz over the loop
 * (s_memtime against the constant-rate s_memrealtime).  Allocates and frees
 * its own small buffers and synchronises with the stream; about 0.1 s at
 * iters = 2^20.  Errors: NS_ERR_DTYPE, NS_ERR_INVALID_ARG (null outputs,
 * iters out of range), NS_ERR_ARCH, NS_ERR_HIP.
 */
int ns_peak_mfma(int dtype, int64_t iters, double* tflops, double* clock_mhz, void* stream);

/* ---- single stages (the same kernels ns_orthogonalize runs) ------------- */
/* Shapes: a slice of x is rows x cols, both multiples of 8 (the stages do
 * not pad); m = min(rows, cols).  The Gram side is the short one: A = X Xᵀ
 * when rows <= cols, A = Xᵀ X when rows > cols. */

/* X0 = x / (||x||_F + 1e-7) per slice, same shape, layout and dtype.
 * norms (optional, may be NULL): fp32 [batch] receives ||x||_F per slice.
 * x0 may equal x. */
int ns_stage_normalize(const void* x, void* x0, float* norms, int64_t batch,
                       int64_t rows, int64_t cols, int dtype, void* stream);

/* Gram of each slice: a_off [batch, m, m] (dtype) receives the off-diagonal
 * entries with exact zeros on the diagonal and is bitwise symmetric;
 * a_diag fp32 [batch, m] receives the diagonal. */
int ns_stage_gram(const void* x, void* a_off, float* a_diag, int64_t batch,
                  int64_t rows, int64_t cols, int dtype, void* stream);

/* C = a I + b A + c A A from A = a_off + diag(a_diag), stored the same way:
 * c_off [batch, m, m] (zero diagonal, bitwise symmetric), c_diag fp32
 * [batch, m].  a_off must be symmetric with a zero diagonal. */
int ns_stage_poly(const void* a_off, const float* a_diag, void* c_off,
                  float* c_diag, int64_t batch, int64_t m, int dtype, float a,
                  float b, float c, void* stream);

/* One update with C = c_off + diag(c_diag):
 *   rows <= cols:  x_out = C x         (C is rows x rows)
 *   rows >  cols:  x_out = x C         (C is cols x cols)
 * x_out must not overlap x. */
int ns_stage_update(const void* x, const void* c_off, const float* c_diag,
                    void* x_out, int64_t batch, int64_t rows, int64_t cols,
                    int dtype, void* stream);

/* ---- the mixture-of-experts sublayer ------------------------------------ */
/*
 * What stands around the expert stacks whose gradients ns_orthogonalize
 * takes: layer norm, routing of tokens to experts, the experts' products with
 * their gradients (the weight gradient is a stack [experts, fan_out, fan_in])
 * and the weighted sum of the experts' outputs per token.
 *
 * The conventions above hold, with these additions:
 *   - Matrices of tokens are row-major; where a leading dimension (ld...) is
 *     given, rows are that many elements apart.  Every other operand is
 *     contiguous.  Index, offset and fp32 vectors need 4-byte alignment only.
 *   - Outputs share no memory with inputs or with each other
 *     (NS_ERR_INVALID_ARG).
 *   - A row's length, and the elements between rows, are at most 2^20, a row
 *     count below 2^31; tokens * top_k of ns_route and n_rows of the experts'
 *     products are at most 2^31 - 1024.
 *   - Sums are taken in fp32 and every result is rounded once to its type.
 *     No atomics touch a floating-point value: the same inputs give the same
 *     bits.
 *   - Index data on the device (ids, offsets, rows, slots) is not trusted:
 *     values out of range are skipped, as said at each entry point, and never
 *     lead outside a buffer.
 */

/*
 * ns_layer_norm - y = (x - mean) rstd weight + bias over the columns of each
 * row, rstd = 1 / sqrt(var + eps), var the mean squared distance from mean.
 *
 *   x         [rows, cols] dtype, rows ldx >= cols elements apart.
 *   weight, bias
 *             [cols] param_dtype, or NULL (1 and 0).
 *   y         [rows, cols] dtype.
 *   mean, rstd
 *             fp32 [rows], or NULL; the backward pass needs them.
 *   rows == 0 enqueues nothing.
 */
int ns_layer_norm(const void* x, int64_t ldx, const void* weight, const void* bias,
                  void* y, float* mean, float* rstd, int64_t rows, int64_t cols,
                  int dtype, int param_dtype, float eps, void* stream);

/*
 * ns_layer_norm_backward - gradients of ns_layer_norm from dy [rows, cols]:
 *   dx [rows, cols] dtype, dweight and dbias [cols] param_dtype; each may be
 *   NULL.  weight is the forward pass's (NULL: 1), mean and rstd are what it
 *   returned.  With rows == 0 dweight and dbias become zero.  Uses library
 *   workspace (8 bytes per column and block, at most 256 MiB).
 */
int ns_layer_norm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                           const void* weight, const float* mean, const float* rstd,
                           void* dx, void* dweight, void* dbias, int64_t rows,
                           int64_t cols, int dtype, int param_dtype, void* stream);

enum {
  NS_SCORE_SOFTMAX = 0, /* over all the token's logits */
  NS_SCORE_SIGMOID = 1  /* of each logit               */
};

/*
 * ns_route - chooses top_k of `experts` experts for each token.
 *
 *   logits    [tokens, experts] dtype, rows ld elements apart.
 *   bias      fp32 [experts], or NULL.  It moves the choice, not the weights.
 *   ids       int32 [tokens, top_k]: the experts with the largest keys, in
 *             descending order, equal keys by index.  The key is score + bias,
 *             or with no bias the logit itself; that of a logit of -inf is
 *             -inf in both.
 *   groups, top_groups, group_best
 *             the experts form `groups` groups of neighbours, ranked by the
 *             sum of their group_best (1 or 2) largest keys (scores with no
 *             bias), in which keys of -inf count for nothing; a group of
 *             nothing else comes last.  Only experts of the best top_groups
 *             are chosen.  1, 1 for no groups.
 *   weights   fp32 [tokens, top_k]: scale s / (sum of the chosen s + 1e-20)
 *             if renormalize, else scale s; s is the expert's score.
 *   offsets, rows, slots
 *             the plan of the experts' products, or all NULL: the choices
 *             sorted by expert, in token order within one.  Expert e has the
 *             sorted rows offsets[e] .. offsets[e + 1] (int32 [experts + 1]);
 *             sorted row i holds token rows[i] (int32 [tokens * top_k]);
 *             choice j of token t is sorted row slots[t, j] (int32).
 *
 * tokens < 2^25, experts <= 1024, top_k <= 64, groups <= 64 and a divisor of experts.
 * Keys that pass through exp are compared in 64 bits.  A logit of -inf takes
 * an expert out: it has score 0 and comes after all others of the kept groups,
 * whatever its bias; a row of nothing else has weights 0.  A NaN key
 * counts as -inf, a NaN score makes the weights it enters NaN; ids are always
 * top_k distinct experts.
 */
int ns_route(const void* logits, int64_t ld, const float* bias, int32_t* ids,
             float* weights, int32_t* offsets, int32_t* rows, int32_t* slots,
             int64_t tokens, int64_t experts, int64_t top_k, int64_t groups,
             int64_t top_groups, int group_best, int score, int renormalize,
             float scale, int dtype, void* stream);

/*
 * ns_route_backward - dlogits [tokens, experts] dtype from dweights fp32
 * [tokens, top_k], for the choice ids (which has no gradient).  A token's ids
 * are distinct; one outside [0, experts) is left out.
 */
int ns_route_backward(const void* logits, int64_t ld, const int32_t* ids,
                      const float* dweights, void* dlogits, int64_t tokens,
                      int64_t experts, int64_t top_k, int score, int renormalize,
                      float scale, int dtype, void* stream);

/*
 * ns_experts_product - y[i] = x[rows[i]] W_e^T for every sorted row i of every
 * expert e (a linear layer per expert, rows gathered on the way).
 *
 *   x         [n_x, fan_in] dtype, rows ldx elements apart (a multiple of 8);
 *             read through rows it must hold less than 2 GiB.
 *   rows      int32 [n_rows], fewer than 2^29, or NULL: sorted row i is row i
 *             of x.  A row number outside [0, n_x) reads as zeros.
 *   w         [experts, fan_out, fan_in] dtype.
 *   offsets   int32 [experts + 1] on the device, ascending from 0 to n_rows;
 *             values are clamped to [0, n_rows], and rows of y that no expert
 *             has are not written.
 *   y         [n_rows, fan_out] dtype.
 * fan_out and fan_in are multiples of 8 (NS_ERR_ALIGNMENT).
 */
int ns_experts_product(const void* x, int64_t ldx, int64_t n_x, const int32_t* rows,
                       const void* w, const int32_t* offsets, void* y, int64_t n_rows,
                       int64_t experts, int64_t fan_out, int64_t fan_in, int dtype,
                       void* stream);

/* ns_experts_input_grad - dx[i] = dy[i] W_e for every sorted row: dy
 * [n_rows, fan_out], dx [n_rows, fan_in].  ns_experts_combine without weights
 * adds the rows of dx up to the gradient of x. */
int ns_experts_input_grad(const void* dy, const void* w, const int32_t* offsets,
                          void* dx, int64_t n_rows, int64_t experts, int64_t fan_out,
                          int64_t fan_in, int dtype, void* stream);

/* ns_experts_weight_grad - dw[e] = sum over e's sorted rows of
 * dy[i]^T x[rows[i]]: [experts, fan_out, fan_in] dtype, all of it written
 * (zero for an expert without rows).  x, ldx, n_x, rows as in the product. */
int ns_experts_weight_grad(const void* dy, const void* x, int64_t ldx, int64_t n_x,
                           const int32_t* rows, const int32_t* offsets, void* dw,
                           int64_t n_rows, int64_t experts, int64_t fan_out,
                           int64_t fan_in, int dtype, void* stream);

/* ns_experts_combine - out[t] = sum over j of weights[t, j] y[slots[t, j]]:
 * y [n_rows, cols], out [tokens, cols] dtype, weights fp32 [tokens, top_k] or
 * NULL (1).  A slot outside [0, n_rows) adds nothing.  cols is a multiple of
 * 8. */
int ns_experts_combine(const void* y, const int32_t* slots, const float* weights,
                       void* out, int64_t tokens, int64_t top_k, int64_t n_rows,
                       int64_t cols, int dtype, void* stream);

/* ns_experts_combine_backward - dy[slots[t, j]] = weights[t, j] dout[t] and
 * dweights[t, j] = <dout[t], y[slots[t, j]]> (fp32; zero for a slot out of
 * range); either may be NULL.  Rows of dy that no slot names are not
 * written; no two choices may name the same row. */
int ns_experts_combine_backward(const void* dout, const void* y, const int32_t* slots,
                                const float* weights, void* dy, float* dweights,
                                int64_t tokens, int64_t top_k, int64_t n_rows,
                                int64_t cols, int dtype, void* stream);

/* ---- the sublayer in 8 bits ---------------------------------------------- */
/*
 * RMS norm with the residual's addition, values in 8 bits with scales, the
 * experts' product of such values, and the weight gradient from rows that were
 * kept in them.
 *
 * 8-bit values are e4m3 (4 exponent bits, 3 of mantissa, largest value 448, no
 * infinity, 0x7f and 0xff are NaN).  A scale is one byte b (E8M0): 2^(b - 127).
 *   rows      q [rows, cols], scales [rows, ceil(cols / 128)]: one for each 128
 *             columns of a row.
 *   weights   q [experts, fan_out, fan_in], scales [experts, ceil(fan_out / 128),
 *             ceil(fan_in / 128)]: one for each 128 x 128 block.
 * Last blocks may be short; cols, fan_out and fan_in are multiples of 16.  The
 * library's scales are 2^k with the least k >= -126 for which the block's largest
 * finite magnitude is at most 448 2^k; values are divided by it and rounded to the
 * nearest, ties to even; infinities and NaN become NaN.  Bytes 0 to 254 are read;
 * 255 is not a number, and so is every result that it enters.
 *
 * The conventions above hold.  q needs 16-byte alignment, scales none.
 */

/*
 * ns_rms_norm - y = t rstd weight over the columns of each row, t = x + residual,
 * rstd = 1 / sqrt(mean(t^2) + eps), in fp32.  Squares are added in 64 bits, so
 * every finite row has one; below 2^-126 (rows of 2^126 and more) it is rounded to
 * multiples of 2^-149, and where mean(t^2) + eps is below 2^-256 it is infinite.
 *
 *   x, residual
 *             [rows, cols] dtype, rows ldx and ldr elements apart; residual may
 *             be NULL (t = x).
 *   weight    [cols] param_dtype, or NULL (1).
 *   total     [rows, cols] dtype: t, rounded; with a residual, else NULL.  The
 *             norm is taken of t as it is stored.
 *   y         [rows, cols] dtype, or NULL.
 *   q, scales y as 8-bit rows (not rounded to dtype before), or both NULL.  One of
 *             y and q is given.
 *   rstd      fp32 [rows], or NULL; the backward pass needs it.
 *   rows == 0 enqueues nothing.
 */
int ns_rms_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                const void* weight, void* total, void* y, void* q, uint8_t* scales,
                float* rstd, int64_t rows, int64_t cols, int dtype, int param_dtype,
                float eps, void* stream);

/*
 * ns_rms_norm_backward - gradients of ns_rms_norm from dy [rows, cols]:
 *   dx [rows, cols] dtype (of x and of the residual alike) and dweight [cols]
 *   param_dtype; each may be NULL.  x is what the norm was taken of (total, where
 *   there was a residual), weight the forward pass's (NULL: 1), rstd what it
 *   returned.  dtotal [rows, cols] dtype, or NULL: the gradient that reaches total
 *   from elsewhere; it is added to dx.  With rows == 0 dweight becomes zero.  Uses
 *   library workspace (4 bytes per column and block, at most 128 MiB).
 */
int ns_rms_norm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                         const void* weight, const float* rstd, const void* dtotal,
                         int64_t lddt, void* dx, void* dweight, int64_t rows,
                         int64_t cols, int dtype, int param_dtype, void* stream);

/* ns_quantize - x [rows, cols] dtype, rows ldx elements apart, as 8-bit rows
 * (rows * ceil(cols / 128) below 2^32). */
int ns_quantize(const void* x, int64_t ldx, void* q, uint8_t* scales, int64_t rows,
                int64_t cols, int dtype, void* stream);

/* ns_quantize_weights - w [experts, fan_out, fan_in] dtype as 8-bit weights, and,
 * where qt and scales_t are not NULL, the same values transposed: qt [experts,
 * fan_in, fan_out] with its scales.  experts <= 1024, fan_out * fan_in < 2^29, fewer
 * than 2^24 blocks. */
int ns_quantize_weights(const void* w, void* q, uint8_t* scales, void* qt,
                        uint8_t* scales_t, int64_t experts, int64_t fan_out,
                        int64_t fan_in, int dtype, void* stream);

/* ns_dequantize - the values x [matrices, rows, cols] dtype of q and its scales;
 * block_rows 1: rows, 128: weights.  Exact in both types, but below 2^-126, where
 * x is rounded, and past the type's largest value (scales of 2^120 and more), where
 * it is infinite. */
int ns_dequantize(const void* q, const uint8_t* scales, void* x, int64_t matrices,
                  int64_t rows, int64_t cols, int block_rows, int dtype, void* stream);

/*
 * ns_experts_product_scaled - ns_experts_product of 8-bit rows and weights:
 * y[i] = x[rows[i]] W_e^T for every sorted row i of every expert e.
 *
 *   x, x_scales
 *             8-bit rows [n_x, fan_in]; read through rows, x must hold less than
 *             2 GiB.
 *   rows      int32 [n_rows], or NULL: sorted row i is row i of x.  A row
 *             outside [0, n_x) counts as zeros.
 *   w, w_scales
 *             8-bit weights [experts, fan_out, fan_in].
 *   offsets   int32 [experts + 1], or NULL for one expert that has all rows
 *             (a linear layer); clamped to [0, n_rows].
 *   y         [n_rows, fan_out] dtype; rows that no expert has are not written.
 *
 * The gradient of x is the same product of dy in 8 bits with the transposed
 * weights.  Results in bf16 come from the 8-bit matrix instructions, which add
 * eight neighbouring products at a time and cut each off at 2^-13 of the largest
 * one's power of two, everything else in fp32: at most 2^-10 of the sum of the
 * eights' largest products, and 1.5e-5 of the result (root mean square) in rows
 * of normal values.  Where large products cancel that may be more than the result's
 * rounding.  Results in fp32 are fp32 sums of exact products of x and w as
 * ns_dequantize gives them in bf16 (infinite past its largest value, which takes a
 * scale of 2^120 or more), at half the rate; rounded, they are the bf16 results of
 * exact products.  A launch of 2^32 threads or
 * more is an error: 2^30 rows and more, where it goes by tiles of 128 rows (fp32, or
 * fan_in of at most 384).
 */
int ns_experts_product_scaled(const void* x, const uint8_t* x_scales, int64_t n_x,
                              const int32_t* rows, const void* w,
                              const uint8_t* w_scales, const int32_t* offsets, void* y,
                              int64_t n_rows, int64_t experts, int64_t fan_out,
                              int64_t fan_in, int dtype, void* stream);

/*
 * ns_experts_weight_grad_scaled - ns_experts_weight_grad from rows x that were
 * kept in 8 bits: dw[e] = sum over its rows of dy[i]^T x[rows[i]], dy [n_rows,
 * fan_out] and dw [experts, fan_out, fan_in] in dtype.  offsets may be NULL for one
 * expert that has all rows, as in the product (a linear layer's gradient).  x is
 * restored in dtype in library workspace (n_x rows, or n_rows without rows), which
 * is less than 2 GiB where there are rows, and has no such limit without; it stays
 * allocated as every workspace does (ns_orthogonalize, ns_release_workspace).
 */
int ns_experts_weight_grad_scaled(const void* dy, const void* x, const uint8_t* x_scales,
                                  int64_t n_x, const int32_t* rows, const int32_t* offsets,
                                  void* dw, int64_t n_rows, int64_t experts,
                                  int64_t fan_out, int64_t fan_in, int dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* NS_HIP_H */
