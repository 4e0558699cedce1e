/*
 * muon_mi355x.h - C ABI of the batched Muon optimizer step for AMD MI355X (gfx950).
 *
 * The operation.  Muon is the optimizer used for almost all weight matrices of
 * the model described on "How PyTorch Scaled a Near-1T MoE on Europe's Public
 * Supercomputer" (§Three optimizations that changed the economics, FlexShard
 * bullet).  Its Newton-Schulz update works on whole matrices; placing whole
 * experts on one rank lets every rank orthogonalize its own matrices with no
 * communication, and running Newton-Schulz on the GPU instead of the host CPU
 * is what shortened the optimizer step there.  Muon keeps one optimizer state
 * per matrix ("Domyn is training a 1T-parameter MoE on Europe's Jupiter
 * supercomputer, and published the recipe", §What moved the number).
 *
 * For each matrix of a ragged batch, muon_step_batched computes
 *     M' = beta*M + G                          (momentum, the single state)
 *     U  = G + beta*M'  if nesterov, else M'
 *     X0 = U / (||U||_F + eps), transposed when rows > cols (short side)
 *     k times:  A = X X^T;  B = b*A + c*A*A;  X = a*X + B*X
 *     O  = X_k, transposed back to rows x cols
 *     W' = W - lr * sqrt(max(1, rows/cols)) * O
 * and muon_ns_batched computes O from U = x alone.  The pages fix no
 * polynomial, step count or epsilon; the usual quintic is
 * (a, b, c) = (3.4445, -4.7750, 2.0315) with k = 5, and (1.5, -0.5, 0) is the
 * cubic iteration that converges to the polar factor.
 *
 * Conventions shared by every entry point:
 *  - Matrices are dense, row-major, contiguous: element (i, j) of a rows x cols
 *    matrix is at ptr[i*cols + j].  One dtype covers every tensor of a call.
 *  - Device pointers (x, out, w, g, m, workspace) must be 16-byte aligned
 *    device memory of the current HIP device (m may be pinned host memory, see
 *    momentum_host).  Host arrays (rows, cols, the pointer arrays, the
 *    parameter structs) are read during the call only.
 *  - The buffers of different matrices of one call must not overlap (this is
 *    not checked); the aliasing allowed within one matrix is stated per entry
 *    point.
 *  - The caller owns every buffer, the workspace included.  The library
 *    allocates no device memory and keeps no pointer after it returns; it owns
 *    only a pool of small pinned host staging buffers for the descriptor
 *    upload, allocated on first use and kept until the process ends, and, once
 *    a step with momentum_host = 1 has run on a device, two copy streams and
 *    their events there.  A call takes a staging buffer whose upload has
 *    completed, or a new one when all are in flight (at most 256 per device).
 *  - Work is enqueued on `stream` (a hipStream_t; NULL is the default stream)
 *    and the call returns without waiting for the GPU, except with more than
 *    256 calls in flight on one device, when it waits for the oldest one's
 *    descriptor upload, and for a step with momentum_host = 1, which first
 *    waits for the previous such step on the device (see muon_step_params).  Buffers must stay alive and untouched until the
 *    stream has finished the work.  Two calls may run concurrently only with
 *    distinct workspaces.
 *  - Every argument is validated before anything is enqueued; on any error
 *    nothing is launched and the outputs are untouched.  batch == 0 is a no-op
 *    that returns MUON_OK.
 *  - NaN and Inf propagate; there is no check.  A zero input gives a zero
 *    output (eps keeps the normalization finite).
 *  - Results are deterministic: the kernels use no floating-point atomics.  The
 *    matrix-core launches hand out the last tiles of each XCD's share with
 *    integer atomics on counters in the workspace, to whichever XCD is free;
 *    which CU computes a tile never changes its value.
 *  - A call on a stream that is being captured into a HIP graph (per-kernel timing
 *    off) sends its descriptor table in kernel launches instead of a copy, so the
 *    graph can be replayed; it uses its workspace at every replay.  A step with
 *    momentum_host = 1 is refused there (MUON_ERR_UNSUPPORTED).
 *  - No C++ exception crosses this interface.
 *
 * Precision.  MUON_BF16: tensors are bf16; products accumulate in fp32 on the
 * matrix cores; every stored intermediate (X, A, B, M', W') is rounded to
 * nearest even.  MUON_FP32: tensors and all arithmetic are fp32.
 */
#ifndef MUON_MI355X_H
#define MUON_MI355X_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of every tensor in a call. */
typedef enum { MUON_BF16 = 0, MUON_FP32 = 1 } muon_dtype;

/* Return codes. */
typedef enum {
  MUON_OK = 0,
  MUON_ERR_INVALID_ARG = 1, /* null pointer, dim <= 0, misaligned pointer, bad dtype, steps < 0,
                               aliasing that is not allowed, non-finite parameter */
  MUON_ERR_UNSUPPORTED = 2, /* a dimension beyond the supported maximum (MUON_MAX_DIM) */
  MUON_ERR_WORKSPACE = 3,   /* workspace null or smaller than muon_workspace_bytes() */
  MUON_ERR_HIP = 4          /* a HIP runtime call or launch failed; see muon_last_error_detail() */
} muon_status;

/* Largest supported rows or cols of one matrix. */
#define MUON_MAX_DIM 65536

/* Newton-Schulz settings: X <- a*X + (b*A + c*A^2)*X with A = X X^T, `steps` times,
 * after X0 = U / (||U||_F + eps).  steps == 0 returns X0.  c == 0 skips A^2. */
typedef struct {
  int32_t steps;
  float a, b, c;
  float eps;
  /* 0: the matrix-core launches fill the GPU.  N > 0: each of them (bf16) keeps
   * at most N workgroups resident, one per CU, each looping over tiles, so that
   * work on other streams keeps the remaining CUs; this is for orthogonalizing
   * the dense matrices while expert compute goes on ("How PyTorch Scaled a
   * Near-1T MoE on Europe's Public Supercomputer", §Three optimizations that
   * changed the economics, FlexShard bullet).  Results do not depend on it,
   * bit for bit: with N = 0 the products that store the iterate take tiles of
   * 256 x 384 where every matrix allows it (bf16, every long side padded to a
   * multiple of 384), with N > 0 tiles of 256 x 256, and both add up every
   * element the same way. */
  int32_t cu_budget;
  /* e4m3 operands in the first fp8_steps iterations (0: none; bf16 only,
   * 0 <= fp8_steps < steps, no cu_budget).  FP8 for expert matrix math is an
   * open question on "Domyn is training a 1T-parameter MoE on Europe's Jupiter
   * supercomputer, and published the recipe" (§What moved the number, closing
   * paragraph).  In those iterations the three products take e4m3 operands
   * with one power-of-two scale per 32 elements along the contracted side
   * (the block maximum at most 448), formed from the bf16 X, A and B; the
   * products accumulate in fp32, the a X and b A terms are added in fp32 from
   * the bf16 matrices, and every result is stored in bf16 as before.  With
   * fp8_steps = 2 of 5 the output is as close to the exact iteration as the
   * bf16 path's; more e4m3 steps are not (the polynomial amplifies their
   * noise once the singular values have grown).  Such a call needs
   * muon_workspace_bytes_ex(..., MUON_WS_FP8) bytes of workspace. */
  int32_t fp8_steps;
} muon_ns_params;

/*
 * Full step settings: learning rate, momentum coefficient, Nesterov flag (0/1),
 * and where the momentum lives.
 *
 * momentum_host = 1 keeps the optimizer state in host memory, as the pages do
 * when they move optimizer state off the accelerator ("Domyn is training a
 * 1T-parameter MoE on Europe's Jupiter supercomputer, and published the
 * recipe", §What moved the number, Offloading bullet).  Every m[i] must then be
 * pinned host memory (hipHostMalloc, or a pinned torch tensor), updated in
 * place.  The batch then runs in up to 16 chunks of about equal momentum bytes:
 * a chunk's momentum is copied to the device by DMA, updated there, and copied
 * back as soon as the momentum pass is done, on two library-owned streams of
 * default priority, so that the copies of neighbouring chunks overlap this
 * chunk's Newton-Schulz work.  The results are bit-identical to momentum in
 * device memory.  The workspace must hold
 * muon_workspace_bytes_ex(..., MUON_WS_MOMENTUM_HOST) bytes, and m[i] must not
 * be touched by the host until the stream has finished the work.  Such a call
 * may block the calling thread: it first waits until the previous such call on
 * this device has finished on the GPU (with the copies of two calls queued at
 * once, the copies slow down by a large and varying factor).  It cannot be
 * captured into a HIP graph.
 * Otherwise (0) m[i] are device memory.
 */
typedef struct {
  float lr;
  float beta;
  int32_t nesterov;
  muon_ns_params ns;
  int32_t momentum_host;
} muon_step_params;

/*
 * Bytes of device workspace a call over this batch needs (the same for
 * muon_ns_batched and muon_step_batched).  rows[i], cols[i]: shape of matrix i.
 * Returns SIZE_MAX on invalid arguments (detail in muon_last_error_detail()).
 * batch == 0 returns 0.  Host-only: launches nothing, needs no GPU.
 */
size_t muon_workspace_bytes(int32_t batch, const int64_t* rows, const int64_t* cols, int32_t dtype);

/*
 * Bytes of device workspace a call with the options in `flags` needs:
 *   MUON_WS_FP8            a bf16 call with fp8_steps > 0: two e4m3 copies of
 *                          each padded iterate more (s_pad * l_pad bytes each,
 *                          plus a scale byte per 32)
 *   MUON_WS_MOMENTUM_HOST  a step with momentum_host = 1: the batch runs in up
 *                          to 16 chunks, each with its own part, plus two
 *                          staging slots for a chunk's momentum
 * flags = 0 is muon_workspace_bytes().  Returns SIZE_MAX on invalid arguments
 * or unknown flags.  Host-only.
 */
#define MUON_WS_FP8 1u
#define MUON_WS_MOMENTUM_HOST 2u
size_t muon_workspace_bytes_ex(int32_t batch, const int64_t* rows, const int64_t* cols,
                               int32_t dtype, uint32_t flags);

/*
 * Orthogonalize a ragged batch: out[i] = NS_k(x[i]) (shape rows[i] x cols[i]).
 *   batch       number of matrices (>= 0)
 *   rows, cols  host arrays[batch] of shapes, each in [1, MUON_MAX_DIM]
 *   x           host array[batch] of device pointers to the inputs (read only)
 *   out         host array[batch] of device pointers to the outputs; out[i] may equal x[i]
 *               (in place) but must not overlap another matrix's buffers otherwise
 *   dtype       MUON_BF16 or MUON_FP32
 *   p           Newton-Schulz settings (host pointer)
 *   workspace   device buffer of at least muon_workspace_bytes() bytes, 256-byte aligned
 *   stream      hipStream_t to enqueue on
 */
int32_t muon_ns_batched(int32_t batch, const int64_t* rows, const int64_t* cols,
                        const void* const* x, void* const* out, int32_t dtype,
                        const muon_ns_params* p, void* workspace, size_t workspace_bytes,
                        void* stream);

/*
 * For callers that cannot allocate device memory: code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc.  The same
 * orthogonalization as muon_ns_batched (same kernels, bit-identical results),
 * with no workspace argument: the workspace is a library-owned array of
 * MUON_NOALLOC_MAX_WORKSPACE bytes in device memory (one per GPU the library
 * runs on, held until the process ends).  The call allocates no device or
 * pinned memory and creates no HIP objects; it enqueues only kernel launches
 * on `stream` (the descriptor table travels as kernel arguments) and takes no
 * part in per-kernel timing.
 *   Arguments as muon_ns_batched.  A batch whose muon_workspace_bytes() exceeds
 *   MUON_NOALLOC_MAX_WORKSPACE returns MUON_ERR_WORKSPACE and launches nothing.
 *   Every call on one GPU uses that GPU's one array: calls that overlap on a GPU
 *   (on different streams, or from different threads) race and give undefined
 *   results.  Calls in order on one stream are safe; the array keeps the last
 *   call's contents, and every call writes each part it reads before reading it.
 */
#define MUON_NOALLOC_MAX_WORKSPACE ((size_t)256 << 20)
int32_t muon_ns_batched_noalloc(int32_t batch, const int64_t* rows, const int64_t* cols,
                                const void* const* x, void* const* out, int32_t dtype,
                                const muon_ns_params* p, void* stream);

/*
 * One Muon step over a ragged batch, in place on w[i] and m[i].
 *   w           host array[batch] of device pointers to the weights (updated in place)
 *   g           host array[batch] of device pointers to the gradients (read only)
 *   m           host array[batch] of device pointers to the momentum buffers (updated in place)
 *   w[i], g[i], m[i] must be pairwise distinct.  Other arguments as muon_ns_batched.
 */
int32_t muon_step_batched(int32_t batch, const int64_t* rows, const int64_t* cols,
                          void* const* w, const void* const* g, void* const* m, int32_t dtype,
                          const muon_step_params* p, void* workspace, size_t workspace_bytes,
                          void* stream);

/*
 * AdamW for the parameters Muon does not cover.  The model runs Muon on about
 * 99.5% of its parameters and AdamW on the rest ("Domyn is training a
 * 1T-parameter MoE on Europe's Jupiter supercomputer, and published the
 * recipe", §The model and the machine, optimizer row).  The pages do not spell
 * AdamW out; this is Adam with decoupled weight decay in the form PyTorch's
 * AdamW takes, for step number t >= 1 (the step being taken):
 *     p <- p * (1 - lr * weight_decay)
 *     m <- beta1 * m + (1 - beta1) * g
 *     v <- beta2 * v + (1 - beta2) * g^2
 *     p <- p - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
 * The arithmetic is fp32; the bias corrections are formed on the host in double.
 */
typedef struct {
  float lr;
  float beta1, beta2;     /* each in [0, 1) */
  float eps;              /* >= 0 */
  float weight_decay;
  int32_t step;           /* t >= 1 */
} muon_adamw_params;

/*
 * Bytes of device workspace muon_adamw_batched needs for this batch (the
 * descriptor table).  numel[i] >= 0: element count of tensor i.  Returns
 * SIZE_MAX on invalid arguments.  Host-only.
 */
size_t muon_adamw_workspace_bytes(int32_t batch, const int64_t* numel);

/*
 * One AdamW step over a ragged batch of flat tensors, in place.
 *   numel[i]   element count of tensor i (0 allowed: nothing to do)
 *   p[i], g[i] parameters and gradients, `dtype` elements (MUON_BF16 or MUON_FP32);
 *              p is updated in place, g is read only
 *   m[i], v[i] first and second moments, always fp32, updated in place
 *   workspace  device buffer of at least muon_adamw_workspace_bytes() bytes,
 *              256-byte aligned
 * Device pointers must be 16-byte aligned device memory; p, g, m and v of one
 * tensor must be distinct.  Conventions (ownership, stream, validation before
 * any launch, status codes) are those listed at the top of this header.
 */
int32_t muon_adamw_batched(int32_t batch, const int64_t* numel, void* const* p,
                           const void* const* g, float* const* m, float* const* v, int32_t dtype,
                           const muon_adamw_params* params, void* workspace,
                           size_t workspace_bytes, void* stream);

/*
 * Gradient clipping by the global norm, the usual step between the backward
 * pass and the optimizer: one norm over every gradient of the model (the
 * matrices Muon steps and the tensors AdamW steps together), and one factor
 *     n = sqrt(sum_i sum_j g_ij^2)         MUON_NORM_L2
 *     n = max_ij |g_ij|                    MUON_NORM_MAX
 *     s = min(1, max_norm / (n + eps))     (1 when clip = 0 or n + eps = 0)
 * Squares are formed and summed in double; n and s are rounded once, to fp32.
 * A NaN gradient gives n = s = NaN, an infinite one n = inf and s = 0.  The
 * library never looks at n on the host: every call stays asynchronous.
 *
 * The factor can be applied in two ways:
 *  - muon_grad_clip_batched, or muon_grad_scale_batched with a factor that was
 *    formed elsewhere (a norm over several ranks): out_ij = s * g_ij in fp32,
 *    rounded to out's type.  out[i] may be g[i] (of the same type; a factor of
 *    exactly 1 then leaves it untouched), or another buffer of either type: the
 *    fp32 sums of gradients over micro-batches go into the bf16 gradients that
 *    the step reads in the same pass.
 *  - muon_step_batched_scaled and muon_adamw_batched_scaled, which multiply
 *    each gradient by the factor in fp32 as they read it: no extra pass, and no
 *    rounding of s * g to the gradient's type.
 *
 * A tensor may appear more than once in a norm; no output may overlap another
 * tensor's gradient or output.
 *
 * The tensors of a norm, scale or clip may have different types: dtype[i] (and
 * out_dtype[i]) is MUON_BF16 or MUON_FP32 for tensor i.  Other conventions are
 * those at the top of this header.
 */
typedef enum { MUON_NORM_L2 = 0, MUON_NORM_MAX = 1 } muon_norm_kind;

typedef struct {
  int32_t kind;   /* muon_norm_kind */
  int32_t clip;   /* 1: form s from max_norm; 0: s = 1 (max_norm is not read) */
  float max_norm; /* >= 0, finite */
  float eps;      /* >= 0, finite; 1e-6 is usual */
} muon_grad_norm_params;

/* Bytes of device workspace the three calls below need.  numel[i] >= 0.
 * Returns SIZE_MAX on invalid arguments.  Host-only. */
size_t muon_grad_workspace_bytes(int32_t batch, const int64_t* numel);

/*
 * The global norm: result[0] = n, result[1] = s (device memory, 4-byte
 * aligned).  batch == 0 gives n = 0, s = 1.
 *   numel[i]   element count of tensor i (0 allowed)
 *   g[i]       16-byte aligned device pointer (not read when numel[i] is 0)
 *   workspace  at least muon_grad_workspace_bytes() bytes, 256-byte aligned
 */
int32_t muon_grad_norm_batched(int32_t batch, const int64_t* numel, const void* const* g,
                               const int32_t* dtype, const muon_grad_norm_params* p, float* result,
                               void* workspace, size_t workspace_bytes, void* stream);

/* out[i] = scale * g[i], scale[0] in device memory. */
int32_t muon_grad_scale_batched(int32_t batch, const int64_t* numel, const void* const* g,
                                const int32_t* dtype, void* const* out, const int32_t* out_dtype,
                                const float* scale, void* workspace, size_t workspace_bytes,
                                void* stream);

/* Both: result as muon_grad_norm_batched (p->clip must be 1), then
 * out[i] = result[1] * g[i].  result must lie outside every g[i] and out[i]. */
int32_t muon_grad_clip_batched(int32_t batch, const int64_t* numel, const void* const* g,
                               const int32_t* dtype, void* const* out, const int32_t* out_dtype,
                               const muon_grad_norm_params* p, float* result, void* workspace,
                               size_t workspace_bytes, void* stream);

/* muon_step_batched with every gradient multiplied by grad_scale[0] (fp32,
 * device memory, 4-byte aligned) in fp32 as it is read:
 *     M' = beta*M + s*G;  U = s*G + beta*M' if nesterov, else M'.
 * grad_scale is read on the stream, so it may be the result of an earlier call
 * there.  The workspace is that of muon_step_batched. */
int32_t muon_step_batched_scaled(int32_t batch, const int64_t* rows, const int64_t* cols,
                                 void* const* w, const void* const* g, void* const* m,
                                 int32_t dtype, const muon_step_params* p, const float* grad_scale,
                                 void* workspace, size_t workspace_bytes, void* stream);

/* muon_adamw_batched with g replaced by grad_scale[0] * g, likewise. */
int32_t muon_adamw_batched_scaled(int32_t batch, const int64_t* numel, void* const* p,
                                  const void* const* g, float* const* m, float* const* v,
                                  int32_t dtype, const muon_adamw_params* params,
                                  const float* grad_scale, void* workspace,
                                  size_t workspace_bytes, void* stream);

/*
 * Block-scaled e4m3 operands and their product, for the expert matrices whose
 * gradients the step takes: FP8 for expert matrix math is an open question on
 * "Domyn is training a 1T-parameter MoE on Europe's Jupiter supercomputer, and
 * published the recipe" (§What moved the number, closing paragraph).
 *
 * An operand of R rows, contracted over K columns, is two arrays, with
 * Kp = K rounded up to a multiple of MUON_F8_BLOCK and Rp = R rounded up to a
 * multiple of 16:
 *   values  R x Kp bytes, row-major: OCP e4m3 (no infinity, largest 448),
 *           columns K .. Kp-1 zero
 *   scales  Kp/MUON_F8_BLOCK x Rp bytes, row-major: byte [kb][r] = e + 127 (0 .. 254), the
 *           power of two 2^e that scales columns 128 kb .. 128 kb + 127 of row r;
 *           entries r >= R zero
 * Both 16-byte aligned.  A value stands for e4m3 * 2^e.
 *
 * muon_f8_quantize_batched forms the operands of a ragged batch of matrices
 * x[i] (rows[i] x cols[i], row-major, contiguous, `dtype`), of their
 * transposes, or of both from one read:
 *   block_rows  1: a scale of its own for each 1 x 128 block along the contracted
 *               side (activations, gradients); MUON_F8_BLOCK: one for each
 *               128 x 128 block of the matrix, written out for every row
 *               (weights: the operand and its transpose then hold the same values)
 *   q, s        values and scales of x[i] (contracted over its columns); both
 *               arrays null: not formed
 *   qt, st      those of x[i] transposed (contracted over its rows); likewise
 * e is the smallest exponent, at least -127, with the block's largest finite
 * magnitude at most 448 * 2^e, so nothing saturates; values are rounded to
 * nearest even.  An infinity or NaN becomes NaN and takes no part in the scale.
 *
 * muon_f8_matmul_batched: c[i] = A_i B_i^T (+ c[i] when accumulate = 1), A_i of
 * m[i] rows and B_i of n[i] rows, both contracted over k[i]:
 *   c[i]   m[i] x n[i], row-major, contiguous, `dtype` (MUON_BF16 or MUON_FP32)
 * summed in fp32 and rounded once, at the store (the old c is added in fp32
 * before it).  With a bf16 c the matrix cores first add 8 consecutive products
 * on a common grid: one of 2^-13 of the 8's largest counts, one of 2^-14 is lost.
 * The error of that is below 2^-10 of the sum of the products' magnitudes, and
 * 1.5e-5 of the result on Gaussian operands (measured); sums that cancel, or hold
 * a few large products among small ones, can lose more of the result.  With an
 * fp32 c the sums keep fp32 precision throughout, and operand values are taken
 * as fp32 holds them: below 2^-133 they are lost, from 2^128 on (what the
 * quantization makes of magnitudes of 3.3e38 and more) they are infinite.  How a
 * product is cut into blocks, and so the order of its sum, depends on the sizes
 * of the whole batch; equal calls give equal bits.  k[i] = 0 gives zeros (or
 * leaves c).  Of Y = X W^T, the backward products take the same call: dX = dY W
 * with operands dY and W^T, and dW = dY^T X with operands dY^T and X^T.
 *
 * Every size lies in [0, MUON_F8_MAX_DIM] (MUON_ERR_UNSUPPORTED otherwise).  A
 * launch holds fewer than 2^24 blocks: a quantization whose matrices have that many
 * tiles of 128 x 128 is refused likewise, and so may be a product whose outputs have
 * that many of 16 x 64 (partial ones counted whole).  Pointers of empty operands are
 * not read.  workspace: at least muon_f8_workspace_bytes(batch) bytes, 256-byte
 * aligned.
 */
#define MUON_F8_BLOCK 128
#define MUON_F8_MAX_DIM 1048576

size_t muon_f8_workspace_bytes(int32_t batch);

int32_t muon_f8_quantize_batched(int32_t batch, const int64_t* rows, const int64_t* cols,
                                 const void* const* x, int32_t dtype, int32_t block_rows,
                                 void* const* q, void* const* s, void* const* qt, void* const* st,
                                 void* workspace, size_t workspace_bytes, void* stream);

int32_t muon_f8_matmul_batched(int32_t batch, const int64_t* m, const int64_t* n,
                               const int64_t* k, const void* const* a, const void* const* sa,
                               const void* const* b, const void* const* sb, void* const* c,
                               int32_t dtype, int32_t accumulate, void* workspace,
                               size_t workspace_bytes, void* stream);

/*
 * Tokens to the experts and back, around the products of an expert layer.  Token t
 * of `tokens` has top_k slots s = t * top_k + k, each with an expert's id; an id
 * outside [0, experts) drops the slot (padding, or an expert that is full).
 *
 * muon_moe_sort makes the plan that the other calls read, on the device: kept
 * slots by expert, those of one expert in the order of s.
 *   ids      tokens x top_k integers of id_bytes (4 or 8) bytes
 *   offsets  experts + 1: the sorted rows of expert e are offsets[e] .. offsets[e+1] - 1
 *   active   experts + 1: active[0] experts have rows, active[1 ..] are their ids,
 *            ascending, then -1
 *   rows     tokens x top_k: the sorted row of each slot, -1 for a dropped one
 *   slots    tokens x top_k: the slot of each sorted row, -1 behind the last
 *
 * With that plan (slots that are dropped, or whose row is not below y_rows or
 * out_rows, take no part: their weights and rows are not read, and nothing is
 * written for them):
 *   muon_moe_dispatch          out[rows[s]] = x[t]
 *   muon_moe_combine           out[t] = sum_k w[s] y[rows[s]]
 *   muon_moe_combine_backward  dy[rows[s]] = w[s] dout[t],
 *                              dw[s] = sum_c dout[t][c] y[rows[s]][c]  (0 if dropped)
 * Rows have `cols` elements of `dtype` (MUON_BF16 or MUON_FP32) and lie one after
 * the other; weights and their gradients are fp32.  Sums are fp32, rounded once:
 * combine's in the order of k; weights may be null there: 1, which is the
 * gradient of dispatch.  Rows behind the last sorted one are left as they were.
 * A token without kept slots gets zeros.
 *
 * tokens * top_k <= MUON_MOE_MAX_SLOTS, top_k in [1, MUON_MOE_MAX_TOP_K], experts in
 * [1, MUON_MOE_MAX_EXPERTS], cols <= MUON_F8_MAX_DIM (MUON_ERR_UNSUPPORTED beyond).
 * x, y, out, dout and dy are 16-byte aligned, the other arrays at their elements'
 * size.  No output may overlap another array of the call (rows of an output that do
 * are refused, and so are dw over w).
 */
#define MUON_MOE_MAX_EXPERTS 1024
#define MUON_MOE_MAX_TOP_K 64
#define MUON_MOE_MAX_SLOTS 16777215

/* Bytes of device workspace of muon_moe_sort; SIZE_MAX on invalid arguments.  Never
 * less for more slots or more experts: the workspace of the largest call serves all. */
size_t muon_moe_workspace_bytes(int64_t tokens, int32_t top_k, int32_t experts);

int32_t muon_moe_sort(int64_t tokens, int32_t top_k, int32_t experts, const void* ids,
                      int32_t id_bytes, int32_t* offsets, int32_t* active, int32_t* rows,
                      int32_t* slots, void* workspace, size_t workspace_bytes, void* stream);

int32_t muon_moe_dispatch(int64_t tokens, int32_t top_k, int64_t cols, const void* x,
                          const int32_t* rows, int64_t out_rows, void* out, int32_t dtype,
                          void* stream);

int32_t muon_moe_combine(int64_t tokens, int32_t top_k, int64_t cols, int64_t y_rows,
                         const void* y, const int32_t* rows, const float* weights, void* out,
                         int32_t dtype, void* stream);

int32_t muon_moe_combine_backward(int64_t tokens, int32_t top_k, int64_t cols, const void* dout,
                                  int64_t y_rows, const void* y, const int32_t* rows,
                                  const float* weights, void* dy, float* dweights, int32_t dtype,
                                  void* stream);

/*
 * Dropout over a ragged batch of tensors, for the rows between an expert's
 * products.  With t = p * 2^16 rounded to the nearest integer,
 *     out_ij = 0 if u_ij < t, else x_ij * 2^16 / (2^16 - t)
 * in fp32, rounded to out's type; t = 2^16 drops everything.  u_ij is 16 bits of
 * Philox 4x32 with 7 rounds, of the block with counter (j / 8, i, low and high half
 * of offset) and key (low and high half of seed): half j % 8 of the block's words
 * (the low half of a word first).  Nothing of it is stored: the gradient is the
 * same call on the gradients.  A dropped element is 0 whatever x_ij is.
 *   numel, dtype, out, out_dtype  as for muon_grad_scale_batched (out[i] may be
 *                 x[i], of the same type), numel[i] below 2^35
 *   rng           null, or device memory (8-byte aligned): seed and offset, read on
 *                 the stream in place of those in `params`, so that a captured call
 *                 takes new ones at every replay
 *   workspace     at least muon_grad_workspace_bytes() bytes, 256-byte aligned
 */
typedef struct {
  double p;        /* in [0, 1] */
  uint64_t seed;
  uint64_t offset; /* another mask for every call of one seed: a step's or layer's number */
} muon_dropout_params;

int32_t muon_dropout_batched(int32_t batch, const int64_t* numel, const void* const* x,
                             const int32_t* dtype, void* const* out, const int32_t* out_dtype,
                             const muon_dropout_params* params, const uint64_t* rng,
                             void* workspace, size_t workspace_bytes, void* stream);

/*
 * 4-bit weights with group scales, and their products with few rows: the expert
 * matrices as they serve single tokens.
 *
 * An operand holds `count` matrices of `rows` x `cols`, contracted over cols, in
 * tiles of 16 rows x 128 columns.  With RT = rows / 16 and KT = cols / 128, rounded up:
 *   q  count x RT x KT x 64 x 16 bytes: chunk 16 c + r of a tile holds columns
 *      32 i + 8 c + j (i < 4, j < 8) of its row r, OCP e2m1 codes (0, 0.5, 1, 1.5, 2, 3,
 *      4, 6; 8 more: negative), column 2 j' in the low half of byte 4 i + j'
 *   s  count x RT x (KT / 4 rounded up) x 16 x 16 bytes: row r's 16 groups of 32
 *      columns of four tiles, byte e + 127 for the scale 2^e, 255: NaN
 * Columns past the matrix are zeros; rows past it, and groups past the last
 * tile, have code 0 and scale 127.  A value stands for code * 2^e.
 *
 * muon_f4_quantize forms the operand of count matrices w[i] (rows x cols of the
 * operand, row-major, contiguous, `dtype`; with transpose = 1 cols x rows, each
 * transposed on the way).  2^e is the smallest power of two, from 2^-125 to 2^125,
 * with the group's largest magnitude at most 6 * 2^e; codes are rounded to nearest
 * even, and saturate (above 6 * 2^125 only).  A group with an infinity or NaN is NaN.
 *
 * muon_f4_matmul: y[p] = x[p] W_e^T for the rows p of expert e, offsets[e] <= p <
 * offsets[e+1] and p < m; rows of y that no expert has are left as they were.
 *   x        x_rows x cols, bf16, row-major, contiguous
 *   offsets, active  of muon_moe_sort with experts = count; both null: matrix 0 (count
 *            must be 1) takes all m rows
 *   slots    null: row p is x's row p (x_rows >= m); else of muon_moe_sort (m entries
 *            at least): row p is x's row slots[p] / top_k, the token's own, which
 *            saves the dispatch.  Needs offsets and active.
 *   y        m x rows, `dtype` (MUON_BF16 or MUON_FP32); may not overlap x
 * Products are exact, sums fp32 in an order that the sizes fix, rounded once.
 * Scale bytes are to lie in [2, 252] or be 255.
 * Meant for up to some 64 rows an expert, where the weights' bytes bound it.  Where m is
 * at most 16 min(m, count), an expert's weights are read again for every 16 of its
 * rows, else for every 64: rows that all fall on a few of many experts take longer
 * than with an operand of those experts alone.  muon_f8_matmul_batched is for many
 * rows.
 *
 * count in [1, MUON_MOE_MAX_EXPERTS], rows and cols in [0, MUON_F8_MAX_DIM], m and
 * x_rows at most MUON_MOE_MAX_SLOTS, fewer than 2^28 tiles (MUON_ERR_UNSUPPORTED
 * beyond).  q, s, x, y: 16-byte aligned.
 */
#define MUON_F4_GROUP 32

/* Bytes of device workspace of muon_f4_quantize; SIZE_MAX on invalid arguments. */
size_t muon_f4_workspace_bytes(int32_t count);

int32_t muon_f4_quantize(int32_t count, int64_t rows, int64_t cols, const void* const* w,
                         int32_t dtype, int32_t transpose, void* q, void* s, void* workspace,
                         size_t workspace_bytes, void* stream);

int32_t muon_f4_matmul(int32_t count, int64_t rows, int64_t cols, const void* q, const void* s,
                       int64_t m, const void* x, int64_t x_rows, const int32_t* offsets,
                       const int32_t* active, const int32_t* slots, int32_t top_k, void* y,
                       int32_t dtype, void* stream);

/* Kernels of the step, and the momentum copies of a step with the momentum in
 * host memory, for per-kernel timing. */
typedef enum {
  MUON_K_PREPARE = 0,   /* momentum, U into the iterate (short side first), sums of squares */
  MUON_K_NORM = 1,      /* 1 / (||U||_F + eps) per matrix */
  MUON_K_GRAM = 2,      /* A = X X^T */
  MUON_K_POLY = 3,      /* B = b A + c A^2 */
  MUON_K_PROD = 4,      /* X <- a X + B X, except the first and (bf16) the last */
  MUON_K_FINISH = 5,    /* W update, or the output copy (fp32, or no Newton-Schulz steps) */
  MUON_K_ADAMW = 6,     /* muon_adamw_batched */
  MUON_K_PROD_FINISH = 7, /* bf16: the last X <- a X + B X, writing W (or the output) itself */
  MUON_K_PROD_FIRST = 8,  /* the first X <- a X + B X (its iterate is U, scaled as it is stored) */
  MUON_K_QUANT8 = 9,      /* e4m3 steps: the block-scaled e4m3 copies of X, A and B */
  MUON_K_GRAM8 = 10,      /* e4m3 steps: A = X X^T */
  MUON_K_POLY8 = 11,      /* e4m3 steps: B = b A + c A^2 */
  MUON_K_PROD8 = 12,      /* e4m3 steps: X <- a X + B X */
  MUON_K_MOM_IN = 13,     /* momentum_host: one chunk's momentum copied to the device (DMA) */
  MUON_K_MOM_OUT = 14,    /* momentum_host: one chunk's momentum copied back to the host (DMA) */
  MUON_K_GRAD_NORM = 15,  /* the global gradient norm */
  MUON_K_GRAD_SCALE = 16, /* gradients times a factor */
  MUON_K_F8_QUANTIZE = 17, /* muon_f8_quantize_batched */
  MUON_K_F8_PROD = 18,    /* muon_f8_matmul_batched */
  MUON_K_MOE_SORT = 19,   /* muon_moe_sort */
  MUON_K_MOE_DISPATCH = 20, /* muon_moe_dispatch */
  MUON_K_MOE_COMBINE = 21, /* muon_moe_combine */
  MUON_K_MOE_BACKWARD = 22, /* muon_moe_combine_backward */
  MUON_K_DROPOUT = 23,    /* muon_dropout_batched */
  MUON_K_F4_QUANTIZE = 24, /* muon_f4_quantize */
  MUON_K_F4_PROD = 25,    /* muon_f4_matmul */
  MUON_K_COUNT = 26
} muon_kernel;

/*
 * Per-kernel timing, off by default.  While enabled (process-wide), every call
 * records a pair of HIP events on its stream around each kernel launch (and, with
 * the momentum in host memory, on the copy streams around each chunk's copies).
 * muon_timing_read waits for the recorded events, adds their elapsed times to
 * per-kernel totals, and returns the total milliseconds and the number of
 * launches of `kernel` since the last muon_timing_reset.  Returns MUON_OK,
 * MUON_ERR_INVALID_ARG (bad kernel id or null output) or MUON_ERR_HIP.
 */
int32_t muon_timing_enable(int32_t enable);
int32_t muon_timing_read(int32_t kernel, double* total_ms, int64_t* launches);
int32_t muon_timing_reset(void);

/*
 * Measurement aid: a plain HBM stream with the access pattern of the momentum
 * pass (16-byte vectors, lane-contiguous, every load of a block issued before
 * its first store), for the read + write ceiling that the bandwidth-bound
 * kernels are held against.  Output k receives input k % n_in, except that
 * with two inputs and one output it receives their bitwise XOR; `bytes` bytes
 * each, with the nontemporal hint when `nontemporal` is 1.
 *   n_in, n_out  1 or 2
 *   in, out      host arrays of 16-byte aligned device pointers
 *   bytes        a multiple of 16384 (0: no-op)
 * Returns MUON_OK, MUON_ERR_INVALID_ARG (nothing launched) or MUON_ERR_HIP
 * (launch failure; muon_last_error_detail() is not set by this call).
 */
int32_t muon_hbm_stream(int32_t n_in, const void* const* in, int32_t n_out, void* const* out,
                        size_t bytes, int32_t nontemporal, void* stream);

/* Static string naming a status code. */
const char* muon_status_string(int32_t status);

/* Detail of the last error returned on this thread ("" if none).  Valid until the
 * next call on this thread. */
const char* muon_last_error_detail(void);

#ifdef __cplusplus
}
#endif

#endif /* MUON_MI355X_H */
