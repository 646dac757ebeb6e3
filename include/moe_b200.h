/*
 * moe_b200.h -- C ABI of the B200 (sm_100a) forward pass of one capacity-limited
 * Mixture-of-Experts layer.
 *
 * The layer (sources are the pages' titles and sections):
 *   1. router: softmax over the E router logits of each token, keep the k largest
 *      ("Dynamic Token Routing AI", How it works: a gating network scores each token and
 *      picks experts);
 *   2. capacity: every expert has K = floor(C * T * k / E) slots (at most T); an expert that
 *      receives more than K (token, expert) pairs keeps the K with the highest router weight
 *      and drops the rest ("Expert Networks > Worked Example: Expert Specialization", capacity
 *      paragraph: K = 1.25 * (8/4) rounded down to 2, the lowest-confidence token is dropped;
 *      "Some Tokens Do Not Get In", "Why there is a buffer": t*k slots, fixed buffer per
 *      expert);
 *   3. expert FFN on the kept pairs: h = W1 x + b1, a = SiLU(h), y = W2 a + b2 (worked
 *      example, trace of token 0);
 *   4. combine: out = x + sum_j w_j * y_j over the token's kept pairs; a token whose pairs
 *      were all dropped leaves the layer exactly as it entered (worked example, token 4;
 *      "Some Tokens Do Not Get In", "Past the edge"; the k outputs of a token are summed back
 *      in token order as in the fused-MoE dataflow diagram's moe_sum step).
 *
 * Conventions for every call:
 *   - All pointers except `p` and the out-parameters of the host-only queries are DEVICE
 *     pointers owned by the caller.  The library never allocates device memory: scratch comes
 *     from the caller's workspace `ws` of `ws_bytes` bytes (size from moe_workspace_size,
 *     256-byte aligned).  A workspace serves one call at a time: calls that share one are ordered
 *     (on one stream, or by events); calls that may overlap, on other streams or in graphs replayed
 *     at once, take a workspace each.
 *   - Every compute call is asynchronous on `stream` (a cudaStream_t; NULL = legacy default
 *     stream) and performs no host synchronisation.  Kernels are launched with programmatic
 *     stream serialization: a kernel may be scheduled while the preceding work on `stream`
 *     drains, but it waits for that work to complete (griddepcontrol.wait) before it reads or
 *     writes any memory that this work may touch, so stream order is kept for every input and
 *     output.
 *   - Host-checkable errors (bad shapes, k > E, negative or NaN capacity factor, null or
 *     misaligned pointers, workspace too small, unsupported shape) return a non-zero status
 *     BEFORE anything is launched; outputs are then untouched.
 *   - Errors the device detects (a pipeline wait that ran out, an index out of range) are
 *     recorded in a status word at the start of `ws`; read it with moe_get_device_status.
 *     The calls never clear it (the first error stays; a timeout replaces a bad index, as it
 *     leaves work out), so clear it once with moe_reset_device_status after allocating a
 *     workspace, and again after handling an error.  A recorded bad index does not change what
 *     later calls compute; after a timeout outputs are undefined until the word is cleared.
 *   - Layouts are row-major and dense.  Pair p = t * k + j addresses the j-th expert of token
 *     t (j = 0 is the largest logit).  W1 is [E, d_ff, d_model] and W2 is [E, d_model, d_ff]
 *     ("out x in", so h = W1 x).  b1 is [E, d_ff] and b2 is [E, d_model], float32 always.
 *   - dtype MOE_BF16: x, W1, W2, out and expert outputs are bfloat16, accumulation is float32
 *     on the tensor cores; d_model and d_ff must be multiples of 64, and bf16 pointers and the
 *     biases 16-byte aligned.  dtype MOE_F32: everything float32 on CUDA cores (small layers).
 */
#ifndef MOE_B200_H
#define MOE_B200_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = 1,  /* bad shape, pointer, alignment or capacity factor */
    MOE_ERR_UNSUPPORTED = 2,  /* well-formed problem this build does not run */
    MOE_ERR_WORKSPACE = 3,    /* workspace null or smaller than moe_workspace_size */
    MOE_ERR_CUDA = 4,         /* a CUDA runtime call or launch failed */
    MOE_ERR_DEVICE = 5        /* the device status word holds an error */
} moe_status;

typedef enum { MOE_F32 = 0, MOE_BF16 = 1 } moe_dtype;

/* Device status codes (moe_get_device_status). */
#define MOE_DEV_OK 0
#define MOE_DEV_TIMEOUT 1      /* a pipeline wait in a kernel gave up after about 2 s */
#define MOE_DEV_BAD_INDEX 2    /* an index read from an input was out of range */

typedef struct {
    int32_t T;                /* tokens, >= 0 */
    int32_t d_model;          /* model width, >= 1 */
    int32_t d_ff;             /* expert hidden width, >= 1 */
    int32_t E;                /* experts, 1..1024 */
    int32_t k;                /* experts per token, 1..min(E, 32) */
    float capacity_factor;    /* C >= 0; +INFINITY = dropless (K = T) */
    int32_t dtype;            /* moe_dtype */
    uint32_t flags;           /* MOE_FLAG_* below; other bits must be 0 */
} moe_problem;

/* Routing-policy variants (flags of moe_problem).  Default (0): softmax weights over all E,
 * not renormalised; an overflowing expert keeps its K highest-weight pairs.
 *   MOE_FLAG_RENORMALIZE: each token's k weights are divided by their sum (formed in fp32 over
 *     j = 0..k-1, one correctly rounded division each); the renormalised weights are the ones
 *     reported, used for drop priority and in the combine.
 *   MOE_FLAG_ARRIVAL_ORDER: an overflowing expert keeps the first K pairs in token order, the
 *     reading of "Some Tokens Do Not Get In", "Past the edge" (each expert's fixed buffer fills
 *     first come, first served, and later tokens are turned away), instead of the highest
 *     weights. */
#define MOE_FLAG_RENORMALIZE 1u
#define MOE_FLAG_ARRIVAL_ORDER 2u
/* Expert variant: gated FFN, after the fused-MoE dataflow diagram (GEMM 1 writes gate and up
 * halves, "SiLU x mul" combines them, GEMM 2 follows).  W1 is then [E, 2*d_ff, d_model] (rows
 * [0, d_ff) the gate, [d_ff, 2*d_ff) the up projection) and b1 [E, 2*d_ff]; the expert computes
 * a = SiLU(W1_gate x + b1_gate) * (W1_up x + b1_up), y = W2 a + b2.  bf16 needs d_ff % 128 == 0. */
#define MOE_FLAG_GATED 4u
/* Router weights prepared once: moe_forward skips splitting Wr into its two bfloat16 terms and
 * reads the terms moe_prepare_router left in the workspace (bf16 batches above 1024 tokens; the
 * other paths use Wr directly and ignore the flag).  The caller prepares again after Wr changes
 * or after the workspace was used for another problem; with stale terms the logits are wrong. */
#define MOE_FLAG_ROUTER_PREPARED 8u

/* 4-bit weights [E, N, K] with group scales (moe_quantize_packed makes them; any program may).
 * Columns are cut into groups of `group` (32, 64 or 128; the last group of a row may be short).
 *   q [E, N, 16 ceil(K / 128)] uint32: word 4 t + j of a row's 128-column chunk c holds columns
 *     128 c + 32 j + 8 t + i, i = 0..7 (t, j in 0..3), column i as the nibble at bit
 *     4 (4 (i % 2) + i / 2); columns past K hold 8.
 *   scale, zero [E, ceil(K / group), N] bfloat16; zero may be NULL (no offsets).
 * Value of column k of row n: scale * (nibble - 8) + zero, of group k / group.
 * All three 16-byte aligned. */
typedef struct {
    const void* q;
    const void* scale;
    const void* zero;
    int32_t group;
} moe_w4;

/* The layer norm in front of a block: parameters [d_model] float32, and where its output
 * y [T, d_model] (x's dtype), mean and rstd [T] float32 go (kept for the backward pass). */
typedef struct {
    const float* gamma;
    const float* beta;
    float eps;
    void* y;
    float* mean;
    float* rstd;
} moe_norm;

/* Host only.  Per-expert capacity K = min(T, floor(C * T * k / E)) evaluated in double
 * (worked example, capacity paragraph; generalised to k slots per token as in "Some Tokens Do
 * Not Get In").  Returns MOE_ERR_INVALID_ARG for a malformed problem. */
moe_status moe_capacity(const moe_problem* p, int64_t* K);

/* Host only.  Workspace bytes needed by any call below for problem p (the largest, moe_forward,
 * decides).  A workspace of this size serves every call for that problem. */
moe_status moe_workspace_size(const moe_problem* p, size_t* bytes);

/* Router + capacity (steps 1-2).
 *   logits [T, E] float32 in;  ids [T*k] int32, w [T*k] float32 (softmax weight, not
 *   renormalised), slot [T*k] int32 (rank of t among the expert's kept tokens in ascending
 *   token order, -1 if dropped), drop [T*k] uint8 (1 = dropped), counts [2E] int32 (pairs
 *   received per expert, then pairs kept per expert).
 * Drop priority inside one expert: weight descending, then token index ascending.  Top-k ties
 * in the logits go to the lower expert index.  The softmax uses a fixed summation order and
 * its own exp, so ids, w, slot and drop are bit-for-bit functions of the logits.  NaN logits
 * are a precondition violation (result unspecified). */
moe_status moe_route(const moe_problem* p, const float* logits, int32_t* ids, float* w,
                     int32_t* slot, uint8_t* drop, int32_t* counts, void* ws, size_t ws_bytes,
                     void* stream);

/* Capacity-limited dispatch of a given routing, steps 2-3 without the router ("Expert Networks >
 * Worked Example: Expert Specialization", capacity paragraph; "Some Tokens Do Not Get In",
 * "Past the edge"): for routings formed elsewhere, and for the owner of a set of experts under
 * expert parallelism, which selects among candidates gathered from every rank.
 *   p: T, E, k and flags (MOE_FLAG_ARRIVAL_ORDER keeps an overflowing expert's first K pairs in
 *   token order; MOE_FLAG_RENORMALIZE is ignored: the weights are given); capacity_factor,
 *   d_model and d_ff size the workspace only (moe_workspace_size with the same p).
 *   K >= 0: the capacity of every expert, given explicitly (it need not be C*T*k/E of p).
 *   ids [T*k] int32 in: pair p = t*k + j goes to expert ids[p]; a token's k ids must be
 *   distinct (as a top-k gives them).  w [T*k] float32 in: its weight, >= +0 and finite.
 *   slot, drop [T*k] and counts [2E] out, as moe_route gives them for the same ids and w.
 *   offsets [E+1] int32 out (nullable): exclusive prefix of the kept counts.
 *   rowtok (nullable; needs offsets) int32 out, min(T*k, E*K) entries: rowtok[offsets[e] +
 *   slot] = token t of that kept pair.
 * Errors: MOE_ERR_INVALID_ARG for K < 0 or missing buffers; device-detected bad ids (outside
 * [0, E)) or weights (negative, -0, NaN) go to the status word as MOE_DEV_BAD_INDEX. */
moe_status moe_capacity_dispatch(const moe_problem* p, long long K, const int32_t* ids,
                                 const float* w, int32_t* slot, uint8_t* drop, int32_t* counts,
                                 int32_t* offsets, int32_t* rowtok, void* ws, size_t ws_bytes,
                                 void* stream);

/* Splits Wr [d_model, E] float32 into the two bfloat16 terms the tensor-core router reads (hi =
 * bf16(w), mid = bf16(w - hi)) and keeps them in ws, for moe_forward calls with
 * MOE_FLAG_ROUTER_PREPARED on the same p and ws.  Weights are constant during inference, so the
 * split need not be repeated per call.  A no-op for problems that do not use the tensor-core
 * router (fp32, or at most 1024 tokens). */
moe_status moe_prepare_router(const moe_problem* p, const float* Wr, void* ws, size_t ws_bytes,
                              void* stream);

/* Router logits alone, step 1's first half ("Dynamic Token Routing AI", How it works: the gating
 * network scores every token): logits [T, E] float32 = x Wr + br, with moe_forward's kernels, so
 * the values equal its logits_out bit for bit.  x [T, d_model] in p's dtype (16-byte aligned for
 * bf16), Wr [d_model, E] float32, br [E] float32 or NULL.  bf16 batches above 1024 tokens need
 * d_model a multiple of 64 (else MOE_ERR_UNSUPPORTED). */
moe_status moe_router_logits(const moe_problem* p, const void* x, const float* Wr,
                             const float* br, float* logits, void* ws, size_t ws_bytes,
                             void* stream);

/* Dispatch layout from a routing.
 *   ids, slot [T*k] in;  offsets [E+1] int32 out (exclusive prefix of kept counts);
 *   rowtok [min(T*k, E*K)] int32 out: rowtok[offsets[e] + slot] = token of that kept pair.
 *   x_perm (nullable) [rows, d_model] in x's dtype: when given, receives x[rowtok[r]] in row
 *   r (the permuted token buffer; the FFN does not need it, it gathers rows itself). */
moe_status moe_dispatch(const moe_problem* p, const int32_t* ids, const int32_t* slot,
                        int32_t* offsets, int32_t* rowtok, const void* x, void* x_perm,
                        void* ws, size_t ws_bytes, void* stream);

/* Expert FFN over the kept rows (step 3): for each expert e and row r in
 * [offsets[e], offsets[e+1]): Y[r] = W2[e] SiLU(W1[e] x[rowtok[r]] + b1[e]) + b2[e].
 * The token gather is folded into the first GEMM's operand load; nothing is materialised but
 * the hidden activations (in ws, x's dtype).  Y is [min(T*k, E*K), d_model] in x's dtype.
 * b1, b2 may be NULL (zero bias).
 * The kernels check offsets on the device: offsets[0] = 0, non-decreasing, offsets[E] <=
 * min(T*k, E*K).  If not, nothing is written to Y or H and MOE_DEV_BAD_INDEX is recorded.  A
 * rowtok entry outside [0, T) is recorded the same way and its row is computed from zeros. */
moe_status moe_expert_ffn(const moe_problem* p, const void* x, const int32_t* offsets,
                          const int32_t* rowtok, const void* W1, const float* b1,
                          const void* W2, const float* b2, void* Y, void* ws, size_t ws_bytes,
                          void* stream);

/* Combine (step 4): out[t] = x[t] + sum over kept j (ascending) of w[t*k+j] * Y[offsets[id]
 * + slot], accumulated in float32 and rounded once; out[t] = x[t] bit for bit when no pair of
 * t is kept.  out must not alias x or Y.  Y has min(T*k, E*K) rows.
 *   ws (nullable, 256-byte aligned, ws_bytes >= 256): only its status word is used.  A kept
 *   pair whose expert id is out of range, or whose row offsets[id] + slot lies outside
 *   [offsets[id], offsets[id+1]) or outside Y, is skipped (its term is left out) and recorded
 *   as MOE_DEV_BAD_INDEX in ws's status word; with ws = NULL it is skipped silently. */
moe_status moe_combine(const moe_problem* p, const void* x, const void* Y, const float* w,
                       const int32_t* ids, const int32_t* slot, const int32_t* offsets,
                       void* out, void* ws, size_t ws_bytes, void* stream);

/* The whole layer: logits = x Wr + br (Wr [d_model, E] float32, br [E] float32 or NULL), then
 * the four steps.  out [T, d_model] in x's dtype.  Optional outputs (NULL = keep in ws):
 * logits_out [T, E], ids_out, w_out, slot_out [T*k], drop_out [T*k], counts_out [2E].
 * With dtype MOE_BF16 the logits come from the tensor cores with Wr split into two bfloat16 terms
 * (hi = bf16(Wr), mid = bf16(Wr - hi); the remainder is below 2^-18 |Wr|) and float32
 * accumulation; the routing of those logits is bit for bit the routing moe_route gives for them
 * (logits_out exports them). */
moe_status moe_forward(const moe_problem* p, const void* x, const float* Wr, const float* br,
                       const void* W1, const float* b1, const void* W2, const float* b2,
                       void* out, float* logits_out, int32_t* ids_out, float* w_out,
                       int32_t* slot_out, uint8_t* drop_out, int32_t* counts_out, void* ws,
                       size_t ws_bytes, void* stream);

/* ---- 4-bit expert weights ------------------------------------------------------------------
 * Quantises W [E, N, K] (dtype MOE_BF16 or MOE_F32, dense, 16-byte aligned; values below 2^126 in
 * magnitude) to the format of moe_w4.  A group that holds a NaN or an infinity gets a scale that is
 * not finite and reads back as values that are not finite; the other groups do not see it.
 * Per group, zero = NULL: scale = max|w| / 7; else scale = (max - min) / 15 and zero = min + 8 scale.
 * Both are rounded to bfloat16 first (the differences, products with the float32 reciprocal of 7 or
 * 15, and sums in float32), then nibble - 8 = round-half-even((w - zero) / scale), clamped to
 * [-8, 7]; 0 where scale = 0.
 * K must be a multiple of 64 and at most 2^30, N at most 2097120 and E at most 65535 (else
 * MOE_ERR_UNSUPPORTED). */
moe_status moe_quantize_packed(const void* W, int32_t dtype, int32_t E, int32_t N, int32_t K,
                           int32_t group, void* q, void* scale, void* zero, void* stream);

/* Reads 4-bit weights back: W [E, N, K] bfloat16, each value formed in float32 and rounded once.
 * The same limits as moe_quantize_packed. */
moe_status moe_dequantize_packed(const moe_w4* w, int32_t E, int32_t N, int32_t K, void* W,
                             void* stream);

/* Host only.  Workspace bytes for moe_expert_ffn_packed and moe_forward_block with 4-bit weights
 * (at least moe_workspace_size, which suffices for the other calls). */
moe_status moe_workspace_size_packed(const moe_problem* p, size_t* bytes);

/* moe_expert_ffn over 4-bit weights: W1 is [E, d_ff, d_model] ([E, 2 d_ff, d_model] with
 * MOE_FLAG_GATED), W2 [E, d_model, d_ff]; their groups may differ.  p's dtype is MOE_BF16 (else
 * MOE_ERR_UNSUPPORTED; so are weights of over 2097120 rows an expert or 2^31 - 1 in all), with
 * moe_expert_ffn's rules for widths, alignment, offsets and rowtok; rows of Y behind offsets[E] are
 * left as they were.
 * Few rows per expert (min(T k, E K) <= 64 E): the products read the 4-bit weights and form
 * sum_k (nibble - 8) x_k per group, of exact products added in float32, before the scale; b1, b2
 * nullable.  More rows: each weight is first read back to bfloat16 (one rounding per value) into the
 * workspace, for the grouped tensor-core GEMM.  The hidden activations are kept in bfloat16 either
 * way. */
moe_status moe_expert_ffn_packed(const moe_problem* p, const void* x, const int32_t* offsets,
                             const int32_t* rowtok, const moe_w4* W1, const float* b1,
                             const moe_w4* W2, const float* b2, void* Y, void* ws,
                             size_t ws_bytes, void* stream);

/* ---- Layer norm ----------------------------------------------------------------------------
 * y = gamma (x - mean) rstd + beta per token, rstd = 1 / sqrt(variance + eps), the variance over
 * d_model without bias correction.  x, y [T, d_model] in p's dtype, any d_model; gamma, beta
 * [d_model] float32; mean, rstd [T] float32 out.  eps >= 0 and finite (with eps = 0 the y of a row of
 * equal values is undefined: the rounding of its mean decides; where a float32 variance overflows but
 * the row's sum does not, rstd is 0 and y is beta); d_model at most 2^30.  y must not alias x.
 * Statistics are float32, y is rounded once. */
moe_status moe_layer_norm(const moe_problem* p, const void* x, const float* gamma,
                          const float* beta, float eps, void* y, float* mean, float* rstd,
                          void* stream);

/* Its backward pass from dy, with the forward's x, mean and rstd: dx [T, d_model] in p's dtype,
 * dgamma and dbeta [d_model] float32, written (not added to).  dres (nullable, [T, d_model], p's
 * dtype) is added to dx before its one rounding: the gradient that reaches x past the norm, over
 * the residual.  dx must not alias an input.  Results do not depend on scheduling. */
moe_status moe_layer_norm_backward(const moe_problem* p, const void* dy, const void* x,
                                   const float* gamma, const float* mean, const float* rstd,
                                   const void* dres, void* dx, float* dgamma, float* dbeta,
                                   void* ws, size_t ws_bytes, void* stream);

/* ---- Router training -----------------------------------------------------------------------
 * Losses of a routing over the n tokens that mask [T] (nullable) leaves (0 leaves a token out;
 * its logits and ids are not used and may hold anything).  With p_t = softmax(logits_t):
 *   counts [E+1] int32: pairs (t, j) with ids[t k + j] = e, then n (before any capacity);
 *   probs [E] float32: P_e = sum_t p_te / n;
 *   losses [2] float32: E sum_e counts_e / (n k) P_e (load balance), sum_t lse_t^2 / n (z-loss,
 *     lse_t = log sum_e exp logits_te).
 * n = 0 gives zeros.  A token's logits hold at least one finite value, no NaN and no +infinity;
 * -infinity is an expert it cannot take.  An id outside [0, E) is not counted and recorded as
 * MOE_DEV_BAD_INDEX.  Results do not depend on scheduling. */
moe_status moe_balance_loss(const moe_problem* p, const float* logits, const int32_t* ids,
                            const uint8_t* mask, float* losses, int32_t* counts, float* probs,
                            void* ws, size_t ws_bytes, void* stream);

/* Gradient with respect to the logits, dlogits [T, E] float32 (written; zero rows for tokens the
 * mask leaves out):  of grad_losses[0] losses[0] + grad_losses[1] losses[1] (grad_losses [2]
 * float32 on the device, with counts as moe_balance_loss gives them, or summed over the ranks of
 * a group; NULL leaves this part out), plus that of the k routing weights w_tj, given their
 * gradient grad_w [T k] float32 (NULL leaves it out; ids is read only with it, and is held
 * constant).  MOE_FLAG_RENORMALIZE: the weights are the renormalised ones, a softmax over the k
 * named logits wherever these lie in the row (named experts of -infinity have weight 0; where all
 * are, this part is 0).  At least one of the two is given.  An id outside [0, E) is left out and
 * recorded as MOE_DEV_BAD_INDEX; an id named twice by a token adds up.  dlogits must not alias
 * logits. */
moe_status moe_route_backward(const moe_problem* p, const float* logits, const int32_t* ids,
                              const uint8_t* mask, const int32_t* counts,
                              const float* grad_losses, const float* grad_w, float* dlogits,
                              void* ws, size_t ws_bytes, void* stream);

/* moe_forward as a block of a model: with norm (nullable) the router and the experts read
 * norm(x) and the combine adds onto x, out = x + sum_j w_j FFN_j(norm(x)); with Q1 and Q2 (both,
 * and W1 = W2 = NULL) the experts' weights are 4-bit, and ws_bytes must hold
 * moe_workspace_size_packed.  Otherwise as moe_forward, bit for bit with neither. */
moe_status moe_forward_block(const moe_problem* p, const void* x, const moe_norm* norm,
                             const float* Wr, const float* br, const void* W1, const void* W2,
                             const moe_w4* Q1, const moe_w4* Q2, const float* b1,
                             const float* b2, void* out, float* logits_out, int32_t* ids_out,
                             float* w_out, int32_t* slot_out, uint8_t* drop_out,
                             int32_t* counts_out, void* ws, size_t ws_bytes, void* stream);

/* Profiling aid, host only, per calling thread.  With n >= MOE_STAGE_EVENTS, moe_forward and
 * moe_forward_block record events[0..6] (cudaEvent_t handles owned by the caller) on their stream at:
 * entry, after the norm (if any) and the router logits, after softmax/top-k, after capacity
 * selection and dispatch, after the first expert GEMM, after the second expert GEMM (each with the
 * reading back of its 4-bit weights, if any), after the combine.  n = 0 (or events NULL) turns it
 * off.  Recording adds no synchronisation; the handles must outlive the calls that use them. */
#define MOE_STAGE_EVENTS 7
moe_status moe_set_stage_events(void* const* events, int32_t n);

/* moe_route without a workspace, for callers that cannot allocate device memory: plug-ins of an
 * inference engine that owns all device memory and gives its plug-ins no allocator, and serving
 * loops that may not call cudaMalloc/cudaFree on the request path (an allocation can
 * synchronise the device).  The source pages describe no such call; it is a deployment aid.
 *   Same arguments, outputs and results as moe_route (bit for bit), minus ws/ws_bytes.  The
 *   router/capacity scratch lives in one fixed 8 MiB array of device memory per GPU, part of the
 *   library image and held by every GPU that loads the library until the process exits.  Needs
 *   256 + 4*E*2049 + 4*E*T bytes (each part rounded up to 256; above T = 262144 tokens also
 *   8*E*ceil(T/32) for the selection's token bitmaps); larger problems get MOE_ERR_WORKSPACE
 *   before anything is launched (T=16384 with E=64 fits; T=65536 with E=128 does not).
 *   The first call in a CUDA context (for runtime-API callers: the first call on a device) looks
 *   up the array's device address in that context and caches it.  The cached address dies with
 *   its context: do not call it across a cudaDeviceReset of that device.
 *   The status word lives in the array too: each call clears it when it starts, and
 *   moe_get_device_status(NULL, 0, stream, &code) reads it (MOE_DEV_BAD_INDEX for an id out of
 *   range).
 *   Every call on a device shares the one array: calls that overlap on the GPU (other streams,
 *   other host threads) race and corrupt each other's results; serialise them.  Nothing is
 *   allocated, and no allocating routine is called. */
moe_status moe_route_static(const moe_problem* p, const float* logits, int32_t* ids, float* w,
                            int32_t* slot, uint8_t* drop, int32_t* counts, void* stream);

/* Failure-detection self-test: launches one kernel that waits on a pipeline barrier nothing
 * ever arrives on, using the same bounded wait as the layer's kernels but with a limit of
 * `limit_us` microseconds (1..10^7).  The wait gives up, records MOE_DEV_TIMEOUT in the status
 * word of `ws` and the kernel returns; the GPU context stays usable.  Asynchronous on `stream`;
 * read the result with moe_get_device_status. */
moe_status moe_selftest_wait_timeout(void* ws, size_t ws_bytes, int32_t limit_us, void* stream);

/* Reads the device status word of `ws` (synchronises `stream`).  ws = NULL reads the status word
 * of moe_route_static's fixed scratch on the current device, which that call clears when it
 * starts: it holds the result of the latest moe_route_static call there. */
moe_status moe_get_device_status(const void* ws, size_t ws_bytes, void* stream, int32_t* code);

/* Clears the device status word of `ws` (asynchronous on `stream`); ws = NULL: the status word of
 * moe_route_static's scratch on the current device. */
moe_status moe_reset_device_status(void* ws, size_t ws_bytes, void* stream);

/* Kernel launches made by the most recent successful compute call on this host thread. */
int32_t moe_last_launch_count(void);

/* Static, never NULL. */
const char* moe_status_string(moe_status s);

#ifdef __cplusplus
}
#endif

#endif /* MOE_B200_H */
