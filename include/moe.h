/*
 * moe.h - C ABI of the single-GPU fine-grained Mixture-of-Experts FFN layer
 * forward for AMD Instinct MI355X (gfx950).
 *
 * The layer has five steps, one entry point each:
 *   moe_route      gate scores, softmax, top-k, renormalised weights
 *   moe_dispatch   expert histogram, offsets, stable permutation, row gather
 *                  (moe_dispatch_capped: the same with each expert's capacity enforced)
 *   moe_expert_ffn grouped Linear -> erf-GeLU -> Linear over ragged segments
 *                  (plus the optional always-on shared expert; moe_expert_ffn_gather:
 *                  the same reading the token rows through perm, no xs copy)
 *   moe_combine    weighted sum of each token's k expert rows (+ shared row)
 *   moe_load_stats capacity, overflow / drops, skew, Gini, stragglers
 * around it, for a whole decoder block and for gated experts:
 *   moe_norm, moe_norm_residual  norm before the block; norm, gate, scale and
 *                  residual behind it (with the next block's norm)
 *   moe_route_grouped  sigmoid / softmax scores, choice bias, groups, top-k
 *   moe_linear, moe_linear_grouped  product with bias, activation or gate, and
 *                  residual; grouped: over the experts' segments
 * for a decode step:
 *   moe_layer_few  the whole layer for up to 64 tokens in two or three launches
 * the same products in 8-bit floating point:
 *   moe_quantize, moe_quantize_weight  rows and weights to e4m3 with block scales
 *   moe_linear_fp8, moe_linear_grouped_fp8  products of such operands
 * and, after the layer, the routing-bias feedback of the next step:
 *   moe_bias_update dynamic bias B from the expert counts, load fractions f_i
 *   (the mean router probabilities P_i are an optional output of moe_route)
 *
 * Sources of the method (three web pages; cited by title and section):
 *   [K3]   "hncyxsy.com Kimi K3 fine-grained MoE" article: router listing
 *          (FineGrainedMoERouter), the dispatch / local expert FFN / combine
 *          flow, the shared expert, the FFN cost equation.
 *   [DIAG] "Kimi K3 专家路由不均衡诊断" (bjdmk.com.cn): section 3 diagnostics
 *          module (MoERouteDiagnostics) and section 4.2 (biased score).
 *   [BLOG] "lpqz.cn MoE engineering blog": section 3.1 (expert = two Linear
 *          layers with GeLU; dispatcher with one shared buffer).
 *
 * Conventions for every call:
 *   - All tensor pointers are DEVICE memory owned by the caller, row-major and
 *     contiguous, 16-byte aligned. The library never allocates, frees or keeps
 *     a pointer past the call. Scratch memory comes from a caller-provided
 *     workspace whose size the *_workspace_bytes queries return.
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream). Every
 *     call only enqueues work on it and returns; there is no host
 *     synchronisation, so device-resident results (e.g. offsets) feed the next
 *     call directly. Calls keep no global state and are re-entrant.
 *   - Return value: MOE_OK (0) or a negative moe_status. Arguments are
 *     validated on the host before any HIP call; on error nothing is
 *     enqueued. A failed launch returns MOE_ERR_HIP. A row or weight tensor
 *     (x, wg, xs, w1, w2, ws1, ws2, ys, ysh, out) or workspace whose address
 *     is not a multiple of 16 returns MOE_ERR_INVALID_ARG.
 *   - dtype: MOE_F32 (fp32 activations, weights, arithmetic) or MOE_BF16
 *     (bf16 activations and weights, fp32 accumulation, bf16 results rounded
 *     to nearest even).
 *   - Supported shapes: 1 <= E <= 256, 1 <= k <= min(E, 8), H % 64 == 0,
 *     F % 64 == 0, Fs % 64 == 0 (or Fs == 0), T >= 1, T*k < 2^31.
 *     Anything else returns MOE_ERR_UNSUPPORTED (or MOE_ERR_INVALID_ARG for
 *     null pointers / non-positive sizes).
 *   - Weights use the [out, in] layout of a Linear layer: Wg [E,H],
 *     W1 [E,F,H], W2 [E,H,F], Ws1 [Fs,H], Ws2 [H,Fs]. No Linear has a bias.
 */
#ifndef MOE_H_
#define MOE_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { MOE_F32 = 0, MOE_BF16 = 1 } moe_dtype;

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = -1, /* null or misaligned pointer, non-positive size, bad enum */
  MOE_ERR_UNSUPPORTED = -2, /* shape outside the supported range */
  MOE_ERR_WORKSPACE = -3,   /* workspace missing or smaller than the query */
  MOE_ERR_HIP = -4,         /* a HIP launch failed */
  MOE_ERR_SCRATCH = -5      /* beyond the fixed scratch of moe_dispatch_noalloc */
} moe_status;

/* Load diagnostics of one step ([DIAG] section 3). Written to device memory. */
typedef struct {
  int64_t num_tokens;      /* T */
  int64_t assignments;     /* T*k */
  int64_t capacity;        /* int((T*k / E) * cf), evaluated in double */
  int64_t max_load;        /* max_e counts[e] */
  int64_t min_load;        /* min_e counts[e] */
  int64_t dropped;         /* sum_e max(0, counts[e] - capacity); counted only */
  int64_t num_stragglers;  /* #{e : counts[e] > capacity} */
  int64_t gini_num;        /* 2*sum_i i*c_(i) - (E+1)*sum c  (c sorted ascending, i = 1..E) */
  int64_t gini_den;        /* E * sum c (1 when sum c == 0) */
  double load_skew_ratio;  /* (double)max / ((double)min + 1e-5) */
  double gini;             /* (double)gini_num / (double)gini_den, one division; 0 if sum c == 0 */
  double drop_rate;        /* (double)dropped / (double)(T*k) */
} moe_load_stats_t;

/*
 * moe_route - top-k softmax gating ([K3] router listing; [DIAG] section 4.2).
 *   s[t,e]  = sum_h x[t,h] * wg[e,h] + bias[e]          (fp32 accumulation)
 *   topk_idx[t,0..k-1] = the k largest s[t,:], descending; equal scores take
 *                        the lower expert id first
 *   topk_w[t,j] = exp(s[t,idx_j] - m) / sum_j' exp(s[t,idx_j'] - m), m = max_e s[t,e]
 *               (the softmax over all E experts renormalised over the k chosen
 *                ones; the full-E denominator cancels)
 *   prob_mean[e] = (1/T) sum_t p[t,e], p[t,e] = exp(s[t,e] - m) / sum_e' exp(s[t,e'] - m)
 *               (the P_i of [DIAG] section 4.1: mean router probability of the
 *                biased softmax over all E experts; fp32 sums per workgroup in
 *                token order, summed over workgroups in double in a fixed
 *                order, so repeated calls give the same bits)
 * x        [T,H] dtype          device, read
 * wg       [E,H] dtype          device, read
 * bias     [E]   fp32 or NULL   device, read (NULL = no routing bias)
 * topk_idx [T,k] int32          device, written
 * topk_w   [T,k] fp32           device, written
 * prob_mean [E]  fp32 or NULL   device, written (NULL = not computed)
 * ws / ws_bytes: device workspace of at least moe_route_workspace_bytes(T,H,E,k,dtype)
 *          (NULL / 0 allowed when prob_mean is NULL and the query's score part is 0)
 */
int moe_route(const void* x, const void* wg, const float* bias, int T, int H, int E, int k,
              int dtype, int32_t* topk_idx, float* topk_w, float* prob_mean, void* ws,
              size_t ws_bytes, void* stream);

/* Workspace bytes moe_route needs for (T, H, E, k, dtype) with prob_mean
 * requested: partial score tiles when few tokens (T < 2048, bf16) take the
 * two-launch path, plus one row of E partial probability sums per workgroup.
 * Without prob_mean only the score part is needed, which is 0 for T >= 2048
 * or fp32. Returns 0 on unsupported sizes. */
size_t moe_route_workspace_bytes(int T, int H, int E, int k, int dtype);

/* Workspace bytes moe_dispatch needs for (T, E, k); 0 on unsupported sizes. */
size_t moe_dispatch_workspace_bytes(int T, int E, int k);

/*
 * moe_dispatch - group the T*k (token, slot) assignments by expert
 * ([BLOG] section 3.1 dispatcher; histogram as in [DIAG] section 3).
 *   counts[e]   = #{(t,j) : topk_idx[t,j] == e}
 *   offsets[0]  = 0, offsets[e+1] = offsets[e] + counts[e]
 *   perm[p]     = t*k + j for buffer row p, in expert-major, token-ascending
 *                 order (a stable sort of the row-major assignments by expert)
 *   inv[t*k+j]  = p, the inverse of perm
 *   xs[p,:]     = x[perm[p] / k, :] (exact copy)
 * topk_idx [T,k] int32 in [0,E)  device, read (ids of one token are distinct)
 * x        [T,H] dtype           device, read
 * counts [E], offsets [E+1], perm [T*k], inv [T*k] int32; xs [T*k,H] dtype: device, written
 * xs may be NULL: then no rows are copied (x is not read and may be NULL too),
 * for moe_expert_ffn_gather, which reads x through perm itself.
 * ws / ws_bytes: device workspace of at least moe_dispatch_workspace_bytes(T,E,k)
 */
int moe_dispatch(const int32_t* topk_idx, const void* x, int T, int H, int E, int k, int dtype,
                 int32_t* counts, int32_t* offsets, int32_t* perm, int32_t* inv, void* xs,
                 void* ws, size_t ws_bytes, void* stream);

/*
 * moe_dispatch_noalloc - moe_dispatch for callers that cannot allocate
 * device memory (code under HIP graph capture, tight serving loops, harnesses
 * that forbid hipMalloc): the same kernels and results, bit for bit, with the
 * histogram table in a fixed 1 MiB device array of the library instead of a
 * caller workspace. The library itself never allocates in this call.
 * Limit: the table needs E * ceil(T / 256) * 4 bytes (64-token blocks for
 * 256 < T <= 4096 with k >= 4), which must fit 1 MiB: every T <= 2^26 / E
 * (T <= 262144 at E = 256). A larger request returns MOE_ERR_SCRATCH and
 * enqueues nothing.
 * Each GPU holds one copy of the array until the process ends, and every call
 * on that GPU shares it: two calls that may run at the same time on one GPU
 * (on different streams, or from different host threads) race and give wrong
 * results; calls ordered on one stream do not. Nothing in the array needs
 * clearing between calls (the histogram launch writes every entry the rank
 * launch reads). Arguments, outputs and other errors as moe_dispatch.
 */
int moe_dispatch_noalloc(const int32_t* topk_idx, const void* x, int T, int H, int E, int k,
                         int dtype, int32_t* counts, int32_t* offsets, int32_t* perm,
                         int32_t* inv, void* xs, void* stream);

/*
 * moe_capacity - the per-expert capacity of [DIAG] section 3 (its
 * diagnostics listing: the mean assignments per expert times the capacity
 * factor, truncated to an integer):
 *   capacity = int(((double)(T*k) / (double)E) * capacity_factor)
 * evaluated in double in that order, the value moe_load_stats reports in
 * moe_load_stats_t.capacity and the one to pass to moe_dispatch_capped.
 * Host-only: reads no device memory and enqueues nothing.
 * Returns -1 if T < 1, k < 1, E < 1 or capacity_factor is not a finite
 * value > 0; a capacity above INT32_MAX is returned as INT32_MAX (every
 * assignment is then kept, since T*k < 2^31).
 */
int64_t moe_capacity(int T, int k, int E, double capacity_factor);

/*
 * moe_dispatch_capped - moe_dispatch with each expert's capacity enforced
 * ([DIAG] section 3 counts the assignments past an expert's capacity
 * int(T*k/E*cf); section 5 describes dropping them). Every expert keeps its
 * first `capacity` assignments in token order (the order of moe_dispatch);
 * the others are dropped: they get no buffer row and inv = -1.
 *   counts[e]  = raw count, as in moe_dispatch (before dropping)
 *   offsets[0] = 0, offsets[e+1] = offsets[e] + min(counts[e], capacity)
 *   perm[p], xs[p] for p < offsets[E]: the kept rows, as in moe_dispatch
 *                  (entries p >= offsets[E] are not written)
 *   inv[t*k+j]  = the buffer row of a kept assignment, -1 for a dropped one
 * moe_expert_ffn then runs on the kept rows (pass rows = T*k: an upper bound)
 * and moe_combine skips the dropped assignments without renormalising the
 * kept weights. capacity >= 0 (0 drops every assignment); the layer's value
 * is moe_capacity(T, k, E, capacity_factor). Other arguments, the workspace
 * and errors as moe_dispatch.
 */
int moe_dispatch_capped(const int32_t* topk_idx, const void* x, int T, int H, int E, int k,
                        int capacity, int dtype, int32_t* counts, int32_t* offsets, int32_t* perm,
                        int32_t* inv, void* xs, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes moe_expert_ffn needs; 0 on unsupported sizes. */
size_t moe_expert_ffn_workspace_bytes(int rows, int T, int H, int E, int F, int Fs, int dtype);

/*
 * moe_expert_ffn - grouped expert FFN over the expert-contiguous buffer
 * ([BLOG] section 3.1: each expert is Linear -> GeLU -> Linear; [K3]: one
 * always-on shared expert; FLOPs 4*rows*H*F + 4*T*H*Fs as in [K3]'s
 * compute-time equation).
 *   for each expert e and row p in [offsets[e], offsets[e+1]):
 *     h      = GeLU(xs[p,:] . W1[e]^T)      GeLU(a) = 0.5*a*(1 + erf(a/sqrt(2)))
 *     ys[p,:] = h . W2[e]^T
 *   shared expert (when Fs > 0): ysh[t,:] = GeLU(x[t,:] . Ws1^T) . Ws2^T
 * xs [rows,H], offsets [E+1] (device, from moe_dispatch or moe_dispatch_capped;
 *   offsets[E] <= rows: rows is an upper bound that sizes the launch and the
 *   workspace, and ys rows past offsets[E] are not written)
 * w1 [E,F,H], w2 [E,H,F]; x [T,H], ws1 [Fs,H], ws2 [H,Fs] (NULL / Fs = 0: no shared expert)
 * ys [rows,H], ysh [T,H] (NULL when Fs = 0): device, written.
 * In bf16 mode h is rounded to bf16 before the second Linear (fp32 accumulation
 * in both); ys and ysh are rounded to bf16; erf is evaluated with Abramowitz &
 * Stegun formula 7.1.26 (|error| <= 1.5e-7, far below the bf16 step of h). fp32
 * mode uses the device library's erff.
 * ws / ws_bytes: device workspace of at least moe_expert_ffn_workspace_bytes(...)
 */
int moe_expert_ffn(const void* xs, const int32_t* offsets, int rows, int E, int H, int F,
                   const void* w1, const void* w2, const void* x, const void* ws1,
                   const void* ws2, int T, int Fs, int dtype, void* ys, void* ysh, void* ws,
                   size_t ws_bytes, void* stream);

/*
 * moe_expert_ffn_gather - moe_expert_ffn with the dispatch gather fused into
 * the first Linear: buffer row p of the routed experts is read from the token
 * rows directly, xs[p,:] = x[perm[p] / k, :] ([BLOG] section 3.1 groups token
 * indices by expert; the copy into a shared buffer is not materialised).
 * Results are bit-identical to moe_dispatch (with xs) followed by moe_expert_ffn.
 * x [T,H] dtype, perm [rows] int32 (device, from moe_dispatch or
 *   moe_dispatch_capped, which may run with xs = NULL), 1 <= k <= 8 the
 *   experts per token of that dispatch; a perm entry outside [0, T*k) is
 *   clamped into it (never read out of bounds).
 * All other arguments, the workspace (moe_expert_ffn_workspace_bytes) and the
 * errors as moe_expert_ffn; x is required (it is the routed input as well as
 * the shared expert's).
 */
int moe_expert_ffn_gather(const void* x, const int32_t* perm, int k, const int32_t* offsets,
                          int rows, int E, int H, int F, const void* w1, const void* w2,
                          const void* ws1, const void* ws2, int T, int Fs, int dtype, void* ys,
                          void* ysh, void* ws, size_t ws_bytes, void* stream);

/*
 * moe_expert_ffn_gather_timed - moe_expert_ffn_gather that also records
 * caller-created HIP events on `stream`, for timing the grouped GEMM kernel
 * itself (the FFN's dominant kernel) with events on the stream it runs on:
 * events[0] / events[1] right before / after the up projection's GEMM launch,
 * events[2] / events[3] the same for the down projection. The planning launch
 * and any split-K reduce launch fall outside the pairs. events: host array of
 * 4 hipEvent_t (as void*), owned by the caller; NULL, or a NULL entry, records
 * nothing there. Results, arguments and errors as moe_expert_ffn_gather; a
 * failed event record returns MOE_ERR_HIP.
 */
int moe_expert_ffn_gather_timed(const void* x, const int32_t* perm, int k, const int32_t* offsets,
                                int rows, int E, int H, int F, const void* w1, const void* w2,
                                const void* ws1, const void* ws2, int T, int Fs, int dtype,
                                void* ys, void* ysh, void* ws, size_t ws_bytes, void* stream,
                                void* const* events);

/*
 * moe_combine - weighted combine back to token order ([K3] combine phase;
 * [BLOG] section 3.1 "scatter back to the original positions").
 *   out[t,:] = sum_{j=0..k-1} topk_w[t,j] * ys[inv[t*k+j],:]  (+ ysh[t,:])
 * summed in fp32, j ascending, shared row last; one write per token (no atomics).
 * An assignment with inv < 0 (dropped by moe_dispatch_capped) adds nothing;
 * the other weights are used as they are.
 * ys [T*k,H] dtype, inv [T*k] int32, topk_w [T,k] fp32, ysh [T,H] dtype or NULL: device, read
 * out [T,H] dtype: device, written
 */
int moe_combine(const void* ys, const int32_t* inv, const float* topk_w, const void* ysh, int T,
                int H, int k, int dtype, void* out, void* stream);

/*
 * moe_load_stats - per-step load diagnostics ([DIAG] section 3) from the
 * expert counts that moe_dispatch produced (the routing actually taken).
 * counts        [E] int32            device, read (sum must be T*k)
 * stats         moe_load_stats_t     device, written
 * overflow      [E] int32 or NULL    device, written: max(0, counts[e] - capacity)
 * straggler_ids [E] int32            device, written: ids with counts[e] > capacity,
 *                                    ascending, then -1 up to E entries
 * capacity_factor > 0.
 */
int moe_load_stats(const int32_t* counts, int T, int E, int k, double capacity_factor,
                   moe_load_stats_t* stats, int32_t* overflow, int32_t* straggler_ids,
                   void* stream);

/*
 * moe_bias_update - one step of the dynamic routing bias ([DIAG] section 4.2:
 * lower the bias of an overloaded expert by a small step, raise that of an
 * idle one) and the load fractions of [DIAG] section 4.1.
 *   mean = sum_e counts[e] / E (compared exactly: counts[e]*E vs sum)
 *   bias[e] <- bias[e] - gamma  if counts[e] > mean   (fp32 arithmetic)
 *              bias[e] + gamma  if counts[e] < mean
 *              bias[e]          otherwise
 *   load_frac[e] = counts[e] / sum_e' counts[e'] (double division, rounded
 *                  to fp32; 0 when the sum is 0)
 * counts    [E] int32 >= 0  device, read (one step's counts from moe_dispatch,
 *                           or counts summed by the caller over a window)
 * bias      [E] fp32        device, read and written in place
 * load_frac [E] fp32 or NULL device, written
 * gamma: finite, >= 0. 1 <= E <= 256.
 * The bias feeds the next moe_route; calls on one stream keep that order.
 */
int moe_bias_update(const int32_t* counts, int E, float gamma, float* bias, float* load_frac,
                    void* stream);

typedef enum { MOE_NORM_NONE = 0, MOE_NORM_RMS = 1, MOE_NORM_LAYER = 2 } moe_norm_kind;

/*
 * moe_norm - the norm in front of a block, row by row:
 *   MOE_NORM_RMS:   out = x / sqrt(mean(x^2) + eps) * weight + bias
 *   MOE_NORM_LAYER: out = (x - mu) / sqrt(mean((x - mu)^2) + eps) * weight + bias,
 *                   mu = mean(x)
 * Means over the H elements of a row; statistics and arithmetic in fp32 (the
 * variance around the mean, not as a difference of squares), one rounding to
 * the output type. Any H from 1 to 16384 (H % 64 is not required; rows of
 * 16-byte multiples are faster); a larger one is MOE_ERR_UNSUPPORTED. A row
 * with a NaN or infinity affects only its own output row; a row without
 * variance under eps = 0 divides by zero as the formula does.
 * x      [rows,H] dtype          device, read
 * weight [H] dtype or NULL       device, read (NULL = 1)
 * bias   [H] dtype or NULL       device, read (NULL = 0)
 * out    [rows,H] dtype          device, written; may be x itself (any other
 *                                overlap with an input is MOE_ERR_INVALID_ARG)
 * eps: finite, >= 0. All pointers 16-byte aligned. No workspace.
 */
int moe_norm(const void* x, const void* weight, const void* bias, int rows, int H, float eps,
             int kind, int dtype, void* out, void* stream);

typedef enum {
  MOE_GATE_NONE = 0,    /* 1 */
  MOE_GATE_TOKEN = 1,   /* [rows]: one value a row */
  MOE_GATE_CHANNEL = 2, /* [H]: one value a channel */
  MOE_GATE_FULL = 3     /* [rows,H] */
} moe_gate_mode;

/*
 * moe_norm_residual - what stands between two blocks, in one pass over the rows:
 *   z        = norm(y) by kind, weight, bias (MOE_NORM_NONE: z = y)
 *   h        = res + scale * gate * z
 *   res_out  = h                        rounded to dtype
 *   next_out = norm(h) by next_kind, next_weight, next_bias (of h before its
 *              rounding); not written for MOE_NORM_NONE
 * y, res [rows,H] dtype, gate [rows] / [H] / [rows,H] dtype by gate_mode (NULL
 *   for MOE_GATE_NONE): device, read
 * weight, bias, next_weight, next_bias [H] dtype or NULL: device, read; NULL
 *   with the kind MOE_NORM_NONE
 * res_out, next_out [rows,H] dtype: device, written. res_out may be res itself,
 *   next_out may be y itself and either may be a full gate itself; any other
 *   overlap of an output with the other one or an input is
 *   MOE_ERR_INVALID_ARG. next_out NULL with
 *   next_kind MOE_NORM_NONE.
 * scale: finite. eps, H, alignment and arithmetic as moe_norm.
 */
int moe_norm_residual(const void* y, int kind, const void* weight, const void* bias,
                      const void* res, const void* gate, int gate_mode, float scale,
                      int next_kind, const void* next_weight, const void* next_bias, int rows,
                      int H, float eps, int dtype, void* res_out, void* next_out, void* stream);

typedef enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 } moe_score;

/*
 * moe_route_grouped - top-k gating with a choice bias and groups of experts
 * ([K3] router listing for scores, top-k and renormalisation; the balance bias
 * of [DIAG] section 4.2 moves the choice here, not the weights: moe_route has
 * it inside the softmax).
 *   s[t,e] = sum_h x[t,h] * wg[e,h]                       (fp32 accumulation)
 *   p[t,e] = softmax over e of s[t,:], or 1 / (1 + exp(-s[t,e]))
 *   v[t,e] = p[t,e] + bias[e]
 *   group j = the experts [j*E/groups, (j+1)*E/groups); its score is the
 *            largest v in it (group_top 1) or the sum of the two largest (2)
 *   chosen groups: the topk_groups best, equal scores to the lower group
 *   topk_idx[t,0..k-1] = the k largest v among the experts of the chosen
 *            groups, descending, equal ones to the lower expert id
 *   topk_w[t,j] = scale * p[t,idx_j] / (renorm ? sum_j' p[t,idx_j'] : 1)
 * Without a bias the experts are ordered by s (the same order as p, kept where
 * p rounds to 0 or 1). v is worked out with the hardware's exp2 and reciprocal,
 * as is the softmax's sum (about 2e-7 relative); the weights' p with expf.
 * An expert with a bias of -inf or NaN, or a NaN score, is off: it counts in no
 * group's score (a group with one expert left scores that one alone) and is
 * chosen only when fewer than k experts of the chosen groups are on, then with
 * weight 0 (lower ids first). A NaN score counts as -inf in the softmax. If the
 * chosen p are all 0 the weights are 0.
 * x [T,H], wg [E,H] dtype, bias [E] fp32 or NULL: device, read
 * topk_idx [T,k] int32, topk_w [T,k] fp32: device, written
 * 1 <= groups <= 64, E % groups == 0, 1 <= topk_groups <= groups,
 * k <= topk_groups * E / groups, T <= 2^27, scale finite; else MOE_ERR_UNSUPPORTED (or
 * MOE_ERR_INVALID_ARG for non-positive sizes, unknown enums and outputs or a
 * workspace that overlap another operand).
 * ws / ws_bytes: device workspace of at least
 *   moe_route_grouped_workspace_bytes(T,H,E,k,dtype) (NULL allowed when that is 0)
 */
int moe_route_grouped(const void* x, const void* wg, const float* bias, int T, int H, int E, int k,
                      int score, int groups, int topk_groups, int group_top, int renorm,
                      float scale, int dtype, int32_t* topk_idx, float* topk_w, void* ws,
                      size_t ws_bytes, void* stream);
size_t moe_route_grouped_workspace_bytes(int T, int H, int E, int k, int dtype);

typedef enum {
  MOE_ACT_NONE = 0,
  MOE_ACT_GELU = 1,   /* 0.5*a*(1 + erf(a/sqrt(2))) */
  MOE_ACT_SILU = 2,   /* a / (1 + exp(-a)) */
  MOE_ACT_GEGLU = 3,  /* gelu(a_0) * a_1 */
  MOE_ACT_SWIGLU = 4  /* silu(a_0) * a_1 */
} moe_act;

/*
 * moe_linear - matrix product with its epilogue:
 *   a[m,n] = sum_k x[m,k] * w[n,k] + bias[n]             (fp32 accumulation)
 *   y[m,n] = act(a[m,n]) + residual[m,n]
 * and for a gated act, with w [2,N,K] and bias [2,N] (half 0 the gate):
 *   y[m,n] = act(a_0[m,n]) * a_1[m,n] + residual[m,n]
 * Bias, activation, gate and residual are applied in fp32 to the accumulator;
 * y is rounded once. The bf16 form evaluates GeLU by a fit of the normal tail
 * (within 4e-6 relative of the formula up to |a| = 6, 6e-9 beyond) and SiLU
 * with the hardware's exp2 and reciprocal (a few fp32 ulp).
 * x [M,K], w [N,K] or [2,N,K], bias [N] or [2,N] or NULL, residual [M,N] or NULL,
 * all dtype: device, read; y [M,N] dtype: device, written. y may be residual
 * itself, and overlaps no other input.
 * K % 64 == 0, N % 64 == 0, any M >= 1 whose tiles fit a launch (about M * N <
 * 2^36; else MOE_ERR_UNSUPPORTED). An output or workspace that overlaps another
 * operand (other than y being residual) is MOE_ERR_INVALID_ARG.
 * ws / ws_bytes: device workspace of at least
 *   moe_linear_workspace_bytes(M,N,K,act,dtype) (NULL allowed when that is 0)
 */
int moe_linear(const void* x, const void* w, const void* bias, int act, const void* residual,
               int M, int N, int K, int dtype, void* y, void* ws, size_t ws_bytes, void* stream);
size_t moe_linear_workspace_bytes(int M, int N, int K, int act, int dtype);

/*
 * moe_linear_grouped - moe_linear over the experts' ragged segments: buffer row
 * p in [offsets[e], offsets[e+1]) takes the weights w[e] and bias[e] of its
 * expert. Two calls make gated experts ([BLOG] section 3.1's pair of Linear
 * layers with a gate): the up half with MOE_ACT_SWIGLU reading x through perm,
 * the down half with MOE_ACT_NONE.
 * x [rows,K], or with perm the token rows [T,K]: buffer row p then reads
 *   x[perm[p] / k] (a perm entry outside [0, T*k) is clamped into it)
 * perm [rows] int32 or NULL, 1 <= k <= 8 (with perm only; T and k are
 *   otherwise not used), rows <= T*k
 * offsets [E+1] int32 from moe_dispatch or moe_dispatch_capped; rows is an upper
 *   bound of offsets[E], and rows of y past offsets[E] are left as they were
 *   (offsets are clamped into the buffer; a segment of no rows is fine)
 * w [E,N,K] or [E,2,N,K], bias [E,N] or [E,2,N] or NULL, residual [rows,N] or NULL,
 * y [rows,N]: as moe_linear. 1 <= E <= 256.
 * ws / ws_bytes: moe_linear_grouped_workspace_bytes(E,rows,N,K,act,dtype)
 */
int moe_linear_grouped(const void* x, const int32_t* perm, int k, int T, const int32_t* offsets,
                       int E, int rows, const void* w, const void* bias, int act,
                       const void* residual, int N, int K, int dtype, void* y, void* ws,
                       size_t ws_bytes, void* stream);
size_t moe_linear_grouped_workspace_bytes(int E, int rows, int N, int K, int act, int dtype);

typedef enum {
  MOE_PATH_ROWS = 0,     /* few rows: weights straight to registers */
  MOE_PATH_TILES = 1,    /* tiles of 64 (fp32 also 32) rows x 64 weight rows, K slices */
  MOE_PATH_256X128 = 2,  /* tiles of 256 rows x 128 weight rows */
  MOE_PATH_256X256 = 3   /* tiles of 256 rows x 256 weight rows */
} moe_path;

/*
 * moe_linear_path - the kernels that a product of these sizes takes (a host
 * query, for profiles and tests; nothing is launched): a moe_path, or a negative
 * status. grouped: 0 for moe_linear (E = 1), 1 for moe_linear_grouped.
 * slices (or NULL) receives the slices of K: of every tile, for the 256-row
 * tiles those of the last round's; 0 where the offsets decide it (grouped
 * 256-row tiles of K >= 8192). A grouped product whose gathered x passes 4 GiB
 * takes MOE_PATH_TILES with one slice in place of the 256-row tiles.
 */
int moe_linear_path(int E, int rows, int N, int K, int act, int grouped, int dtype, int* slices);

/*
 * moe_quantize - rows to 8-bit floating point (e4m3, the OCP form without
 * infinities, largest value 448) with one scale for each block of 128 elements:
 *   amax       = the largest finite |x| of elements 128 b .. 128 b + 127 of row r
 *   scale[b,r] = the least power of two s with amax / s <= 448, 2^-126 at least;
 *                1 if amax = 0
 *   q[r,c]     = x[r,c] / scale[c / 128, r], rounded once (nearest, ties to even);
 *                NaN for an infinity or NaN, which the scale leaves out
 * x     [rows,K] dtype         device, read
 * q     [rows,K] e4m3 bytes    device, written
 * scale [K/128,rows] fp32      device, written (the rows of a block side by side)
 * Power-of-two scales keep a block's largest element less exactly than amax / 448 does
 * (error relative to the data's norm: 2.7e-2 against 2.6e-2 on Gaussian data, against 1.0e-2
 * where 1 % of the elements are up to 200 times as large).
 * K % 128 == 0; rows * K up to about 2^37 (else MOE_ERR_UNSUPPORTED). x and q
 * 16-byte, scale 4-byte aligned; outputs that overlap each other or x are
 * MOE_ERR_INVALID_ARG. No workspace.
 */
int moe_quantize(const void* x, int rows, int K, int dtype, void* q, float* scale, void* stream);

/*
 * moe_quantize_weight - the same for weights, with one scale for each block of 128
 * rows x 128 elements (the last block of an N that is no multiple of 128 has fewer
 * rows):
 *   scale[i,n/128,b] as above over the block, q[i,n,c] = w[i,n,c] / scale
 * w [count,N,K] dtype, q [count,N,K] e4m3, scale [count,ceil(N/128),K/128] fp32. count:
 * the matrices (experts, and gate and up halves). N % 64 == 0, else as moe_quantize.
 */
int moe_quantize_weight(const void* w, int count, int N, int K, int dtype, void* q, float* scale,
                        void* stream);

/*
 * moe_linear_fp8 - moe_linear of e4m3 operands with block scales, in bf16:
 *   a[m,n] = sum_b x_scale[b,m] * w_scale[n/128,b] *
 *            sum_{k = 128 b .. 128 b + 127} x[m,k] * w[n,k]      + bias[n]
 *   y[m,n] = act(a[m,n]) + residual[m,n], or with a gate as moe_linear
 * The products of a block are summed by the matrix cores (8 neighbours of K at a time, cut
 * at 2^-13 of the largest of the 8, then in fp32), the blocks scaled and summed in fp32;
 * bias, act, gate and residual as moe_linear's bf16 form; one rounding.
 * x [M,K] e4m3, x_scale [K/128,M] fp32, w [N,K] or [2,N,K] e4m3, w_scale
 *   [ceil(N/128),K/128] or [2,ceil(N/128),K/128] fp32 (those of moe_quantize and
 *   moe_quantize_weight, or a checkpoint's, of any mantissa; x_scale[b,m] * w_scale[n/128,b]
 *   is one fp32 number, so it has to stay below 2^128, where a block's sum would become
 *   infinite or, if it is 0, NaN, and loses bits below 2^-126), bias [N] or [2,N] bf16 or
 *   NULL, residual [M,N] bf16 or NULL: device, read; y [M,N] bf16: device, written; it
 *   may be residual itself.
 * K % 128 == 0, N % 64 == 0. Scales 4-byte, the others 16-byte aligned. Sizes whose
 * tiles do not fit a launch are MOE_ERR_UNSUPPORTED, an output or workspace that
 * overlaps another operand (other than y being residual) MOE_ERR_INVALID_ARG.
 * ws / ws_bytes: moe_linear_fp8_workspace_bytes(M,N,K,act) (NULL allowed when that is 0)
 */
int moe_linear_fp8(const void* x, const float* x_scale, const void* w, const float* w_scale,
                   const void* bias, int act, const void* residual, int M, int N, int K, void* y,
                   void* ws, size_t ws_bytes, void* stream);
size_t moe_linear_fp8_workspace_bytes(int M, int N, int K, int act);

/*
 * moe_linear_grouped_fp8 - moe_linear_fp8 over the experts' ragged segments, as
 * moe_linear_grouped: buffer row p in [offsets[e], offsets[e+1]) takes w[e], w_scale[e]
 * and bias[e]; rows of y past offsets[E] are left as they were.
 * x [rows,K] and x_scale [K/128,rows], or with perm the token rows [T,K] and
 *   [K/128,T]: buffer row p then reads row perm[p] / k (clamped into x)
 * w [E,N,K] or [E,2,N,K], w_scale [E,ceil(N/128),K/128] or [E,2,ceil(N/128),K/128].
 * perm, k, T, offsets, rows, bias, residual, y as moe_linear_grouped; the rest as
 * moe_linear_fp8.
 * ws / ws_bytes: moe_linear_grouped_fp8_workspace_bytes(E,rows,N,K,act)
 */
int moe_linear_grouped_fp8(const void* x, const float* x_scale, const int32_t* perm, int k, int T,
                           const int32_t* offsets, int E, int rows, const void* w,
                           const float* w_scale, const void* bias, int act, const void* residual,
                           int N, int K, void* y, void* ws, size_t ws_bytes, void* stream);
size_t moe_linear_grouped_fp8_workspace_bytes(int E, int rows, int N, int K, int act);

typedef enum {
  MOE_FP8_ROWS = 0,    /* few rows: weights straight to registers */
  MOE_FP8_64X64 = 1,   /* tiles of 64 rows x 64 weight rows */
  MOE_FP8_128X128 = 2, /* tiles of 128 rows x 128 weight rows */
  MOE_FP8_256X256 = 3  /* tiles of 256 rows x 256 weight rows */
} moe_fp8_path;

/* The kernels and K slices that an 8-bit product of these sizes takes, as
 * moe_linear_path: a moe_fp8_path, or a negative status. (Rows gathered from an x of 4 GiB
 * or more take MOE_FP8_ROWS, whatever the sizes.) */
int moe_linear_fp8_path(int E, int rows, int N, int K, int act, int grouped, int* slices);

/* What a routing bias moves. */
typedef enum {
  MOE_BIAS_CHOICE = 0, /* the choice, not the weights (moe_route_grouped) */
  MOE_BIAS_SCORE = 1   /* the scores themselves (moe_route) */
} moe_bias_mode;

/*
 * moe_layer_few - a whole MoE layer for a few tokens (1 <= T <= 64), in two or three launches.
 * Called one by one it is faster than the separate calls (route, dispatch, products, combine)
 * wherever those are bound by the host, some 65 us. Against a HIP graph of them it pays for
 * experts of about 3 MB of weights (1024 x 512 gated, bf16) or more with up to 4 pairs of a
 * token and an expert each (T k / E); a graph of the separate calls is up to 1.2 times as
 * fast with 8 pairs an expert, 1.5 with 16, and 1.7 with smaller experts from 4 tokens on.
 *   s[t,e] = sum_h x[t,h] * wg[e,h]  (+ bias[e] with MOE_BIAS_SCORE)
 *   topk_idx, topk_w from s as moe_route_grouped (bias as its bias with
 *            MOE_BIAS_CHOICE, none with MOE_BIAS_SCORE; softmax, MOE_BIAS_SCORE, one
 *            group, renorm and scale 1 are moe_route)
 *   h_j    = act(x[t] . w_up[e_j]^T + b_up[e_j]), e_j = topk_idx[t,j]   rounded to dtype
 *   out[t] = sum_j topk_w[t,j] * (h_j . w_down[e_j]^T + b_down[e_j])
 *            + act(x[t] . ws_up^T) . ws_down^T              (shared expert, Fs > 0)
 * Products and sums in fp32; h and out are rounded once each (an expert's row is not
 * rounded before the weighted sum, as moe_combine's ys are). A gated act has a gate and
 * an up half as moe_linear. Sums are in an order fixed by the sizes and the choice:
 * equal calls give equal bits.
 * x [T,H], wg [E,H], w_up [E,F,H] or [E,2,F,H], w_down [E,H,F], b_up [E,F] or
 *   [E,2,F] or NULL, b_down [E,H] or NULL, ws_up [Fs,H] or [2,Fs,H], ws_down [H,Fs]
 *   (NULL / Fs = 0: no shared expert), all dtype; bias [E] fp32 or NULL: device, read
 * out [T,H] dtype, topk_idx [T,k] int32, topk_w [T,k] fp32: device, written
 * E, k, H, F, Fs as the layer's, H, F, Fs <= 2^20; routing options as moe_route_grouped.
 * T > 64 and a gate half of one expert of 4 GiB or more are MOE_ERR_UNSUPPORTED; an
 * output or workspace that overlaps another operand MOE_ERR_INVALID_ARG.
 * ws / ws_bytes: device workspace of at least
 *   moe_layer_few_workspace_bytes(T,H,E,k,F,Fs,dtype); its content does not matter. Calls
 *   that may run at the same time need workspaces of their own: with a shared one the
 *   outputs of both are undefined (no access leaves the operands, and both calls end).
 */
int moe_layer_few(const void* x, const void* wg, const float* bias, int bias_mode,
                  const void* w_up, const void* w_down, const void* b_up, const void* b_down,
                  const void* ws_up, const void* ws_down, int T, int H, int E, int k, int F, int Fs,
                  int act, int score, int groups, int topk_groups, int group_top, int renorm,
                  float scale, int dtype, void* out, int32_t* topk_idx, float* topk_w, void* ws,
                  size_t ws_bytes, void* stream);
size_t moe_layer_few_workspace_bytes(int T, int H, int E, int k, int F, int Fs, int dtype);

/* Static, human-readable text for a status code. */
const char* moe_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H_ */
