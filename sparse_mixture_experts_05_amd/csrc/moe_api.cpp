// C ABI of the MoE layer library: argument validation (always before any HIP
// call, so a rejected call enqueues nothing), workspace sizing, launches on
// the caller's stream. The semantics of each entry point are documented in
// include/moe.h.
#include "moe.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <initializer_list>

#include "kernels.hpp"

namespace {

constexpr int kMaxExperts = 256;
constexpr int kMaxTopK = 8;

bool dtype_ok(int dt) { return dt == MOE_F32 || dt == MOE_BF16; }

// Shared shape checks of (T, H, E, k). Returns MOE_OK or an error status.
int check_tokens(int T, int H, int E, int k) {
  if (T < 1 || H < 1 || E < 1 || k < 1) return MOE_ERR_INVALID_ARG;
  if (E > kMaxExperts || k > kMaxTopK || k > E) return MOE_ERR_UNSUPPORTED;
  if (H % 64 != 0) return MOE_ERR_UNSUPPORTED;
  if ((long long)T * k >= (1LL << 31)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int from_hip(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// Rows and weights are read and written with 16-byte vector accesses.
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

}  // namespace

extern "C" {

const char* moe_status_string(int status) {
  switch (status) {
    case MOE_OK: return "ok";
    case MOE_ERR_INVALID_ARG: return "invalid argument (null or misaligned pointer, non-positive size, bad dtype or an output over another operand)";
    case MOE_ERR_UNSUPPORTED: return "unsupported shape (needs 1<=E<=256, 1<=k<=min(E,8), H%64==0, F%64==0, T*k<2^31; norms: H<=16384; moe_route_grouped: E%groups==0, groups<=64, topk_groups<=groups, k<=topk_groups*E/groups; products: N%64==0, K%64==0)";
    case MOE_ERR_WORKSPACE: return "workspace missing or smaller than the size query returned";
    case MOE_ERR_HIP: return "HIP launch failed";
    case MOE_ERR_SCRATCH: return "request exceeds the fixed 1 MiB scratch of moe_dispatch_noalloc (needs E * ceil(T / 256) * 4 <= 1 MiB; use moe_dispatch with a workspace)";
    default: return "unknown status";
  }
}

size_t moe_route_workspace_bytes(int T, int H, int E, int k, int dtype) {
  if (!dtype_ok(dtype) || check_tokens(T, H, E, k) != MOE_OK) return 0;
  return moe::route_ws_bytes(T, H, E, dtype == MOE_BF16, true);
}

int moe_route(const void* x, const void* wg, const float* bias, int T, int H, int E, int k,
              int dtype, int32_t* topk_idx, float* topk_w, float* prob_mean, void* ws,
              size_t ws_bytes, void* stream) {
  if (!x || !wg || !topk_idx || !topk_w || !dtype_ok(dtype)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(wg) || (ws && !aligned16(ws))) return MOE_ERR_INVALID_ARG;
  const int st = check_tokens(T, H, E, k);
  if (st != MOE_OK) return st;
  const size_t need = moe::route_ws_bytes(T, H, E, dtype == MOE_BF16, prob_mean != nullptr);
  if (need > 0 && (!ws || ws_bytes < need)) return MOE_ERR_WORKSPACE;
  return from_hip(moe::launch_route(x, wg, bias, T, H, E, k, dtype == MOE_BF16, topk_idx, topk_w,
                                    prob_mean, ws, as_stream(stream)));
}

size_t moe_dispatch_workspace_bytes(int T, int E, int k) {
  if (check_tokens(T, 64, E, k) != MOE_OK) return 0;
  return moe::dispatch_ws_bytes(T, E, k);
}

int moe_dispatch(const int32_t* topk_idx, const void* x, int T, int H, int E, int k, int dtype,
                 int32_t* counts, int32_t* offsets, int32_t* perm, int32_t* inv, void* xs,
                 void* ws, size_t ws_bytes, void* stream) {
  if (!topk_idx || !counts || !offsets || !perm || !inv || !dtype_ok(dtype))
    return MOE_ERR_INVALID_ARG;
  if (xs && (!x || !aligned16(x) || !aligned16(xs))) return MOE_ERR_INVALID_ARG;
  const int st = check_tokens(T, H, E, k);
  if (st != MOE_OK) return st;
  if (!ws || ws_bytes < moe::dispatch_ws_bytes(T, E, k)) return MOE_ERR_WORKSPACE;
  return from_hip(moe::launch_dispatch(topk_idx, x, T, H, E, k, -1, dtype == MOE_BF16, counts,
                                       offsets, perm, inv, xs, ws, as_stream(stream)));
}

int moe_dispatch_noalloc(const int32_t* topk_idx, const void* x, int T, int H, int E, int k,
                         int dtype, int32_t* counts, int32_t* offsets, int32_t* perm,
                         int32_t* inv, void* xs, void* stream) {
  if (!topk_idx || !counts || !offsets || !perm || !inv || !dtype_ok(dtype))
    return MOE_ERR_INVALID_ARG;
  if (xs && (!x || !aligned16(x) || !aligned16(xs))) return MOE_ERR_INVALID_ARG;
  const int st = check_tokens(T, H, E, k);
  if (st != MOE_OK) return st;
  if (moe::dispatch_ws_bytes(T, E, k) > moe::noalloc_scratch_bytes()) return MOE_ERR_SCRATCH;
  return from_hip(moe::launch_dispatch_noalloc(topk_idx, x, T, H, E, k, dtype == MOE_BF16, counts,
                                               offsets, perm, inv, xs, as_stream(stream)));
}

int64_t moe_capacity(int T, int k, int E, double capacity_factor) {
  if (T < 1 || k < 1 || E < 1) return -1;
  if (!(capacity_factor > 0.0) || !std::isfinite(capacity_factor)) return -1;
  // the same double operations as the statistics kernel: (T*k)/E first, then *cf
  const double cap = ((double)((long long)T * k) / (double)E) * capacity_factor;
  if (cap >= 2147483647.0) return 2147483647;
  return (int64_t)cap;
}

int moe_dispatch_capped(const int32_t* topk_idx, const void* x, int T, int H, int E, int k,
                        int capacity, int dtype, int32_t* counts, int32_t* offsets, int32_t* perm,
                        int32_t* inv, void* xs, void* ws, size_t ws_bytes, void* stream) {
  if (!topk_idx || !counts || !offsets || !perm || !inv || !dtype_ok(dtype) || capacity < 0)
    return MOE_ERR_INVALID_ARG;
  if (xs && (!x || !aligned16(x) || !aligned16(xs))) return MOE_ERR_INVALID_ARG;
  const int st = check_tokens(T, H, E, k);
  if (st != MOE_OK) return st;
  if (!ws || ws_bytes < moe::dispatch_ws_bytes(T, E, k)) return MOE_ERR_WORKSPACE;
  return from_hip(moe::launch_dispatch(topk_idx, x, T, H, E, k, capacity, dtype == MOE_BF16,
                                       counts, offsets, perm, inv, xs, ws, as_stream(stream)));
}

static int check_ffn(int rows, int T, int H, int E, int F, int Fs, int dtype) {
  if (rows < 1 || T < 1 || H < 1 || E < 1 || F < 1 || Fs < 0 || !dtype_ok(dtype))
    return MOE_ERR_INVALID_ARG;
  if (E > kMaxExperts || H % 64 != 0 || F % 64 != 0 || Fs % 64 != 0) return MOE_ERR_UNSUPPORTED;
  if ((long long)rows > (long long)T * kMaxTopK) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

size_t moe_expert_ffn_workspace_bytes(int rows, int T, int H, int E, int F, int Fs, int dtype) {
  if (check_ffn(rows, T, H, E, F, Fs, dtype) != MOE_OK) return 0;
  return moe::ffn_ws_bytes(rows, T, E, H, F, Fs, dtype == MOE_BF16);
}

int moe_expert_ffn(const void* xs, const int32_t* offsets, int rows, int E, int H, int F,
                   const void* w1, const void* w2, const void* x, const void* ws1,
                   const void* ws2, int T, int Fs, int dtype, void* ys, void* ysh, void* ws,
                   size_t ws_bytes, void* stream) {
  if (!xs || !offsets || !w1 || !w2 || !ys) return MOE_ERR_INVALID_ARG;
  if (!aligned16(xs) || !aligned16(w1) || !aligned16(w2) || !aligned16(ys)) return MOE_ERR_INVALID_ARG;
  const int st = check_ffn(rows, T, H, E, F, Fs, dtype);
  if (st != MOE_OK) return st;
  if (Fs > 0 && (!x || !ws1 || !ws2 || !ysh)) return MOE_ERR_INVALID_ARG;
  if (Fs > 0 && (!aligned16(x) || !aligned16(ws1) || !aligned16(ws2) || !aligned16(ysh)))
    return MOE_ERR_INVALID_ARG;
  if (ws && !aligned16(ws)) return MOE_ERR_INVALID_ARG;
  if (!ws || ws_bytes < moe::ffn_ws_bytes(rows, T, E, H, F, Fs, dtype == MOE_BF16))
    return MOE_ERR_WORKSPACE;
  return from_hip(moe::launch_expert_ffn(xs, nullptr, 0, offsets, rows, E, H, F, w1, w2, x, ws1,
                                         ws2, T, Fs, dtype == MOE_BF16, ys,
                                         Fs > 0 ? ysh : nullptr, ws, as_stream(stream)));
}

int moe_expert_ffn_gather(const void* x, const int32_t* perm, int k, const int32_t* offsets,
                          int rows, int E, int H, int F, const void* w1, const void* w2,
                          const void* ws1, const void* ws2, int T, int Fs, int dtype, void* ys,
                          void* ysh, void* ws, size_t ws_bytes, void* stream) {
  return moe_expert_ffn_gather_timed(x, perm, k, offsets, rows, E, H, F, w1, w2, ws1, ws2, T, Fs,
                                     dtype, ys, ysh, ws, ws_bytes, stream, nullptr);
}

int moe_expert_ffn_gather_timed(const void* x, const int32_t* perm, int k, const int32_t* offsets,
                                int rows, int E, int H, int F, const void* w1, const void* w2,
                                const void* ws1, const void* ws2, int T, int Fs, int dtype,
                                void* ys, void* ysh, void* ws, size_t ws_bytes, void* stream,
                                void* const* events) {
  if (!x || !perm || !offsets || !w1 || !w2 || !ys) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w1) || !aligned16(w2) || !aligned16(ys)) return MOE_ERR_INVALID_ARG;
  if (k < 1) return MOE_ERR_INVALID_ARG;
  if (k > kMaxTopK || (long long)T * k >= (1LL << 31)) return MOE_ERR_UNSUPPORTED;
  const int st = check_ffn(rows, T, H, E, F, Fs, dtype);
  if (st != MOE_OK) return st;
  if ((long long)rows > (long long)T * k) return MOE_ERR_UNSUPPORTED;
  if (Fs > 0 && (!ws1 || !ws2 || !ysh)) return MOE_ERR_INVALID_ARG;
  if (Fs > 0 && (!aligned16(ws1) || !aligned16(ws2) || !aligned16(ysh))) return MOE_ERR_INVALID_ARG;
  if (ws && !aligned16(ws)) return MOE_ERR_INVALID_ARG;
  if (!ws || ws_bytes < moe::ffn_ws_bytes(rows, T, E, H, F, Fs, dtype == MOE_BF16))
    return MOE_ERR_WORKSPACE;
  return from_hip(moe::launch_expert_ffn(x, perm, k, offsets, rows, E, H, F, w1, w2, x, ws1, ws2,
                                         T, Fs, dtype == MOE_BF16, ys, Fs > 0 ? ysh : nullptr, ws,
                                         as_stream(stream), events));
}

int moe_combine(const void* ys, const int32_t* inv, const float* topk_w, const void* ysh, int T,
                int H, int k, int dtype, void* out, void* stream) {
  if (!ys || !inv || !topk_w || !out || !dtype_ok(dtype)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(ys) || !aligned16(out) || (ysh && !aligned16(ysh))) return MOE_ERR_INVALID_ARG;
  const int st = check_tokens(T, H, kMaxTopK, k);
  if (st != MOE_OK) return st;
  return from_hip(moe::launch_combine(ys, inv, topk_w, ysh, T, H, k, dtype == MOE_BF16, out,
                                      as_stream(stream)));
}

int moe_load_stats(const int32_t* counts, int T, int E, int k, double capacity_factor,
                   moe_load_stats_t* stats, int32_t* overflow, int32_t* straggler_ids,
                   void* stream) {
  if (!counts || !stats || !straggler_ids) return MOE_ERR_INVALID_ARG;
  if (!(capacity_factor > 0.0) || !std::isfinite(capacity_factor)) return MOE_ERR_INVALID_ARG;
  const int st = check_tokens(T, 64, E, k);
  if (st != MOE_OK) return st;
  return from_hip(moe::launch_load_stats(counts, T, E, k, capacity_factor, stats, overflow,
                                         straggler_ids, as_stream(stream)));
}

int moe_bias_update(const int32_t* counts, int E, float gamma, float* bias, float* load_frac,
                    void* stream) {
  if (!counts || !bias || E < 1 || !std::isfinite(gamma) || gamma < 0.0f)
    return MOE_ERR_INVALID_ARG;
  if (E > kMaxExperts) return MOE_ERR_UNSUPPORTED;
  return from_hip(moe::launch_bias_update(counts, E, gamma, bias, load_frac, as_stream(stream)));
}

namespace {

constexpr int kMaxNormH = 16384;
constexpr int kMaxGroupedT = 1 << 27;  // 16 threads a token in one grid dimension

bool norm_kind_ok(int kind) { return kind >= MOE_NORM_NONE && kind <= MOE_NORM_LAYER; }
bool aligned_or_null(const void* p) { return !p || aligned16(p); }

// Whether the n bytes at p and the m bytes at q share any (null or none: no).
bool overlap(const void* p, size_t n, const void* q, size_t m) {
  if (!p || !q || n == 0 || m == 0) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + m && b < a + n;
}
// Buffers that a launch reads or writes, and whether the n bytes at p (which it writes)
// share any with one of them.
struct Span {
  const void* p;
  size_t n;
};
bool overlap_any(const void* p, size_t n, std::initializer_list<Span> others) {
  for (const Span& o : others)
    if (overlap(p, n, o.p, o.n)) return true;
  return false;
}
size_t elem(int dtype) { return dtype == MOE_BF16 ? 2 : 4; }

int check_norm(int rows, int H, float eps, int dtype) {
  if (rows < 1 || H < 1 || !dtype_ok(dtype) || !std::isfinite(eps) || eps < 0.0f)
    return MOE_ERR_INVALID_ARG;
  return H > kMaxNormH ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

int check_grouped(int T, int E, int k, int score, int groups, int topk_groups, int group_top, int renorm,
                  float scale) {
  if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (groups < 1 || topk_groups < 1 || (group_top != 1 && group_top != 2) ||
      (renorm != 0 && renorm != 1) || !std::isfinite(scale))
    return MOE_ERR_INVALID_ARG;
  if (groups > 64 || E % groups != 0 || topk_groups > groups || T > kMaxGroupedT)
    return MOE_ERR_UNSUPPORTED;
  return k > topk_groups * (E / groups) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

int check_linear(int E, int M, int N, int K, int act, bool grouped, int dtype) {
  if (E < 1 || M < 1 || N < 1 || K < 1 || !dtype_ok(dtype) || act < MOE_ACT_NONE ||
      act > MOE_ACT_SWIGLU)
    return MOE_ERR_INVALID_ARG;
  if (E > kMaxExperts || N % 64 != 0 || K % 64 != 0) return MOE_ERR_UNSUPPORTED;
  return moe::linear_fits(E, M, N, K, act, grouped, dtype == MOE_BF16) ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

int run_linear(const void* x, const int32_t* perm, int k, int T, const int32_t* offsets, int E,
               int M, const void* w, const void* bias, int act, const void* residual, int N, int K,
               int dtype, void* y, void* ws, size_t ws_bytes, void* stream) {
  if (!aligned16(x) || !aligned16(w) || !aligned16(y) || !aligned_or_null(bias) ||
      !aligned_or_null(residual) || !aligned_or_null(ws))
    return MOE_ERR_INVALID_ARG;
  // other tiles still read what a tile's outputs or partials would write over
  const size_t b = elem(dtype), ny = (size_t)M * N * b;
  const size_t cols = (size_t)E * (act == MOE_ACT_GEGLU || act == MOE_ACT_SWIGLU ? 2 : 1) * N;
  const Span sx{x, (size_t)(perm ? T : M) * K * b}, sw{w, cols * K * b}, sb{bias, cols * b};
  const Span so{offsets, (size_t)(E + 1) * sizeof(int32_t)}, sp{perm, (size_t)M * sizeof(int32_t)};
  if (overlap_any(y, ny, {sx, sw, sb, so, sp}) || (y != residual && overlap(y, ny, residual, ny)))
    return MOE_ERR_INVALID_ARG;
  const size_t need =
      moe::linear_ws_bytes(E, M, N, K, act, offsets != nullptr, dtype == MOE_BF16);
  if (need > 0 && (!ws || ws_bytes < need)) return MOE_ERR_WORKSPACE;
  if (overlap_any(ws, need, {sx, sw, sb, so, sp, Span{residual, ny}, Span{y, ny}}))
    return MOE_ERR_INVALID_ARG;
  return from_hip(moe::launch_linear(x, perm, k, T, offsets, E, M, N, K, w, bias, act, residual,
                                     dtype == MOE_BF16, y, ws, as_stream(stream)));
}

}  // namespace

int moe_norm(const void* x, const void* weight, const void* bias, int rows, int H, float eps,
             int kind, int dtype, void* out, void* stream) {
  if (!x || !out || !norm_kind_ok(kind) || kind == MOE_NORM_NONE) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(out) || !aligned_or_null(weight) || !aligned_or_null(bias))
    return MOE_ERR_INVALID_ARG;
  const int st = check_norm(rows, H, eps, dtype);
  if (st != MOE_OK) return st;
  const size_t n = (size_t)rows * H * elem(dtype), row = (size_t)H * elem(dtype);
  if ((out != x && overlap(out, n, x, n)) || overlap_any(out, n, {{weight, row}, {bias, row}}))
    return MOE_ERR_INVALID_ARG;
  return from_hip(moe::launch_norm(x, weight, bias, rows, H, eps, kind, dtype == MOE_BF16, out,
                                   as_stream(stream)));
}

int moe_norm_residual(const void* y, int kind, const void* weight, const void* bias,
                      const void* res, const void* gate, int gate_mode, float scale,
                      int next_kind, const void* next_weight, const void* next_bias, int rows,
                      int H, float eps, int dtype, void* res_out, void* next_out, void* stream) {
  if (!y || !res || !res_out || !norm_kind_ok(kind) || !norm_kind_ok(next_kind))
    return MOE_ERR_INVALID_ARG;
  if (gate_mode < MOE_GATE_NONE || gate_mode > MOE_GATE_FULL || !std::isfinite(scale))
    return MOE_ERR_INVALID_ARG;
  if ((gate_mode == MOE_GATE_NONE) != (gate == nullptr)) return MOE_ERR_INVALID_ARG;
  if (kind == MOE_NORM_NONE && (weight || bias)) return MOE_ERR_INVALID_ARG;
  if (next_kind == MOE_NORM_NONE && (next_weight || next_bias)) return MOE_ERR_INVALID_ARG;
  if ((next_kind == MOE_NORM_NONE) != (next_out == nullptr)) return MOE_ERR_INVALID_ARG;
  for (const void* p : {y, weight, bias, res, gate, next_weight, next_bias, (const void*)res_out,
                        (const void*)next_out})
    if (!aligned_or_null(p)) return MOE_ERR_INVALID_ARG;
  const int st = check_norm(rows, H, eps, dtype);
  if (st != MOE_OK) return st;
  const size_t n = (size_t)rows * H * elem(dtype);
  if (overlap(res_out, n, y, n) || overlap(next_out, n, res, n) || overlap(next_out, n, res_out, n) ||
      (res_out != res && overlap(res_out, n, res, n)) || (next_out != y && overlap(next_out, n, y, n)))
    return MOE_ERR_INVALID_ARG;
  // what other rows still read; a full gate is read where it would be written, like res
  const size_t b = elem(dtype), row = H * b;
  const size_t ng = gate_mode == MOE_GATE_FULL ? n : gate_mode == MOE_GATE_TOKEN ? rows * b : row;
  for (const void* out : {(const void*)res_out, (const void*)next_out})
    if (overlap_any(out, n, {{weight, row}, {bias, row}, {next_weight, row}, {next_bias, row}}) ||
        (!(gate_mode == MOE_GATE_FULL && out == gate) && overlap(out, n, gate, ng)))
      return MOE_ERR_INVALID_ARG;
  return from_hip(moe::launch_norm_residual(y, kind, weight, bias, res, gate, gate_mode, scale,
                                            next_kind, next_weight, next_bias, rows, H, eps,
                                            dtype == MOE_BF16, res_out, next_out,
                                            as_stream(stream)));
}

size_t moe_route_grouped_workspace_bytes(int T, int H, int E, int k, int dtype) {
  if (!dtype_ok(dtype) || check_tokens(T, H, E, k) != MOE_OK) return 0;
  return moe::route_grouped_ws_bytes(T, H, E, dtype == MOE_BF16);
}

int moe_route_grouped(const void* x, const void* wg, const float* bias, int T, int H, int E, int k,
                      int score, int groups, int topk_groups, int group_top, int renorm,
                      float scale, int dtype, int32_t* topk_idx, float* topk_w, void* ws,
                      size_t ws_bytes, void* stream) {
  if (!x || !wg || !topk_idx || !topk_w || !dtype_ok(dtype)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(wg) || !aligned_or_null(ws)) return MOE_ERR_INVALID_ARG;
  int st = check_tokens(T, H, E, k);
  if (st != MOE_OK) return st;
  st = check_grouped(T, E, k, score, groups, topk_groups, group_top, renorm, scale);
  if (st != MOE_OK) return st;
  const Span sx{x, (size_t)T * H * elem(dtype)}, sg{wg, (size_t)E * H * elem(dtype)};
  const Span sb{bias, E * sizeof(float)};
  const Span si{topk_idx, (size_t)T * k * sizeof(int32_t)}, sw{topk_w, (size_t)T * k * sizeof(float)};
  if (overlap_any(si.p, si.n, {sx, sg, sb, sw}) || overlap_any(sw.p, sw.n, {sx, sg, sb}))
    return MOE_ERR_INVALID_ARG;
  const size_t need = moe::route_grouped_ws_bytes(T, H, E, dtype == MOE_BF16);
  if (need > 0 && (!ws || ws_bytes < need)) return MOE_ERR_WORKSPACE;
  if (overlap_any(ws, need, {sx, sg, sb, si, sw})) return MOE_ERR_INVALID_ARG;
  return from_hip(moe::launch_route_grouped(x, wg, bias, T, H, E, k, score == MOE_SCORE_SOFTMAX,
                                            groups, topk_groups, group_top, renorm != 0, scale,
                                            dtype == MOE_BF16, topk_idx, topk_w, ws,
                                            as_stream(stream)));
}

size_t moe_linear_workspace_bytes(int M, int N, int K, int act, int dtype) {
  if (check_linear(1, M, N, K, act, false, dtype) != MOE_OK) return 0;
  return moe::linear_ws_bytes(1, M, N, K, act, false, dtype == MOE_BF16);
}

int moe_linear(const void* x, const void* w, const void* bias, int act, const void* residual,
               int M, int N, int K, int dtype, void* y, void* ws, size_t ws_bytes, void* stream) {
  if (!x || !w || !y) return MOE_ERR_INVALID_ARG;
  const int st = check_linear(1, M, N, K, act, false, dtype);
  if (st != MOE_OK) return st;
  return run_linear(x, nullptr, 1, M, nullptr, 1, M, w, bias, act, residual, N, K, dtype, y, ws,
                    ws_bytes, stream);
}

size_t moe_linear_grouped_workspace_bytes(int E, int rows, int N, int K, int act, int dtype) {
  if (check_linear(E, rows, N, K, act, true, dtype) != MOE_OK) return 0;
  return moe::linear_ws_bytes(E, rows, N, K, act, true, dtype == MOE_BF16);
}

int moe_linear_path(int E, int rows, int N, int K, int act, int grouped, int dtype, int* slices) {
  if ((grouped != 0 && grouped != 1) || (grouped == 0 && E != 1)) return MOE_ERR_INVALID_ARG;
  const int st = check_linear(E, rows, N, K, act, grouped != 0, dtype);
  if (st != MOE_OK) return st;
  int n = 1;
  const int path = moe::linear_path(E, rows, N, K, act, grouped != 0, dtype == MOE_BF16, &n);
  if (slices) *slices = n;
  return path;
}

int moe_linear_grouped(const void* x, const int32_t* perm, int k, int T, const int32_t* offsets,
                       int E, int rows, const void* w, const void* bias, int act,
                       const void* residual, int N, int K, int dtype, void* y, void* ws,
                       size_t ws_bytes, void* stream) {
  if (!x || !offsets || !w || !y) return MOE_ERR_INVALID_ARG;
  const int st = check_linear(E, rows, N, K, act, true, dtype);
  if (st != MOE_OK) return st;
  if (perm) {
    if (T < 1 || k < 1) return MOE_ERR_INVALID_ARG;
    if (k > kMaxTopK || (long long)T * k >= (1LL << 31) || rows > (long long)T * k)
      return MOE_ERR_UNSUPPORTED;
  }
  return run_linear(x, perm, k, T, offsets, E, rows, w, bias, act, residual, N, K, dtype, y, ws,
                    ws_bytes, stream);
}

namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
size_t scale_blocks(int n) { return ((size_t)n + 127) / 128; }

int check_quantize(int count, int N, int K, int dtype, const void* x, const void* q,
                   const float* scale, size_t scales) {
  if (!x || !q || !scale || count < 1 || N < 1 || K < 1 || !dtype_ok(dtype)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(q) || !aligned4(scale)) return MOE_ERR_INVALID_ARG;
  if (K % 128 != 0) return MOE_ERR_UNSUPPORTED;
  const size_t n = (size_t)count * N * K;
  const Span sx{x, n * elem(dtype)}, ss{scale, scales * sizeof(float)};
  return overlap_any(q, n, {sx, ss}) || overlap_any(scale, ss.n, {sx}) ? MOE_ERR_INVALID_ARG : MOE_OK;
}

int check_linear_fp8(int E, int M, int N, int K, int act, bool grouped, int gather_rows = 0) {
  if (E < 1 || M < 1 || N < 1 || K < 1 || act < MOE_ACT_NONE || act > MOE_ACT_SWIGLU)
    return MOE_ERR_INVALID_ARG;
  if (E > kMaxExperts || N % 64 != 0 || K % 128 != 0) return MOE_ERR_UNSUPPORTED;
  return moe::linear_fp8_fits(E, M, N, K, act, grouped, gather_rows) ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

int run_linear_fp8(const void* x, const float* x_scale, const int32_t* perm, int k, int T,
                   const int32_t* offsets, int E, int M, const void* w, const float* w_scale,
                   const void* bias, int act, const void* residual, int N, int K, void* y, void* ws,
                   size_t ws_bytes, void* stream) {
  if (!aligned16(x) || !aligned16(w) || !aligned16(y) || !aligned_or_null(bias) ||
      !aligned_or_null(residual) || !aligned_or_null(ws) || !aligned4(x_scale) || !aligned4(w_scale))
    return MOE_ERR_INVALID_ARG;
  const size_t ny = (size_t)M * N * 2, xr = (size_t)(perm ? T : M), nkb = (size_t)K / 128;
  const size_t mats = (size_t)E * (act == MOE_ACT_GEGLU || act == MOE_ACT_SWIGLU ? 2 : 1);
  const Span sx{x, xr * K}, sxs{x_scale, xr * nkb * 4}, sw{w, mats * N * K};
  const Span sws{w_scale, mats * scale_blocks(N) * nkb * 4}, sb{bias, mats * N * 2};
  const Span so{offsets, (size_t)(E + 1) * sizeof(int32_t)}, sp{perm, (size_t)M * sizeof(int32_t)};
  if (overlap_any(y, ny, {sx, sxs, sw, sws, sb, so, sp}) ||
      (y != residual && overlap(y, ny, residual, ny)))
    return MOE_ERR_INVALID_ARG;
  const size_t need = moe::linear_fp8_ws_bytes(E, M, N, K, act, offsets != nullptr);
  if (need > 0 && (!ws || ws_bytes < need)) return MOE_ERR_WORKSPACE;
  if (overlap_any(ws, need, {sx, sxs, sw, sws, sb, so, sp, Span{residual, ny}, Span{y, ny}}))
    return MOE_ERR_INVALID_ARG;
  return from_hip(moe::launch_linear_fp8(x, x_scale, perm, k, T, offsets, E, M, N, K, w, w_scale, bias,
                                         act, residual, y, ws, as_stream(stream)));
}

}  // namespace

int moe_quantize(const void* x, int rows, int K, int dtype, void* q, float* scale, void* stream) {
  const int st = check_quantize(1, rows, K, dtype, x, q, scale, rows < 1 || K < 1 ? 0 : (size_t)rows * (K / 128));
  if (st != MOE_OK) return st;
  if (!moe::quantize_fits(rows, K)) return MOE_ERR_UNSUPPORTED;
  return from_hip(moe::launch_quantize(x, rows, K, dtype == MOE_BF16, q, scale, as_stream(stream)));
}

int moe_quantize_weight(const void* w, int count, int N, int K, int dtype, void* q, float* scale,
                        void* stream) {
  const bool sized = count >= 1 && N >= 1 && K >= 1;
  const int st = check_quantize(count, N, K, dtype, w, q, scale,
                                sized ? (size_t)count * scale_blocks(N) * (K / 128) : 0);
  if (st != MOE_OK) return st;
  if (N % 64 != 0 || !moe::quantize_weight_fits(count, N, K)) return MOE_ERR_UNSUPPORTED;
  return from_hip(moe::launch_quantize_weight(w, count, N, K, dtype == MOE_BF16, q, scale,
                                              as_stream(stream)));
}

size_t moe_linear_fp8_workspace_bytes(int M, int N, int K, int act) {
  if (check_linear_fp8(1, M, N, K, act, false) != MOE_OK) return 0;
  return moe::linear_fp8_ws_bytes(1, M, N, K, act, false);
}

int moe_linear_fp8(const void* x, const float* x_scale, const void* w, const float* w_scale,
                   const void* bias, int act, const void* residual, int M, int N, int K, void* y,
                   void* ws, size_t ws_bytes, void* stream) {
  if (!x || !x_scale || !w || !w_scale || !y) return MOE_ERR_INVALID_ARG;
  const int st = check_linear_fp8(1, M, N, K, act, false);
  if (st != MOE_OK) return st;
  return run_linear_fp8(x, x_scale, nullptr, 1, M, nullptr, 1, M, w, w_scale, bias, act, residual, N, K,
                        y, ws, ws_bytes, stream);
}

size_t moe_linear_grouped_fp8_workspace_bytes(int E, int rows, int N, int K, int act) {
  if (check_linear_fp8(E, rows, N, K, act, true) != MOE_OK) return 0;
  return moe::linear_fp8_ws_bytes(E, rows, N, K, act, true);
}

int moe_linear_grouped_fp8(const void* x, const float* x_scale, const int32_t* perm, int k, int T,
                           const int32_t* offsets, int E, int rows, const void* w,
                           const float* w_scale, const void* bias, int act, const void* residual,
                           int N, int K, void* y, void* ws, size_t ws_bytes, void* stream) {
  if (!x || !x_scale || !offsets || !w || !w_scale || !y) return MOE_ERR_INVALID_ARG;
  const int st = check_linear_fp8(E, rows, N, K, act, true, perm && T > 0 ? T : 0);
  if (st != MOE_OK) return st;
  if (perm) {
    if (T < 1 || k < 1) return MOE_ERR_INVALID_ARG;
    if (k > kMaxTopK || (long long)T * k >= (1LL << 31) || rows > (long long)T * k)
      return MOE_ERR_UNSUPPORTED;
  }
  return run_linear_fp8(x, x_scale, perm, k, T, offsets, E, rows, w, w_scale, bias, act, residual, N,
                        K, y, ws, ws_bytes, stream);
}

int moe_linear_fp8_path(int E, int rows, int N, int K, int act, int grouped, int* slices) {
  if ((grouped != 0 && grouped != 1) || (grouped == 0 && E != 1)) return MOE_ERR_INVALID_ARG;
  const int st = check_linear_fp8(E, rows, N, K, act, grouped != 0);
  if (st != MOE_OK) return st;
  int n = 1;
  const int path = moe::linear_fp8_path(E, rows, N, K, act, grouped != 0, &n);
  if (slices) *slices = n;
  return path;
}

namespace {

constexpr int kMaxFewSize = 1 << 20;
constexpr int kFewRows = 16;  // weight rows that a task reads side by side

int check_few(int T, int H, int E, int k, int F, int Fs, int dtype) {
  if (T < 1 || F < 1 || Fs < 0 || !dtype_ok(dtype)) return MOE_ERR_INVALID_ARG;
  const int st = check_tokens(T, H, E, k);
  if (st != MOE_OK) return st;
  if (T > moe::few_max_tokens() || F % 64 != 0 || Fs % 64 != 0 || H > kMaxFewSize || F > kMaxFewSize ||
      Fs > kMaxFewSize)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

size_t moe_layer_few_workspace_bytes(int T, int H, int E, int k, int F, int Fs, int dtype) {
  if (check_few(T, H, E, k, F, Fs, dtype) != MOE_OK) return 0;
  return moe::few_ws_bytes(T, H, E, k, F, Fs, dtype == MOE_BF16);
}

int moe_layer_few(const void* x, const void* wg, const float* bias, int bias_mode,
                  const void* w_up, const void* w_down, const void* b_up, const void* b_down,
                  const void* ws_up, const void* ws_down, int T, int H, int E, int k, int F, int Fs,
                  int act, int score, int groups, int topk_groups, int group_top, int renorm,
                  float scale, int dtype, void* out, int32_t* topk_idx, float* topk_w, void* ws,
                  size_t ws_bytes, void* stream) {
  if (!x || !wg || !w_up || !w_down || !out || !topk_idx || !topk_w) return MOE_ERR_INVALID_ARG;
  if (act < MOE_ACT_NONE || act > MOE_ACT_SWIGLU ||
      (bias_mode != MOE_BIAS_CHOICE && bias_mode != MOE_BIAS_SCORE))
    return MOE_ERR_INVALID_ARG;
  int st = check_few(T, H, E, k, F, Fs, dtype);
  if (st != MOE_OK) return st;
  st = check_grouped(T, E, k, score, groups, topk_groups, group_top, renorm, scale);
  if (st != MOE_OK) return st;
  if ((Fs > 0) != (ws_up != nullptr) || (Fs > 0) != (ws_down != nullptr)) return MOE_ERR_INVALID_ARG;
  for (const void* p : {x, wg, w_up, w_down, b_up, b_down, ws_up, ws_down, (const void*)out, (const void*)ws})
    if (!aligned_or_null(p)) return MOE_ERR_INVALID_ARG;
  const size_t b = elem(dtype), two = act == MOE_ACT_GEGLU || act == MOE_ACT_SWIGLU ? 2 : 1;
  const size_t e = (size_t)E, t = (size_t)T;
  // a lane's offset of gate and up rows has 32 bits
  if (two == 2 && ((size_t)(F > Fs ? F : Fs) + kFewRows) * H * b > UINT32_MAX) return MOE_ERR_UNSUPPORTED;
  const Span in[] = {{x, t * H * b}, {wg, e * H * b}, {bias, e * 4}, {w_up, e * two * F * H * b},
                     {w_down, e * H * F * b}, {b_up, e * two * F * b}, {b_down, e * H * b},
                     {ws_up, two * Fs * H * b}, {ws_down, (size_t)H * Fs * b}};
  const Span outs[] = {{out, t * H * b}, {topk_idx, t * k * 4}, {topk_w, t * k * 4}};
  for (int i = 0; i < 3; ++i) {
    for (const Span& s : in)
      if (overlap(outs[i].p, outs[i].n, s.p, s.n)) return MOE_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return MOE_ERR_INVALID_ARG;
  }
  const size_t need = moe::few_ws_bytes(T, H, E, k, F, Fs, dtype == MOE_BF16);
  if (!ws || ws_bytes < need) return MOE_ERR_WORKSPACE;
  for (const Span& s : in)
    if (overlap(ws, need, s.p, s.n)) return MOE_ERR_INVALID_ARG;
  for (const Span& s : outs)
    if (overlap(ws, need, s.p, s.n)) return MOE_ERR_INVALID_ARG;
  moe::FewCall c{};
  c.x = x, c.wg = wg, c.bias = bias, c.bias_in_score = bias_mode == MOE_BIAS_SCORE;
  c.up = w_up, c.down = w_down, c.b_up = b_up, c.b_down = b_down, c.s_up = ws_up, c.s_down = ws_down;
  c.T = T, c.H = H, c.E = E, c.k = k, c.F = F, c.Fs = Fs, c.act = act;
  c.softmax = score == MOE_SCORE_SOFTMAX, c.groups = groups, c.topk_groups = topk_groups;
  c.group_top = group_top, c.renorm = renorm != 0, c.scale = scale, c.bf16 = dtype == MOE_BF16;
  c.out = out, c.idx = topk_idx, c.w = topk_w, c.ws = ws;
  return from_hip(moe::launch_few(c, as_stream(stream)));
}

}  // extern "C"
