// Host-side launchers of the MoE layer kernels (internal to the library).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

size_t route_ws_bytes(int T, int H, int E, bool bf16, bool prob);
hipError_t launch_route(const void* x, const void* wg, const float* bias, int T, int H, int E,
                        int k, bool bf16, int32_t* topk_idx, float* topk_w, float* prob_mean,
                        void* ws, hipStream_t s);

int dispatch_blocks(int T, int k);
size_t dispatch_ws_bytes(int T, int E, int k);
hipError_t launch_dispatch(const int32_t* topk_idx, const void* x, int T, int H, int E, int k,
                           int cap, bool bf16, int32_t* counts, int32_t* offsets, int32_t* perm,
                           int32_t* inv, void* xs, void* ws, hipStream_t s);

size_t noalloc_scratch_bytes();
hipError_t launch_dispatch_noalloc(const int32_t* topk_idx, const void* x, int T, int H, int E,
                                   int k, bool bf16, int32_t* counts, int32_t* offsets,
                                   int32_t* perm, int32_t* inv, void* xs, hipStream_t s);

size_t ffn_ws_bytes(int rows, int T, int E, int H, int F, int Fs, bool bf16);
hipError_t launch_expert_ffn(const void* xs, const int32_t* gather, int gk,
                             const int32_t* offsets, int rows, int E, int H, int F, const void* w1,
                             const void* w2, const void* x, const void* ws1, const void* ws2,
                             int T, int Fs, bool bf16, void* ys, void* ysh, void* ws,
                             hipStream_t s, void* const* events = nullptr);

hipError_t launch_combine(const void* ys, const int32_t* inv, const float* topk_w,
                          const void* ysh, int T, int H, int k, bool bf16, void* out,
                          hipStream_t s);

hipError_t launch_load_stats(const int32_t* counts, int T, int E, int k, double cf,
                             void* stats, int32_t* overflow, int32_t* straggler_ids,
                             hipStream_t s);

// The enumerations of moe.h (moe_norm_kind, moe_gate_mode, moe_act).
enum { kNormNone = 0, kNormRms = 1, kNormLayer = 2 };
enum { kGateNone = 0, kGateToken = 1, kGateChannel = 2, kGateFull = 3 };
enum { kActNone = 0, kActGelu = 1, kActSilu = 2, kActGeglu = 3, kActSwiglu = 4 };

hipError_t launch_norm(const void* x, const void* w, const void* b, int rows, int H, float eps,
                       int kind, bool bf16, void* out, hipStream_t s);
hipError_t launch_norm_residual(const void* y, int kind, const void* w, const void* b,
                                const void* res, const void* gate, int gate_mode, float scale,
                                int next_kind, const void* nw, const void* nb, int rows, int H,
                                float eps, bool bf16, void* res_out, void* next_out,
                                hipStream_t s);

size_t route_grouped_ws_bytes(int T, int H, int E, bool bf16);
hipError_t launch_route_grouped(const void* x, const void* wg, const float* bias, int T, int H,
                                int E, int k, bool softmax, int groups, int topk_groups,
                                int group_top, bool renorm, float scale, bool bf16,
                                int32_t* topk_idx, float* topk_w, void* ws, hipStream_t s);

// Whether every launch of the shape fits one grid.
bool linear_fits(int E, int M, int N, int K, int act, bool grouped, bool bf16);
size_t linear_ws_bytes(int E, int M, int N, int K, int act, bool grouped, bool bf16);
// The product's moe_path and K slices (0: the offsets decide).
int linear_path(int E, int M, int N, int K, int act, bool grouped, bool bf16, int* slices);
hipError_t launch_linear(const void* x, const int32_t* gather, int gk, int gT,
                         const int32_t* offsets, int E, int M, int N, int K, const void* w,
                         const void* bias, int act, const void* res, bool bf16, void* y, void* ws,
                         hipStream_t s);

bool quantize_fits(int rows, int K);
bool quantize_weight_fits(int count, int N, int K);
hipError_t launch_quantize(const void* x, int rows, int K, bool bf16, void* q, float* scale,
                           hipStream_t s);
hipError_t launch_quantize_weight(const void* w, int count, int N, int K, bool bf16, void* q,
                                  float* scale, hipStream_t s);

// gather_rows: rows that perm gathers from (0: none).
bool linear_fp8_fits(int E, int M, int N, int K, int act, bool grouped, int gather_rows);
size_t linear_fp8_ws_bytes(int E, int M, int N, int K, int act, bool grouped);
int linear_fp8_path(int E, int M, int N, int K, int act, bool grouped, int* slices);
hipError_t launch_linear_fp8(const void* x, const float* x_scale, const int32_t* gather, int gk,
                             int gT, const int32_t* offsets, int E, int M, int N, int K,
                             const void* w, const float* w_scale, const void* bias, int act,
                             const void* res, void* y, void* ws, hipStream_t s);

// Arguments of the few-token layer (moe_layer_few, after its checks).
struct FewCall {
  const void *x, *wg;
  const float* bias;
  bool bias_in_score;
  const void *up, *down, *b_up, *b_down, *s_up, *s_down;
  int T, H, E, k, F, Fs, act;
  bool softmax;
  int groups, topk_groups, group_top;
  bool renorm;
  float scale;
  bool bf16;
  void* out;
  int32_t* idx;
  float* w;
  void* ws;
};
int few_max_tokens();
size_t few_ws_bytes(int T, int H, int E, int k, int F, int Fs, bool bf16);
hipError_t launch_few(const FewCall& c, hipStream_t s);

hipError_t launch_bias_update(const int32_t* counts, int E, float gamma, float* bias,
                              float* load_frac, hipStream_t s);

}  // namespace moe
