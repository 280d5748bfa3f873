// What the product kernels share: their arguments, activations and row lookup.
#pragma once

#include "common.hpp"
#include "kernels.hpp"

namespace moe {
namespace lin {

struct LinArgs {
  const void* x;     // [M, K] rows, or [gT, K] token rows with gather
  const void* w;     // [E, N, K] or [E, 2, N, K]
  const void* bias;  // [E, N] or [E, 2, N], or null
  const void* res;   // [M, N] or null
  void* y;           // [M, N]
  const int32_t* offsets;  // [E+1], or null: one segment of all M rows
  const int32_t* gather;   // buffer row p reads token gather[p] / gk, or null
  int gk, gT;
  int E, M, N, K;
  int act;
  float* part;        // split-K partial tiles, or null
  const int4* table;  // big tiles of a grouped launch: tile descriptors (plan.hpp entries)
  int slots;          // big tiles: workgroups of the launch
};

__device__ __forceinline__ bool gated(int act) { return act == kActGeglu || act == kActSwiglu; }

// x / (1 + exp(-x)); the bf16 form has the hardware's exp2 and reciprocal
// (within a few fp32 ulp, far below the bf16 step of the result).
__device__ __forceinline__ float silu_bf16(float a) {
  return a * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(a * -1.44269504f));
}
__device__ __forceinline__ float silu_f32(float a) { return a / (1.0f + expf(-a)); }

template <bool BF16>
__device__ __forceinline__ float activate(int act, float a) {
  if (act == kActGelu || act == kActGeglu) return BF16 ? gelu_bf16(a) : gelu_erf(a);
  if (act == kActSilu || act == kActSwiglu) return BF16 ? silu_bf16(a) : silu_f32(a);
  return a;
}

// Source row in x of buffer row p (perm clamped into [0, T*k): no read leaves x).
__device__ __forceinline__ size_t x_row(const LinArgs& a, int p) {
  if (a.gather == nullptr) return (size_t)p;
  return (size_t)((unsigned)min(max(a.gather[p], 0), a.gT * a.gk - 1) / (unsigned)a.gk);
}

// Big-tile path (linear_big.hip): 256 x 256 tiles.
bool big_ok(const LinArgs& a);           // the shape's offsets fit the kernel's addressing
size_t big_ws_bytes(const LinArgs& a);
hipError_t launch_big(LinArgs a, void* ws, hipStream_t s);

}  // namespace lin
}  // namespace moe
