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
  int tiles;          // 64 x 64 and few-row tiles: at most this many (sizes the partials)
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

// GeLU for bf16 outputs as gelu_bf16 (common.hpp): max(a, 0) - u Phi(-u), u = min(|a|, 6),
// Phi(-u) = 2^p(u), with p of degree 9 (csrc/gelu_fit.py: |p - log2 Phi(-u)| <= 1.45e-6).
// The result is within 4e-6 relative, less than the product's own sum is off for most K;
// degree 6 (5e-5) turned 0.36 % of the bf16 roundings over, this 0.03 % with the sums'
// (700 x 1024 x 2048), as SiLU. Past |a| = 6 it is within 6e-9. Three FMAs an output more:
// 4096^3 106.5 -> 108, 8192 x 8192 x 512 111 -> 116 us.
__device__ __forceinline__ float gelu_product(float a) {
  const float u = __builtin_amdgcn_fmed3f(fabsf(a), 0.0f, 6.0f);
  float p = fmaf(4.99055517e-08f, u, -1.35485152e-06f);
  p = fmaf(p, u, 1.34466763e-05f);
  p = fmaf(p, u, -3.10109026e-05f);
  p = fmaf(p, u, -0.000604944478f);
  p = fmaf(p, u, 0.00783951487f);
  p = fmaf(p, u, -0.0531952716f);
  p = fmaf(p, u, -0.458898306f);
  p = fmaf(p, u, -1.1511575f);
  p = fmaf(p, u, -0.999998569f);
  const float q = __builtin_amdgcn_exp2f(p);
  const float r = !(a <= 0.0f) ? a : 0.0f;  // a NaN passes through
  return fmaf(-u, q, r);
}

template <bool BF16>
__device__ __forceinline__ float activate(int act, float a) {
  if (act == kActGelu || act == kActGeglu) return BF16 ? gelu_product(a) : gelu_erf(a);
  if (act == kActSilu || act == kActSwiglu) return BF16 ? silu_bf16(a) : silu_f32(a);
  return a;
}

// Source row in x of buffer row p (perm clamped into [0, T*k): no read leaves x).
__device__ __forceinline__ size_t x_row(const LinArgs& a, int p) {
  if (a.gather == nullptr) return (size_t)p;
  return (size_t)((unsigned)min(max(a.gather[p], 0), a.gT * a.gk - 1) / (unsigned)a.gk);
}

// Output of one lane: 4 consecutive columns of a row (bf16, 8-byte aligned).
struct Out4 {
  float v[4];
};
__device__ __forceinline__ Out4 widen4(uint2 q) {
  return Out4{{bf16_to_f32(q.x & 0xffffu), __uint_as_float(q.x & 0xffff0000u),
               bf16_to_f32(q.y & 0xffffu), __uint_as_float(q.y & 0xffff0000u)}};
}

// act(g + bg) [* (u + bu)] [+ res] of 4 columns (no bias: zeros).
template <bool BF16>
__device__ __forceinline__ Out4 finish4(int act, const f32x4_t& g, const f32x4_t& u, const Out4& bg,
                                        const Out4& bu, bool has_res, const Out4& res) {
  Out4 o;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    float x = activate<BF16>(act, g[c] + bg.v[c]);
    if (gated(act)) x *= u[c] + bu.v[c];
    if (has_res) x += res.v[c];
    o.v[c] = x;
  }
  return o;
}
__device__ __forceinline__ uint2 pack4(const Out4& o) {
  return make_uint2(cvt_bf16x2(o.v[0], o.v[1]), cvt_bf16x2(o.v[2], o.v[3]));
}

// 4 elements of T at p.
__device__ __forceinline__ Out4 load4(const uint16_t* p) { return widen4(*reinterpret_cast<const uint2*>(p)); }
__device__ __forceinline__ Out4 load4(const float* p) {
  const f32x4_t v = *reinterpret_cast<const f32x4_t*>(p);
  return Out4{{v[0], v[1], v[2], v[3]}};
}

// Bias and residual of the 4 columns c .. c + 3 of buffer row `row`, then finish4
// and the store. e: the row's expert.
template <typename T>
__device__ __forceinline__ void store4(const LinArgs& a, int e, size_t row, int c,
                                       const f32x4_t& g, const f32x4_t& u) {
  constexpr bool BF16 = sizeof(T) == 2;
  const bool gt = gated(a.act);
  Out4 bg{}, bu{}, rv{};
  if (a.bias != nullptr) {
    const T* b = static_cast<const T*>(a.bias) + (size_t)e * (gt ? 2 : 1) * a.N + c;
    bg = load4(b);
    if (gt) bu = load4(b + a.N);
  }
  const size_t at = row * a.N + c;
  if (a.res != nullptr) rv = load4(static_cast<const T*>(a.res) + at);
  const Out4 o = finish4<BF16>(a.act, g, u, bg, bu, a.res != nullptr, rv);
  T* y = static_cast<T*>(a.y) + at;
  if constexpr (BF16) *reinterpret_cast<uint2*>(y) = pack4(o);
  else *reinterpret_cast<f32x4_t*>(y) = f32x4_t{o.v[0], o.v[1], o.v[2], o.v[3]};
}

// Big-tile path (linear_big.hip): 256 rows x 256 weight rows, or half as many
// weight rows.
bool big_ok(const LinArgs& a);         // the shape's offsets fit the kernel's addressing
bool big_gather_ok(const LinArgs& a);  // and those of the gathered rows
size_t big_ws_bytes(const LinArgs& a, bool half);
int big_slices(const LinArgs& a, bool half);  // K slices of the last round's tiles (0: by the offsets)
hipError_t launch_big(LinArgs a, bool half, void* ws, hipStream_t s);

}  // namespace lin
}  // namespace moe
