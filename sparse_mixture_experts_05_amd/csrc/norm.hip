// Norms around a block: the norm in front of it, and behind it the norm of its
// output, gate, residual scale and residual add, with the next block's norm in
// the same pass ("hncyxsy.com Kimi K3 fine-grained MoE" article: the layer's
// output is added to the residual stream; the layer itself returns only the
// MoE output).
//
//   rms:    norm(v) = v / sqrt(mean(v^2) + eps) * w
//   layer:  norm(v) = (v - mu) / sqrt(mean((v - mu)^2) + eps) * w + b
//   moe_norm:          y  = norm(x)
//   moe_norm_residual: r' = r + scale * g * norm(y),  x' = norm_next(r')
//
// Both are bound by memory: one read of every input row and one write of every
// output row. A row stays in the registers of its TR threads (fp32) between
// its loads and its stores, so nothing is read twice: the statistics are sums
// over those registers, the variance is taken around the mean (no E[x^2] -
// mu^2 cancellation), and the next norm works on the fp32 sum r', before its
// rounding to the output type. Each thread loads and stores the same elements
// of a row and loads them all first, so r' may overwrite r and x' may
// overwrite y.
#include <algorithm>

#include "common.hpp"
#include "kernels.hpp"

namespace moe {
namespace {

// VEC consecutive elements at p as fp32, and back with one rounding. 16-byte
// accesses for VEC > 1 (the host picks VEC = 1 where H leaves rows unaligned).
template <int VEC>
__device__ __forceinline__ void load_vec(const uint16_t* p, float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    const u32x4_t q = ld16(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_to_f32(q[i] & 0xffffu);
      v[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = bf16_to_f32(p[i]);
  }
}
template <int VEC>
__device__ __forceinline__ void load_vec(const float* p, float (&v)[VEC]) {
  if constexpr (VEC == 4) {
    const f32x4_t q = *reinterpret_cast<const f32x4_t*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = q[i];
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = p[i];
  }
}
template <int VEC>
__device__ __forceinline__ void store_vec(uint16_t* p, const float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    st16(p, u32x4_t{cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]), cvt_bf16x2(v[4], v[5]),
                    cvt_bf16x2(v[6], v[7])});
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) p[i] = (uint16_t)f32_to_bf16(v[i]);
  }
}
template <int VEC>
__device__ __forceinline__ void store_vec(float* p, const float (&v)[VEC]) {
  if constexpr (VEC == 4) {
    *reinterpret_cast<f32x4_t*>(p) = f32x4_t{v[0], v[1], v[2], v[3]};
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) p[i] = v[i];
  }
}

template <int L>
__device__ __forceinline__ float wave_sum(float v) {
  if constexpr (L < 6) return wave_sum<L + 1>(v + __uint_as_float(partner<L>(__float_as_uint(v))));
  return v;
}

// Sum over the TR threads of a row, in a fixed order (butterfly inside a wave,
// waves in order), the same bits in every thread. red: one slot per wave, of a
// pair of buffers that consecutive calls alternate, so one barrier a call is
// enough: a wave that writes buffer b again has passed the barrier of the call
// in between, and every wave had read b before that one.
template <int TR>
__device__ __forceinline__ float row_sum(float v, float (*red)[TR / 64], int& buf) {
  v = wave_sum<0>(v);
  if constexpr (TR > 64) {
    constexpr int NW = TR / 64;
    if ((threadIdx.x & 63) == 0) red[buf][(threadIdx.x % TR) >> 6] = v;
    lds_barrier();
    v = red[buf][0];
#pragma unroll
    for (int w = 1; w < NW; ++w) v += red[buf][w];
    buf ^= 1;
  }
  return v;
}

// norm of the row held in v (kind MOE_NORM_RMS / MOE_NORM_LAYER). Elements
// past H are never counted and never stored.
template <typename T, int VEC, int TR, int NV>
__device__ __forceinline__ void norm_row(float (&v)[NV][VEC], int kind, const T* w, const T* b,
                                         int H, float eps, int t,
                                         float (*red)[TR / 64], int& buf) {
  if (kind == kNormLayer) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if ((i * TR + t) * VEC < H)
#pragma unroll
        for (int j = 0; j < VEC; ++j) s += v[i][j];
    const float mu = row_sum<TR>(s, red, buf) / (float)H;  // divided: exact for equal elements
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] -= mu;
  }
  float q = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if ((i * TR + t) * VEC < H)
#pragma unroll
      for (int j = 0; j < VEC; ++j) q = fmaf(v[i][j], v[i][j], q);
  const float r = 1.0f / sqrtf(row_sum<TR>(q, red, buf) / (float)H + eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = (i * TR + t) * VEC;
    float wv[VEC], bv[VEC];
    if (w != nullptr && e < H) load_vec<VEC>(w + e, wv);
    if (b != nullptr && e < H) load_vec<VEC>(b + e, bv);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      float o = v[i][j] * r;
      if (w != nullptr) o *= wv[j];
      if (b != nullptr) o += bv[j];
      v[i][j] = o;
    }
  }
}

struct NormArgs {
  const void *x, *w, *b;             // the normed rows, their weight and bias (or null)
  const void *res, *gate;            // residual rows; gate (or null)
  const void *nw, *nb;               // weight and bias of the next norm (or null)
  void *out, *next;                  // norm: the normed rows; residual: r' and x'
  int rows, H, kind, next_kind, gate_mode;
  float eps, scale;
};

// TR threads per row, 256 / TR (at least one) rows per workgroup; the
// workgroups walk the rows with the grid's stride.
template <typename T, int VEC, int TR, int NV, bool RES>
__global__ __launch_bounds__(TR < 256 ? 256 : TR) void norm_kernel(NormArgs a) {
  constexpr int RPB = TR < 256 ? 256 / TR : 1;
  static_assert(TR == 64 || RPB == 1, "a row's threads are a wave or a whole workgroup");
  __shared__ float red[2][TR / 64];
  int buf = 0;
  const int t = threadIdx.x % TR;
  const int H = a.H;
  const T* x = static_cast<const T*>(a.x);
  const T* w = static_cast<const T*>(a.w);
  const T* b = static_cast<const T*>(a.b);
  T* out = static_cast<T*>(a.out);
  for (int row = blockIdx.x * RPB + threadIdx.x / TR; row < a.rows; row += gridDim.x * RPB) {
    const size_t base = (size_t)row * H;
    float v[NV][VEC], r[RES ? NV : 1][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * TR + t) * VEC;
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] = 0.0f;
      if (e < H) load_vec<VEC>(x + base + e, v[i]);
    }
    if constexpr (RES) {
      const T* res = static_cast<const T*>(a.res);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = (i * TR + t) * VEC;
#pragma unroll
        for (int j = 0; j < VEC; ++j) r[i][j] = 0.0f;
        if (e < H) load_vec<VEC>(res + base + e, r[i]);
      }
    }
    if (a.kind != kNormNone) norm_row<T, VEC, TR, NV>(v, a.kind, w, b, H, a.eps, t, red, buf);
    if constexpr (RES) {
      const T* gate = static_cast<const T*>(a.gate);
      const T* g = a.gate_mode == kGateToken ? gate + row
                   : a.gate_mode == kGateFull ? gate + base : gate;
      float gt[1] = {1.0f};
      if (a.gate_mode == kGateToken) load_vec<1>(g, gt);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = (i * TR + t) * VEC;
        float gv[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) gv[j] = gt[0];
        if (a.gate_mode >= kGateChannel && e < H) load_vec<VEC>(g + e, gv);
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[i][j] = fmaf(v[i][j] * gv[j], a.scale, r[i][j]);
        if (e < H) store_vec<VEC>(out + base + e, v[i]);
      }
      if (a.next_kind != kNormNone) {
        norm_row<T, VEC, TR, NV>(v, a.next_kind, static_cast<const T*>(a.nw),
                                 static_cast<const T*>(a.nb), H, a.eps, t, red, buf);
        T* next = static_cast<T*>(a.next);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int e = (i * TR + t) * VEC;
          if (e < H) store_vec<VEC>(next + base + e, v[i]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = (i * TR + t) * VEC;
        if (e < H) store_vec<VEC>(out + base + e, v[i]);
      }
    }
  }
}

template <typename T, int VEC, int TR, int NV, bool RES>
hipError_t run_norm(const NormArgs& a, hipStream_t s) {
  constexpr int RPB = TR < 256 ? 256 / TR : 1;
  const int blocks = std::min((a.rows + RPB - 1) / RPB, 256 * 8);
  hipLaunchKernelGGL((norm_kernel<T, VEC, TR, NV, RES>), dim3(blocks), dim3(TR < 256 ? 256 : TR), 0,
                     s, a);
  return hipGetLastError();
}

// Vectors per thread: the smallest of 1, 2, 4, 8 that hold the row in TR
// threads (H <= 16384: TR = 1024 holds it with 16 single elements).
template <typename T, int VEC, int TR, bool RES>
hipError_t run_norm_tr(const NormArgs& a, hipStream_t s) {
  const int n = (a.H + VEC * TR - 1) / (VEC * TR);
  if (n <= 1) return run_norm<T, VEC, TR, 1, RES>(a, s);
  if (n <= 2) return run_norm<T, VEC, TR, 2, RES>(a, s);
  if (n <= 4) return run_norm<T, VEC, TR, 4, RES>(a, s);
  if (n <= 8) return run_norm<T, VEC, TR, 8, RES>(a, s);
  if constexpr (VEC == 1) return run_norm<T, VEC, TR, 16, RES>(a, s);
  return hipErrorInvalidValue;
}

template <typename T, int VEC, bool RES>
hipError_t run_norm_vec(const NormArgs& a, hipStream_t s) {
  const int vecs = (a.H + VEC - 1) / VEC;
  if (vecs <= 64 * 2) return run_norm_tr<T, VEC, 64, RES>(a, s);
  if constexpr (VEC < 8) {  // 16384 elements are 2048 vectors of 8
    if (vecs > 256 * 8) return run_norm_tr<T, VEC, 1024, RES>(a, s);
  }
  return run_norm_tr<T, VEC, 256, RES>(a, s);
}

template <bool RES>
hipError_t run_norm_dtype(const NormArgs& a, bool bf16, hipStream_t s) {
  if (bf16)
    return a.H % 8 == 0 ? run_norm_vec<uint16_t, 8, RES>(a, s) : run_norm_vec<uint16_t, 1, RES>(a, s);
  return a.H % 4 == 0 ? run_norm_vec<float, 4, RES>(a, s) : run_norm_vec<float, 1, RES>(a, s);
}

}  // namespace

hipError_t launch_norm(const void* x, const void* w, const void* b, int rows, int H, float eps,
                       int kind, bool bf16, void* out, hipStream_t s) {
  NormArgs a{};
  a.x = x, a.w = w, a.b = b, a.out = out;
  a.rows = rows, a.H = H, a.kind = kind, a.eps = eps;
  return run_norm_dtype<false>(a, bf16, s);
}

hipError_t launch_norm_residual(const void* y, int kind, const void* w, const void* b,
                                const void* res, const void* gate, int gate_mode, float scale,
                                int next_kind, const void* nw, const void* nb, int rows, int H,
                                float eps, bool bf16, void* res_out, void* next_out,
                                hipStream_t s) {
  NormArgs a{};
  a.x = y, a.w = w, a.b = b, a.res = res, a.gate = gate, a.nw = nw, a.nb = nb;
  a.out = res_out, a.next = next_out;
  a.rows = rows, a.H = H, a.kind = kind, a.next_kind = next_kind, a.gate_mode = gate_mode;
  a.eps = eps, a.scale = scale;
  return run_norm_dtype<true>(a, bf16, s);
}

}  // namespace moe
