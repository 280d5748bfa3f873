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

// VEC consecutive elements as they lie in memory: 16 bytes at any element's address
// (rows whose length is no multiple of VEC start unaligned, which global loads and
// stores take), or one element for rows shorter than that. Loads are issued raw, from
// addresses clamped into the row, and widened when they are used: a widening next to
// its load, or a load under a branch, would wait for each load in turn.
typedef u32x4_t u32x4_any_t __attribute__((aligned(2)));
template <typename T, int VEC>
struct Raw {
  u32x4_t q;
};
template <typename T>
struct Raw<T, 1> {
  T q;
};
template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> load_raw(const T* p) {
  Raw<T, VEC> r;
  if constexpr (VEC == 1) r.q = *p;
  else r.q = *reinterpret_cast<const u32x4_any_t*>(p);
  return r;
}
template <int VEC>
__device__ __forceinline__ void widen(const Raw<uint16_t, VEC>& r, float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    v[0] = bf16_to_f32(r.q);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_to_f32(r.q[i] & 0xffffu);
      v[2 * i + 1] = __uint_as_float(r.q[i] & 0xffff0000u);
    }
  }
}
template <int VEC>
__device__ __forceinline__ void widen(const Raw<float, VEC>& r, float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    v[0] = r.q;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r.q[i]);
  }
}
// Stores v[skip ..] at p + skip ..
template <int VEC>
__device__ __forceinline__ void store_vec(uint16_t* p, const float (&v)[VEC], int skip) {
  if constexpr (VEC == 8) {
    if (skip == 0) {
      *reinterpret_cast<u32x4_any_t*>(p) = u32x4_t{cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]),
                                                   cvt_bf16x2(v[4], v[5]), cvt_bf16x2(v[6], v[7])};
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < VEC; ++j)
    if (j >= skip) p[j] = (uint16_t)f32_to_bf16(v[j]);
}
template <int VEC>
__device__ __forceinline__ void store_vec(float* p, const float (&v)[VEC], int skip) {
  if constexpr (VEC == 4) {
    if (skip == 0) {
      *reinterpret_cast<u32x4_any_t*>(p) = u32x4_t{__float_as_uint(v[0]), __float_as_uint(v[1]),
                                                   __float_as_uint(v[2]), __float_as_uint(v[3])};
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < VEC; ++j)
    if (j >= skip) p[j] = v[j];
}

// Vector i of thread t covers the elements [e, e + VEC), e = (i * TR + t) * VEC. The
// one that would pass the end of the row is loaded at H - VEC instead; its first
// `skip` elements then belong to the vector before it (all of them past the end) and
// are neither counted nor stored here. The host takes the fewest vectors NV per thread
// that hold the row, so those below NV / 2 are whole.
template <int VEC, int TR, int NV>
__device__ __forceinline__ int vec_start(int i, int t, int H) {
  const int e = (i * TR + t) * VEC;
  return i < NV / 2 ? e : min(e, H - VEC);
}
template <int VEC, int TR, int NV>
__device__ __forceinline__ int vec_skip(int i, int t, int H) {
  return i < NV / 2 ? 0 : max((i * TR + t) * VEC - (H - VEC), 0);
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

// The vectors of a row-long array that this thread holds (null: none).
template <typename T, int VEC, int TR, int NV>
struct RowRaw {
  Raw<T, VEC> r[NV];
  __device__ __forceinline__ void load(const T* p, int H, int t) {
#pragma unroll
    for (int i = 0; i < NV; ++i) r[i] = load_raw<T, VEC>(p + vec_start<VEC, TR, NV>(i, t, H));
  }
};

// norm of the row held in v (kind kNormRms / kNormLayer), whose weight and bias are
// on their way in w and b.
template <typename T, int VEC, int TR, int NV>
__device__ __forceinline__ void norm_row(float (&v)[NV][VEC], int kind, bool has_w, bool has_b,
                                         const RowRaw<T, VEC, TR, NV>& w,
                                         const RowRaw<T, VEC, TR, NV>& b, int H, float eps, int t,
                                         float (*red)[TR / 64], int& buf) {
  if (kind == kNormLayer) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) s += j >= vec_skip<VEC, TR, NV>(i, t, H) ? v[i][j] : 0.0f;
    const float mu = row_sum<TR>(s, red, buf) / (float)H;  // divided: exact for equal elements
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] -= mu;
  }
  float q = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float x = j >= vec_skip<VEC, TR, NV>(i, t, H) ? v[i][j] : 0.0f;
      q = fmaf(x, x, q);
    }
  const float r = 1.0f / sqrtf(row_sum<TR>(q, red, buf) / (float)H + eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float wv[VEC], bv[VEC];
    widen<VEC>(w.r[i], wv);
    widen<VEC>(b.r[i], bv);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      float o = v[i][j] * r;
      if (has_w) o *= wv[j];
      if (has_b) o += bv[j];
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

// TR threads per row, 256 / TR (at least one) rows per workgroup. One row each: in
// a loop over rows the next row's loads wait for this one's stores (16384 x 4096
// bf16: 2048 workgroups walking the rows 63 us, one row each 53 us).
template <typename T, int VEC, int TR, int NV, bool RES>
__global__ __launch_bounds__(TR < 256 ? 256 : TR) void norm_kernel(NormArgs a) {
  constexpr int RPB = TR < 256 ? 256 / TR : 1;
  static_assert(TR == 64 || RPB == 1, "a row's threads are a wave or a whole workgroup");
  using Row = RowRaw<T, VEC, TR, NV>;
  __shared__ float red[2][TR / 64];
  int buf = 0;
  const int t = threadIdx.x % TR;
  const int H = a.H;
  const long long row = ((long long)blockIdx.y * gridDim.x + blockIdx.x) * RPB + threadIdx.x / TR;
  if (row >= a.rows) return;  // whole workgroups, or whole waves where there is no barrier
  const size_t base = (size_t)row * H;
  const T* w = static_cast<const T*>(a.w);
  const T* b = static_cast<const T*>(a.b);
  const T* x = static_cast<const T*>(a.x) + base;
  // every load of the row first; arrays that are not there read the row itself
  Row rx, rw, rb;
  rx.load(x, H, t);
  float v[NV][VEC];
  if constexpr (!RES) {
    rw.load(w != nullptr ? w : x, H, t);
    rb.load(b != nullptr ? b : x, H, t);
#pragma unroll
    for (int i = 0; i < NV; ++i) widen<VEC>(rx.r[i], v[i]);
    norm_row<T, VEC, TR, NV>(v, a.kind, w != nullptr, b != nullptr, rw, rb, H, a.eps, t, red, buf);
  } else {
    const T* gate = static_cast<const T*>(a.gate);
    const T* nw = static_cast<const T*>(a.nw);
    const T* nb = static_cast<const T*>(a.nb);
    const bool gv = a.gate_mode >= kGateChannel;
    Row rr, rg, rnw, rnb;
    rr.load(static_cast<const T*>(a.res) + base, H, t);
    if (w != nullptr) rw.load(w, H, t);
    if (b != nullptr) rb.load(b, H, t);
    if (gv) rg.load(a.gate_mode == kGateFull ? gate + base : gate, H, t);
    constexpr bool kLate = TR == 1024;  // 128 registers a thread: they would spill
    if (!kLate && nw != nullptr) rnw.load(nw, H, t);
    if (!kLate && nb != nullptr) rnb.load(nb, H, t);
    float g1[1] = {1.0f};
    if (a.gate_mode == kGateToken) widen<1>(load_raw<T, 1>(gate + row), g1);
#pragma unroll
    for (int i = 0; i < NV; ++i) widen<VEC>(rx.r[i], v[i]);
    if (a.kind != kNormNone)
      norm_row<T, VEC, TR, NV>(v, a.kind, w != nullptr, b != nullptr, rw, rb, H, a.eps, t, red, buf);
    T* out = static_cast<T*>(a.out) + base;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float r[VEC], g[VEC];
      widen<VEC>(rr.r[i], r);
      if (gv) widen<VEC>(rg.r[i], g);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] = fmaf(v[i][j] * (gv ? g[j] : g1[0]), a.scale, r[j]);
      store_vec<VEC>(out + vec_start<VEC, TR, NV>(i, t, H), v[i], vec_skip<VEC, TR, NV>(i, t, H));
    }
    if (a.next_kind == kNormNone) return;
    if (kLate && nw != nullptr) rnw.load(nw, H, t);
    if (kLate && nb != nullptr) rnb.load(nb, H, t);
    norm_row<T, VEC, TR, NV>(v, a.next_kind, nw != nullptr, nb != nullptr, rnw, rnb, H, a.eps, t, red,
                             buf);
  }
  T* last = static_cast<T*>(RES ? a.next : a.out) + base;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    store_vec<VEC>(last + vec_start<VEC, TR, NV>(i, t, H), v[i], vec_skip<VEC, TR, NV>(i, t, H));
}

template <typename T, int VEC, int TR, int NV, bool RES>
hipError_t run_norm(const NormArgs& a, hipStream_t s) {
  constexpr int RPB = TR < 256 ? 256 / TR : 1;
  // a grid dimension holds less than 2^32 threads: a second one for very many rows
  const unsigned blocks = ((unsigned)a.rows + RPB - 1) / RPB, nx = std::min(blocks, 1u << 20);
  hipLaunchKernelGGL((norm_kernel<T, VEC, TR, NV, RES>), dim3(nx, (blocks + nx - 1) / nx),
                     dim3(TR < 256 ? 256 : TR), 0, s, a);
  return hipGetLastError();
}

// Threads per row: a wave up to 2 vectors a lane, 256 threads up to 4, else 1024
// (16384 elements, the longest row, are 2048 vectors of 8 or 4096 of 4). Vectors per
// thread: the fewest of 1, 2, 4 that hold the row.
template <typename T, int VEC, bool RES>
hipError_t run_norm_vec(const NormArgs& a, hipStream_t s) {
  const int vecs = (a.H + VEC - 1) / VEC;
  if (vecs <= 64) return run_norm<T, VEC, 64, 1, RES>(a, s);
  if constexpr (VEC > 1) {
    if (vecs <= 64 * 2) return run_norm<T, VEC, 64, 2, RES>(a, s);
    if (vecs <= 256) return run_norm<T, VEC, 256, 1, RES>(a, s);
    if (vecs <= 256 * 2) return run_norm<T, VEC, 256, 2, RES>(a, s);
    if (vecs <= 256 * 4) return run_norm<T, VEC, 256, 4, RES>(a, s);
    if (vecs <= 1024 * 2) return run_norm<T, VEC, 1024, 2, RES>(a, s);
    if constexpr (VEC == 4) {
      if (vecs <= 1024 * 4) return run_norm<T, VEC, 1024, 4, RES>(a, s);
    }
  }
  return hipErrorInvalidValue;
}

template <bool RES>
hipError_t run_norm_dtype(const NormArgs& a, bool bf16, hipStream_t s) {
  if (bf16) return a.H >= 8 ? run_norm_vec<uint16_t, 8, RES>(a, s) : run_norm_vec<uint16_t, 1, RES>(a, s);
  return a.H >= 4 ? run_norm_vec<float, 4, RES>(a, s) : run_norm_vec<float, 1, RES>(a, s);
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
