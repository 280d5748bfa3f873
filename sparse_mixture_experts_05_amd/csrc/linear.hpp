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

struct LinTile {
  int e, row0, M, n0;  // expert; first buffer row and rows of the tile; first output column
  int q;               // number of the tile
};

// Row tile `mt` of BM rows of the segments: each wave finds it for itself (no
// barrier): lane l sums the row tiles of experts 4 l .. 4 l + 3, a wave scan
// orders the lanes. Segments are clamped into the buffer, whatever the offsets
// hold. total: all row tiles.
struct SegScan {
  int off[4], cnt[4], nb[4];
  int incl, total;
};
template <int BM>
__device__ __forceinline__ void scan_segments(const LinArgs& a, SegScan& s) {
  const int lane = threadIdx.x & 63;
  int sum = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int e = lane * 4 + j;
    s.off[j] = s.cnt[j] = 0;
    if (e < a.E) {
      s.off[j] = min(max(a.offsets[e], 0), a.M);
      s.cnt[j] = min(max(a.offsets[e + 1], s.off[j]), a.M) - s.off[j];
    }
    s.nb[j] = (s.cnt[j] + BM - 1) / BM;
    sum += s.nb[j];
  }
  s.incl = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(s.incl, d);
    if (lane >= d) s.incl += v;
  }
  s.total = __shfl(s.incl, 63);
}

// Number `local` of a segment's tiles, nm row tiles by ntn column tiles: blocks of GN
// column tiles, row tile by row tile inside a block (GN = 1: column tile by column
// tile). Returns (row tile, column tile).
template <int GN>
__device__ __forceinline__ int2 order_tile(int local, int nm, int ntn) {
  if constexpr (GN == 1) return make_int2(local % nm, local / nm);
  const int blk = local / (nm * GN), li = local - blk * nm * GN;
  const int w = min(GN, ntn - blk * GN);
  return make_int2(li / w, blk * GN + li % w);
}

// The tile of this workgroup, BM rows x bnc output columns. Tiles are numbered
// segment by segment, in a segment by order_tile, and XCD
// x (workgroups x, x + 8, ...) takes a contiguous run of them: the tiles that
// share a weight panel run on one XCD at about one time. M = 0: no work.
template <int BM, int GN = 1>
__device__ __forceinline__ LinTile lin_tile(const LinArgs& a, int bnc) {
  LinTile t{};
  const int ntn = (a.N + bnc - 1) / bnc;
  const int g = blockIdx.x;
  if (a.offsets == nullptr) {
    const int nm = (a.M + BM - 1) / BM;
    const long long total = (long long)nm * ntn;
    const int chunk = (int)((total + 7) / 8);
    const long long q = (long long)(g & 7) * chunk + (g >> 3);
    if ((g >> 3) >= chunk || q >= total) return t;
    t.e = 0;
    t.q = (int)q;
    const int2 at = order_tile<GN>(t.q, nm, ntn);
    t.row0 = at.x * BM;
    t.n0 = at.y * bnc;
    const int left = a.M - t.row0;
    t.M = left < BM ? left : BM;
    return t;
  }
  SegScan s;
  scan_segments<BM>(a, s);
  // offsets that overlap could name more tiles than the launch has room for: the rest is
  // left out
  const long long total = min((long long)s.total * ntn, (long long)a.tiles);
  const int chunk = (int)((total + 7) / 8);
  const long long q = (long long)(g & 7) * chunk + (g >> 3);
  if ((g >> 3) >= chunk || q >= total) return t;
  const int lane = threadIdx.x & 63;
  int excl = s.incl;
#pragma unroll
  for (int j = 0; j < 4; ++j) excl -= s.nb[j];
  const bool mine = q >= (long long)excl * ntn && q < (long long)s.incl * ntn;
  const int src = __ffsll((unsigned long long)__ballot(mine)) - 1;
  int e = 0, off = 0, cnt = 0, nb = 1, base = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (mine && q >= (long long)excl * ntn && q < (long long)(excl + s.nb[j]) * ntn)
      e = lane * 4 + j, off = s.off[j], cnt = s.cnt[j], nb = s.nb[j], base = excl;
    excl += s.nb[j];
  }
  e = __shfl(e, src), off = __shfl(off, src), cnt = __shfl(cnt, src);
  nb = __shfl(nb, src), base = __shfl(base, src);
  const int2 at = order_tile<GN>((int)(q - (long long)base * ntn), nb, ntn);
  t.e = e;
  t.q = (int)q;
  t.row0 = off + at.x * BM;
  const int left = cnt - at.x * BM;
  t.M = left < BM ? left : BM;
  t.n0 = at.y * bnc;
  return t;
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
// ACT: the act where it is known when compiling.
template <typename T, int ACT = -1>
__device__ __forceinline__ void store4(const LinArgs& a, int e, size_t row, int c,
                                       const f32x4_t& g, const f32x4_t& u) {
  constexpr bool BF16 = sizeof(T) == 2;
  const int act = ACT >= 0 ? ACT : a.act;
  const bool gt = gated(act);
  Out4 bg{}, bu{}, rv{};
  if (a.bias != nullptr) {
    const T* b = static_cast<const T*>(a.bias) + (size_t)e * (gt ? 2 : 1) * a.N + c;
    bg = load4(b);
    if (gt) bu = load4(b + a.N);
  }
  const size_t at = row * a.N + c;
  if (a.res != nullptr) rv = load4(static_cast<const T*>(a.res) + at);
  const Out4 o = finish4<BF16>(act, g, u, bg, bu, a.res != nullptr, rv);
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
