// Matrix product with bias, activation, gate and residual in its epilogue,
// dense and over the experts' ragged segments ("lpqz.cn MoE engineering blog"
// section 3.1: an expert is a pair of Linear layers with an activation between
// them; gated experts multiply the activated half by a second product).
//
//   a = x . W^T + bias
//   y = act(a) + residual                  W [N, K], bias [N]
//   y = act(a_0) * a_1 + residual          W [2, N, K], bias [2, N] (gated acts)
//
// x rows: row p of the buffer, or the token perm[p] / k; in the grouped form
// row p takes the weights and bias of the expert whose segment
// [offsets[e], offsets[e+1]) holds it. Everything from the product's fp32
// accumulator to the store happens in fp32, with one rounding to the output
// type.
#include <algorithm>

#include "common.hpp"
#include "kernels.hpp"
#include "linear.hpp"

namespace moe {
namespace {

using namespace lin;

constexpr int kThreads = 256;

// Weight row of row r of a tile of interleaved gate and up rows whose first
// output column is n0: rows 4q, 4q+1 are the gate rows of columns n0 + 2q,
// n0 + 2q + 1 and rows 4q+2, 4q+3 their up rows, so the 4 consecutive rows a
// lane accumulates hold both factors of 2 outputs.
__device__ __forceinline__ int gated_row(int r, int n0, int N) {
  return ((r >> 1) & 1) * N + n0 + (r >> 2) * 2 + (r & 1);
}

struct LinTile {
  int e, row0, M, n0;  // expert; first buffer row and rows of the tile; first output column
};

// The tile of this workgroup: row tiles of BM rows, segment by segment, each
// with its column tiles of BNC output columns. False: no work.
template <int BM, int BNC>
__device__ bool lin_tile(const LinArgs& a, LinTile& t) {
  const int ntn = (a.N + BNC - 1) / BNC;
  const int mt = blockIdx.x / ntn;
  t.n0 = (blockIdx.x % ntn) * BNC;
  if (a.offsets == nullptr) {
    t.e = 0;
    t.row0 = mt * BM;
    t.M = min(BM, a.M - t.row0);
    return t.M > 0;
  }
  __shared__ int pre[256];
  __shared__ int sel[3];
  const int tid = threadIdx.x;
  int off = 0, cnt = 0, tiles = 0;
  if (tid < a.E) {
    // clamped: a segment never leaves the buffer, whatever the offsets hold
    off = min(max(a.offsets[tid], 0), a.M);
    cnt = min(max(a.offsets[tid + 1], off), a.M) - off;
    tiles = (cnt + BM - 1) / BM;
  }
  pre[tid] = tiles;
  if (tid == 0) sel[0] = -1;
  __syncthreads();
  for (int d = 1; d < 256; d <<= 1) {
    const int v = tid >= d ? pre[tid - d] : 0;
    __syncthreads();
    pre[tid] += v;
    __syncthreads();
  }
  if (tid < a.E) {
    const int excl = pre[tid] - tiles;
    if (mt >= excl && mt < pre[tid]) {
      sel[0] = tid;
      sel[1] = off + (mt - excl) * BM;
      sel[2] = min(BM, cnt - (mt - excl) * BM);
    }
  }
  __syncthreads();
  t.e = sel[0];
  t.row0 = sel[1];
  t.M = sel[2];
  return t.e >= 0;
}

// Epilogue of 4 accumulators of one row: 4 outputs from column c, or the
// gate and up halves of 2 outputs from column c (gated). bias: the expert's.
__device__ __forceinline__ void store4_bf16(const LinArgs& a, const uint16_t* bias, size_t row,
                                            int c, const f32x4_t& acc) {
  uint16_t* y = static_cast<uint16_t*>(a.y) + row * a.N + c;
  const uint16_t* res = static_cast<const uint16_t*>(a.res);
  if (res != nullptr) res += row * a.N + c;
  if (gated(a.act)) {
    float o[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float g = acc[j], u = acc[2 + j];
      if (bias != nullptr) {
        g += bf16_to_f32(bias[c + j]);
        u += bf16_to_f32(bias[a.N + c + j]);
      }
      o[j] = activate<true>(a.act, g) * u;
      if (res != nullptr) o[j] += bf16_to_f32(res[j]);
    }
    *reinterpret_cast<uint32_t*>(y) = cvt_bf16x2(o[0], o[1]);
  } else {
    float o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float g = acc[j];
      if (bias != nullptr) g += bf16_to_f32(bias[c + j]);
      o[j] = activate<true>(a.act, g);
      if (res != nullptr) o[j] += bf16_to_f32(res[j]);
    }
    *reinterpret_cast<uint2*>(y) = make_uint2(cvt_bf16x2(o[0], o[1]), cvt_bf16x2(o[2], o[3]));
  }
}

// ----------------------------------------------------------------- bf16 tiles

// BM rows x 64 weight rows (64 output columns, or 32 of a gated product), 4
// waves, wave w the weight rows [16 w, 16 w + 16) for all BM rows. Operand
// rows are copied global -> LDS with global_load_lds (8 rows of 128 bytes an
// instruction) into a ring of 3 stages of 64 k; 16-byte chunk c of row r sits
// at slot c ^ ((r >> 1) & 7), so the 16 lanes of a fragment read (16
// consecutive rows, one chunk) touch 16 distinct 4-bank groups.
// v_mfma_f32_16x16x32_bf16 takes the weights as A and the rows as B: lane l
// ends with 4 consecutive weight rows of row l % 16 of x.
template <int BM>
struct LinTileShape {
  static constexpr int BN = 64, NS = 3;
  static constexpr int STAGE = (BM + BN) * 128;
  static constexpr int NI = (BM + BN) / 8 / 4;  // copies per wave per stage
  static_assert((BM + BN) % 32 == 0, "whole copies");
};

template <int BM>
__global__ __launch_bounds__(kThreads) void lin_bf16_kernel(LinArgs a) {
  using Sh = LinTileShape<BM>;
  constexpr int BN = Sh::BN, NS = Sh::NS, STAGE = Sh::STAGE, NI = Sh::NI, SM = BM / 16;
  __shared__ __attribute__((aligned(16))) uint8_t smem[NS * STAGE];
  const bool gt = gated(a.act);
  LinTile t;
  if (!(gt ? lin_tile<BM, BN / 2>(a, t) : lin_tile<BM, BN>(a, t))) return;
  const int N = a.N, K = a.K;
  const uint16_t* x = static_cast<const uint16_t*>(a.x);
  const uint16_t* w = static_cast<const uint16_t*>(a.w) + (size_t)t.e * (gt ? 2 : 1) * N * K;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;

  const uint16_t* src[NI];
  int dst[NI];
#pragma unroll
  for (int q = 0; q < NI; ++q) {
    const int g = wave * NI + q;
    const int r = 8 * g + (lane >> 3);
    const int chunk = (lane & 7) ^ ((r >> 1) & 7);
    const uint16_t* row;
    if (r < BM) row = x + x_row(a, t.row0 + min(r, t.M - 1)) * K;  // rows past the end: its last
    else row = w + (size_t)(gt ? gated_row(r - BM, t.n0, N) : t.n0 + r - BM) * K;
    src[q] = row + chunk * 8;
    dst[q] = g * 1024;
  }
  const int KT = K / 64;
  auto issue = [&](int kt) {
    uint8_t* base = smem + (kt % NS) * STAGE;
#pragma unroll
    for (int q = 0; q < NI; ++q) lds_dma16(src[q] + kt * 64, base + dst[q]);
  };
  f32x4_t acc[SM];
#pragma unroll
  for (int i = 0; i < SM; ++i) acc[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const int fr = (lane & 15) * 128;
  const int sw = (lane >> 1) & 7;  // (row >> 1) & 7 of every fragment row of this lane

#pragma unroll
  for (int st = 0; st < NS - 1; ++st)
    if (st < KT) issue(st);
  for (int kt = 0; kt < KT; ++kt) {
    if (kt + NS - 2 < KT) wait_vmcnt<(NS - 2) * NI>();
    else wait_vmcnt<0>();
    lds_barrier();  // stage kt landed for every wave; stage kt-1 is no longer read
    if (kt + NS - 1 < KT) issue(kt + NS - 1);
    const uint8_t* cur = smem + (kt % NS) * STAGE;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const int slot = ((ks * 4 + (lane >> 4)) ^ sw) * 16;
      const u32x4_t fw = ld16(cur + (BM + wave * 16) * 128 + fr + slot);
#pragma unroll
      for (int i = 0; i < SM; ++i) {
        const u32x4_t fx = ld16(cur + i * 16 * 128 + fr + slot);
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(fw), as_bf16x8(fx), acc[i], 0, 0, 0);
      }
    }
  }
  const uint16_t* bias = a.bias == nullptr ? nullptr
                             : static_cast<const uint16_t*>(a.bias) + (size_t)t.e * (gt ? 2 : 1) * N;
  const int c = t.n0 + (wave * 16 + (lane >> 4) * 4) / (gt ? 2 : 1);
#pragma unroll
  for (int i = 0; i < SM; ++i) {
    const int r = i * 16 + (lane & 15);
    if (r < t.M) store4_bf16(a, bias, (size_t)(t.row0 + r), c, acc[i]);
  }
}

// ----------------------------------------------------------------- fp32

// 64 x 64 tiles of plain FMA (small fp32 layers); the weight rows of a gated
// product interleaved as in the bf16 tiles.
__global__ __launch_bounds__(kThreads) void lin_f32_kernel(LinArgs a) {
  constexpr int BM = 64, BN = 64, BK = 16;
  __shared__ float As[BK][BM + 4];
  __shared__ float Bs[BK][BN + 4];
  const bool gt = gated(a.act);
  LinTile t;
  if (!(gt ? lin_tile<BM, BN / 2>(a, t) : lin_tile<BM, BN>(a, t))) return;
  const int N = a.N, K = a.K;
  const float* w = static_cast<const float*>(a.w) + (size_t)t.e * (gt ? 2 : 1) * N * K;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int lr = tid >> 2, lk = (tid & 3) * 4;  // loader: row, first k of a float4
  const float* ga = static_cast<const float*>(a.x) + x_row(a, t.row0 + min(lr, t.M - 1)) * K + lk;
  const float* gb = w + (size_t)(gt ? gated_row(lr, t.n0, N) : t.n0 + lr) * K + lk;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < K; k0 += BK) {
    const float4 va = *reinterpret_cast<const float4*>(ga + k0);
    const float4 vb = *reinterpret_cast<const float4*>(gb + k0);
    As[lk + 0][lr] = va.x, As[lk + 1][lr] = va.y, As[lk + 2][lr] = va.z, As[lk + 3][lr] = va.w;
    Bs[lk + 0][lr] = vb.x, Bs[lk + 1][lr] = vb.y, Bs[lk + 2][lr] = vb.z, Bs[lk + 3][lr] = vb.w;
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < BK; ++kk) {
      float fa[4], fb[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) fa[i] = As[kk][ty * 4 + i];
#pragma unroll
      for (int j = 0; j < 4; ++j) fb[j] = Bs[kk][tx * 4 + j];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(fa[i], fb[j], acc[i][j]);
    }
    __syncthreads();
  }
  const float* bias = a.bias == nullptr ? nullptr
                          : static_cast<const float*>(a.bias) + (size_t)t.e * (gt ? 2 : 1) * N;
  const float* res = static_cast<const float*>(a.res);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (ty * 4 + i >= t.M) continue;
    const size_t row = (size_t)(t.row0 + ty * 4 + i) * N;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (gt && j >= 2) continue;
      const int c = t.n0 + (gt ? tx * 2 : tx * 4) + j;
      float g = acc[i][j];
      if (bias != nullptr) g += bias[c];
      float o = activate<false>(a.act, g);
      if (gt) {
        float u = acc[i][j ^ 2];
        if (bias != nullptr) u += bias[N + c];
        o *= u;
      }
      if (res != nullptr) o += res[row + c];
      static_cast<float*>(a.y)[row + c] = o;
    }
  }
}

// ----------------------------------------------------------------- host side

// Workgroups of a launch of BM-row tiles: sum_e ceil(c_e / BM) <= M / BM +
// #{e : c_e > 0} row tiles, each with all column tiles.
long long lin_grid(const LinArgs& a, int BM, int bnc) {
  const long long mt = a.offsets ? (long long)a.M / BM + std::min(a.E, a.M)
                                 : ((long long)a.M + BM - 1) / BM;
  return mt * ((a.N + bnc - 1) / bnc);
}

}  // namespace

bool linear_fits(int E, int M, int N, int K) {
  LinArgs a{};
  a.E = E, a.M = M, a.N = N, a.K = K;
  a.offsets = reinterpret_cast<const int32_t*>(sizeof(int32_t));  // only tested for null
  return lin_grid(a, 32, 32) < (1LL << 31);
}

// Whether a launch takes the 256 x 256 tiles.
static bool use_big(const lin::LinArgs& a, bool grouped) {
  return a.M >= 64 * a.E && a.M >= 256 && lin::big_ok(a);
}

static LinArgs lin_args(const void* x, const int32_t* gather, int gk, int gT, const int32_t* offsets,
                        int E, int M, int N, int K, int act) {
  LinArgs a{};
  a.x = x, a.offsets = offsets, a.gather = gather, a.gk = gk, a.gT = gT;
  a.E = E, a.M = M, a.N = N, a.K = K, a.act = act;
  return a;
}

size_t linear_ws_bytes(int E, int M, int N, int K, int act, bool grouped, bool bf16) {
  if (!bf16) return 0;
  const int32_t some = 0;  // only tested for null
  const LinArgs a = lin_args(nullptr, nullptr, 1, M, grouped ? &some : nullptr, E, M, N, K, act);
  return use_big(a, grouped) ? big_ws_bytes(a) : 0;
}

hipError_t launch_linear(const void* x, const int32_t* gather, int gk, int gT,
                         const int32_t* offsets, int E, int M, int N, int K, const void* w,
                         const void* bias, int act, const void* res, bool bf16, void* y, void* ws,
                         hipStream_t s) {
  LinArgs a = lin_args(x, gather, gk, gT, offsets, E, M, N, K, act);
  a.w = w, a.bias = bias, a.res = res, a.y = y;
  const int bnc = act == kActGeglu || act == kActSwiglu ? 32 : 64;
  if (!bf16) {
    hipLaunchKernelGGL(lin_f32_kernel, dim3((unsigned)lin_grid(a, 64, bnc)), dim3(kThreads), 0, s, a);
    return hipGetLastError();
  }
  if (use_big(a, offsets != nullptr)) return launch_big(a, ws, s);
  hipLaunchKernelGGL((lin_bf16_kernel<64>), dim3((unsigned)lin_grid(a, 64, bnc)), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
