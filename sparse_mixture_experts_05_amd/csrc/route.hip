// Step 1 - router gating: scores, softmax over experts, top-k, renormalisation.
//
// Method: "hncyxsy.com Kimi K3 fine-grained MoE" article, router listing
// (gate Linear without bias, softmax over all experts, top-k, divide the k
// weights by their sum) and "Kimi K3 专家路由不均衡诊断" section 4.2 (the
// per-expert bias B is added inside the softmax).
//
// The k renormalised weights are exp(s_j - m) / sum_j' exp(s_j' - m) with
// m = max_e s_e: the full-E softmax denominator cancels, so only the k chosen
// scores are exponentiated. Selection runs on the scores s (exp is monotone).
//
// Layout of the work: one workgroup of 256 threads owns BT tokens.
//   phase 1: scores [BT x E] into LDS. bf16: MFMA 16x16x32 tiles (tokens x
//            experts, K = H), fp32 accumulation, operands staged in LDS by
//            coalesced global -> LDS copies. fp32: plain dot products.
//   phase 2: the scores plus the bias go to an LDS tile; G = 256/BT lanes
//            per token each keep a sorted top-k list of 64-bit (score, id)
//            keys over a strided subset of the experts, merged across the G
//            lanes by bitonic merges over DPP / ds_swizzle / bpermute
//            exchanges. Ties go to the lower expert id.
// Few tokens (bf16, T < 2048, or T < 3072 when E > 128), and mid-size
// batches (T < 6144) with E > 64, take two launches: partial score tiles over
// K slices into the workspace, then a sum in slice order and the top-k.
#include "common.hpp"
#include "kernels.hpp"
#include "route_tile.hpp"

namespace moe {
namespace {

// Top-k of the BT tokens whose scores (bias included) are in the LDS tile sc
// (row stride tile_stride<BT>()). Token t of the tile uses lanes
// [t*G, t*G + G); lane g reads the experts g, g + G, ... (at most EPX experts
// in all, a compile-time bound, so the scan is unrolled and branch free: all
// reads are issued first, from clamped columns, and columns >= E become
// empty keys), sorts blocks of KP keys and merges each into its running list,
// then the G lists are merged. KP >= k is a power of two.
// When pp is not null, the full softmax p[t, e] = exp(s_e - m) / sum_e' exp(s_e' - m)
// of every token overwrites its scores, and pp[e] receives the sum of p[t, e]
// over the tile's tokens (t ascending).
template <int BT, int KP, int EPX, int NW = 4>
__device__ __forceinline__ void topk_tokens(float* sc, int t0, int T, int E, int k,
                                            int32_t* __restrict__ topk_idx,
                                            float* __restrict__ topk_w, float* __restrict__ pp) {
  constexpr int NT = NW * 64;
  constexpr int G = NT / BT;
  constexpr int S = tile_stride<BT, NW>();
  static_assert(G >= 1 && G <= 64 && BT * G == NT, "one group of lanes per token");
  constexpr int NSUB = (EPX + G - 1) / G;  // experts per lane, at most
  constexpr int NBLK = (NSUB + KP - 1) / KP;
  const int t = threadIdx.x / G, g = threadIdx.x % G;
  const int tok = t0 + t;
  float* row = sc + t * S;
  const int nsub = (E + G - 1) / G;

  float v[NBLK * KP];
#pragma unroll
  for (int i = 0; i < NBLK * KP; ++i) v[i] = row[min(g + G * i, E - 1)];
  uint64_t list[KP];
#pragma unroll
  for (int b = 0; b < NBLK; ++b) {
    uint64_t blk[KP];
#pragma unroll
    for (int i = 0; i < KP; ++i) {
      const int e = g + G * (b * KP + i);
      // columns past E: an empty key (mask, not a select: see topk_key)
      blk[i] = topk_key(v[b * KP + i], e) & (uint64_t)(-(int64_t)(e < E));
    }
    bitonic_sort<KP>(blk);
    if (b == 0) {
#pragma unroll
      for (int i = 0; i < KP; ++i) list[i] = blk[i];
    } else {
      merge_top<KP>(list, blk);
    }
  }
  group_merge<0, G, KP>(list);

  // weights: exp(s_j - m) / sum over the k chosen, m = the best score
  const float m = key_score(list[0]);
  float ex[KP], sum = 0.0f;
#pragma unroll
  for (int j = 0; j < KP; ++j)
    if (j < k) {
      ex[j] = expf(key_score(list[j]) - m);
      sum += ex[j];
    }
  if (tok < T) {
#pragma unroll
    for (int j = 0; j < KP; ++j)
      if (j < k && j % G == g) {
        topk_idx[(size_t)tok * k + j] = key_expert(list[j]);
        topk_w[(size_t)tok * k + j] = ex[j] / sum;
      }
  }

  if (pp != nullptr) {
    // dead or NaN scores give 0; a token whose scores are all -inf or NaN has
    // no distribution and adds nothing
    float zs = 0.0f;
    for (int i = 0; i < nsub; ++i) {
      const int e = g + G * i;
      if (e < E) {
        const float v = row[e];
        const float z = (m > -INFINITY && v == v) ? expf(v - m) : 0.0f;
        row[e] = z;
        zs += z;
      }
    }
    const float Z = group_sum<0, G>(zs);
    for (int i = 0; i < nsub; ++i) {
      const int e = g + G * i;
      if (e < E) row[e] = Z > 0.0f ? row[e] / Z : 0.0f;
    }
    __syncthreads();
    const int nt = min(BT, T - t0);
    for (int e = threadIdx.x; e < E; e += NT) {
      float a = 0.0f;
      for (int q = 0; q < nt; ++q) a += sc[q * S + e];
      pp[e] = a;
    }
  }
}

template <int BT, int EPX, int NW = 4>
__device__ __forceinline__ void topk_phase(float* sc, int t0, int T, int E, int k,
                                           int32_t* __restrict__ topk_idx,
                                           float* __restrict__ topk_w, float* __restrict__ pp) {
  if (k <= 1) topk_tokens<BT, 1, EPX, NW>(sc, t0, T, E, k, topk_idx, topk_w, pp);
  else if (k <= 2) topk_tokens<BT, 2, EPX, NW>(sc, t0, T, E, k, topk_idx, topk_w, pp);
  else if (k <= 4) topk_tokens<BT, 4, EPX, NW>(sc, t0, T, E, k, topk_idx, topk_w, pp);
  else topk_tokens<BT, 8, EPX, NW>(sc, t0, T, E, k, topk_idx, topk_w, pp);
}

// P[e] = (sum over workgroups b, ascending, of part[b][e]) / T, in double.
__global__ __launch_bounds__(kThreads) void prob_mean_kernel(const float* __restrict__ part,
                                                             int nb, int T, int E,
                                                             float* __restrict__ prob_mean) {
  for (int e = threadIdx.x; e < E; e += kThreads) {
    double s = 0.0;
    int b = 0;
    for (; b + 16 <= nb; b += 16) {  // 16 loads in flight, then the sum in order
      float v[16];
#pragma unroll
      for (int u = 0; u < 16; ++u) v[u] = part[(size_t)(b + u) * E + e];
#pragma unroll
      for (int u = 0; u < 16; ++u) s += (double)v[u];
    }
    for (; b < nb; ++b) s += (double)part[(size_t)b * E + e];
    prob_mean[e] = (float)(s / (double)T);
  }
}

// One launch: BT tokens x all E experts (EP >= E) over all of H, then top-k,
// by NW waves.
template <int BT, int EP, int NW = 4>
__global__ __launch_bounds__(NW * 64) void route_bf16_kernel(
    const uint16_t* __restrict__ x, const uint16_t* __restrict__ wg,
    const float* __restrict__ bias, int T, int H, int E, int k, int32_t* __restrict__ topk_idx,
    float* __restrict__ topk_w, float* __restrict__ ppart) {
  using C = RouteTile<BT, EP, NW>;
  __shared__ __align__(16) uint8_t smem[C::LDS];
  const int t0 = blockIdx.x * BT;
  f32x4_t acc[C::MC][C::NC];
  score_tile<BT, EP, NW>(smem, x, wg, t0, T, 0, E, H, 0, H / 64, acc);
  scores_to_lds<BT, EP, NW>(smem, E, bias, acc);
  topk_phase<BT, EP, NW>(reinterpret_cast<float*>(smem), t0, T, E, k, topk_idx, topk_w,
                         ppart != nullptr ? ppart + (size_t)blockIdx.x * E : nullptr);
}

// fp32 scores with plain dot products (small fp32 layers).
__global__ __launch_bounds__(kThreads) void route_f32_kernel(
    const float* __restrict__ x, const float* __restrict__ wg, const float* __restrict__ bias,
    int T, int H, int E, int k, int32_t* __restrict__ topk_idx, float* __restrict__ topk_w,
    float* __restrict__ ppart) {
  constexpr int BT = 16;
  constexpr int S = tile_stride<BT>();
  __shared__ float sc[BT * S];
  const int t0 = blockIdx.x * BT;
  for (int p = threadIdx.x; p < BT * E; p += kThreads) {
    const int t = p / E, e = p % E;
    const float4* xr = reinterpret_cast<const float4*>(x + (size_t)min(t0 + t, T - 1) * H);
    const float4* wr = reinterpret_cast<const float4*>(wg + (size_t)e * H);
    float s = 0.0f;
    for (int h = 0; h < H / 4; ++h) {
      const float4 a = xr[h], b = wr[h];
      s = fmaf(a.x, b.x, s);
      s = fmaf(a.y, b.y, s);
      s = fmaf(a.z, b.z, s);
      s = fmaf(a.w, b.w, s);
    }
    sc[t * S + e] = bias != nullptr ? s + bias[e] : s;
  }
  __syncthreads();
  topk_phase<BT, kMaxE>(sc, t0, T, E, k, topk_idx, topk_w,
                        ppart != nullptr ? ppart + (size_t)blockIdx.x * E : nullptr);
}


// Two launches (bf16). Phase 1: workgroup (token block, expert block, K slice)
// computes its BT x EP partial score tile and stores it in the workspace
// ws[ks][t][e]. Phase 2: a workgroup of 4 or 16 tokens sums each token's K
// slices in a fixed order (ks ascending), adds the bias and runs the top-k.
//   Few tokens: 16 x 64 tiles, so that a few tokens still spread Wg over
//   about 256 workgroups (one workgroup per 16 tokens would stream all of Wg
//   through a single CU).
//   Mid-size batches and E > 64: 64 x 128 (E <= 128) or 128 x 256 tiles, so
//   that Wg is read once per 64 or 128 tokens instead of once per 16-64, the
//   L2 -> LDS traffic that bounds the one-launch kernel at large E.
// BT tokens per workgroup: 256 / BT lanes per token in the top-k. Few lanes
// per token sort whole blocks of experts and merge over fewer levels; many
// lanes per token keep small batches spread over more workgroups.
template <int NKS, int BT, int EPX>
__global__ __launch_bounds__(kThreads) void route_select_kernel(const float* __restrict__ ws,
                                                                const float* __restrict__ bias,
                                                                int T, int E, int k,
                                                                int32_t* __restrict__ topk_idx,
                                                                float* __restrict__ topk_w,
                                                                float* __restrict__ ppart) {
  constexpr int S = tile_stride<BT>();
  __shared__ float sc[BT * S];
  const int t0 = blockIdx.x * BT;
  // PER entries per thread at a time (about 32 loads in flight): all their
  // slice loads are issued first, from addresses clamped into the buffer, then
  // each entry is summed in slice order
  constexpr int PER = NKS >= 8 ? 32 / NKS : 8;
  const int nval = min(BT, T - t0) * E;  // entries of the tile's real tokens (t-major)
  for (int p0 = threadIdx.x; p0 < nval; p0 += PER * kThreads) {
    float v[PER][NKS], bv[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int p = p0 + i * kThreads;
      const int tt = min(t0 + p / E, T - 1), e = p % E;
#pragma unroll
      for (int q = 0; q < NKS; ++q) v[i][q] = ws[((size_t)q * T + tt) * E + e];
      bv[i] = bias != nullptr ? bias[e] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int p = p0 + i * kThreads;
      const int t = p / E, e = p % E;
      if (p < nval) {
        float s = 0.0f;
#pragma unroll
        for (int q = 0; q < NKS; ++q) s += v[i][q];
        sc[t * S + e] = bias != nullptr ? s + bv[i] : s;
      }
    }
  }
  __syncthreads();
  topk_phase<BT, EPX>(sc, t0, T, E, k, topk_idx, topk_w,
                      ppart != nullptr ? ppart + (size_t)blockIdx.x * E : nullptr);
}

// The select for exactly nks K slices (a power of two up to kMaxSlices) and
// at most EPX experts.
template <int BT, int EPX>
hipError_t launch_select_e(int nks, const float* ws, const float* bias, int T, int E, int k,
                           int32_t* idx, float* w, float* pp, hipStream_t s) {
  const dim3 grid((T + BT - 1) / BT), block(kThreads);
  switch (nks) {
    case 1: hipLaunchKernelGGL((route_select_kernel<1, BT, EPX>), grid, block, 0, s, ws, bias, T, E, k, idx, w, pp); break;
    case 2: hipLaunchKernelGGL((route_select_kernel<2, BT, EPX>), grid, block, 0, s, ws, bias, T, E, k, idx, w, pp); break;
    case 4: hipLaunchKernelGGL((route_select_kernel<4, BT, EPX>), grid, block, 0, s, ws, bias, T, E, k, idx, w, pp); break;
    case 8: hipLaunchKernelGGL((route_select_kernel<8, BT, EPX>), grid, block, 0, s, ws, bias, T, E, k, idx, w, pp); break;
    case 16: hipLaunchKernelGGL((route_select_kernel<16, BT, EPX>), grid, block, 0, s, ws, bias, T, E, k, idx, w, pp); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

template <int BT>
hipError_t launch_select(int nks, const float* ws, const float* bias, int T, int E, int k,
                         int32_t* idx, float* w, float* pp, hipStream_t s) {
  if (E <= 64) return launch_select_e<BT, 64>(nks, ws, bias, T, E, k, idx, w, pp, s);
  if (E <= 128) return launch_select_e<BT, 128>(nks, ws, bias, T, E, k, idx, w, pp, s);
  return launch_select_e<BT, kMaxE>(nks, ws, bias, T, E, k, idx, w, pp, s);
}

// Path of a route call. Both two-launch paths write and re-read T x E partial
// scores per K slice, so their time grows faster with T than the one-launch
// path's; the one-launch path re-reads Wg once per 16, 32 or 64 tokens.
// Measured crossovers (H = 4096, k = 8): small tiles against one launch near
// T = 2048 up to E = 128 and near 3072 for E = 256 (graph replay, 4-wave
// tiles); small against big tiles near T = 2048 (E = 128: 18.0 against 18.5
// us at 1024, equal at 2048; E = 256: 26.7 against 27.8 at 1024, 35.0
// against 31.0 at 2048; route alone, read-flushed caches). Big tiles
// against one launch (route alone, read-flushed caches, 8-wave tiles on both
// paths for E >= 128): E = 128 30.0 against 54.7 us at T = 6144, 32.4
// against 33.3 at 8192, 47.5 against 58.9 at 12288, 45.9 against 46.1 at
// 16384; E = 256 39.3 against 85.8 at 6144, 59.6 against 99.3 at 12288,
// 62.9 against 63.1 at 16384. So big tiles up to T = 16384, where the
// one-launch path has 64-token tiles.

template <int BT, int EP, int NW = 4>
hipError_t launch_bf16(const void* x, const void* wg, const float* bias, int T, int H, int E,
                       int k, int32_t* idx, float* w, float* pp, hipStream_t s) {
  const int grid = (T + BT - 1) / BT;
  hipLaunchKernelGGL((route_bf16_kernel<BT, EP, NW>), dim3(grid), dim3(NW * 64), 0, s,
                     static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(wg), bias, T,
                     H, E, k, idx, w, pp);
  return hipGetLastError();
}

template <int BT>
hipError_t launch_bf16_bt(const void* x, const void* wg, const float* bias, int T, int H, int E,
                          int k, int32_t* idx, float* w, float* pp, hipStream_t s) {
  if (E <= 16) return launch_bf16<BT, 16>(x, wg, bias, T, H, E, k, idx, w, pp, s);
  if (E <= 32) return launch_bf16<BT, 32>(x, wg, bias, T, H, E, k, idx, w, pp, s);
  if (E <= 64) return launch_bf16<BT, 64>(x, wg, bias, T, H, E, k, idx, w, pp, s);
  if (E <= 128) return launch_bf16<BT, 128, route_waves<BT, 128>()>(x, wg, bias, T, H, E, k, idx, w, pp, s);
  return launch_bf16<BT, 256, route_waves<BT, 256>()>(x, wg, bias, T, H, E, k, idx, w, pp, s);
}

// Workgroups of the launch that runs the top-k (one partial probability row each).
int topk_blocks(int T, int E, bool bf16) {
  if (route_two_phase(T, E, bf16)) {
    const int bt = select_tokens_per_block(T);
    return (T + bt - 1) / bt;
  }
  const int bt = bf16 ? bf16_tokens_per_block(T) : 16;
  return (T + bt - 1) / bt;
}

}  // namespace

size_t route_ws_bytes(int T, int H, int E, bool bf16, bool prob) {
  size_t b = scores_ws_bytes(T, H, E, bf16);
  if (prob) b += align256((size_t)topk_blocks(T, E, bf16) * E * sizeof(float));
  return b;
}

hipError_t launch_route(const void* x, const void* wg, const float* bias, int T, int H, int E,
                        int k, bool bf16, int32_t* topk_idx, float* topk_w, float* prob_mean,
                        void* ws, hipStream_t s) {
  // partial probability sums sit after the partial score tiles
  float* pp = prob_mean == nullptr
                  ? nullptr
                  : reinterpret_cast<float*>(static_cast<char*>(ws) + scores_ws_bytes(T, H, E, bf16));
  hipError_t err = hipSuccess;
  const RouteMode mode = route_mode(T, E, bf16);
  if (mode != kOneLaunch) {
    const int nks = route_kslices(T, H, E);
    err = launch_partial(x, wg, T, H, E, static_cast<float*>(ws), s);
    if (err != hipSuccess) return err;
    const float* wsf = static_cast<const float*>(ws);
    err = select_tokens_per_block(T) == 16
              ? launch_select<16>(nks, wsf, bias, T, E, k, topk_idx, topk_w, pp, s)
              : launch_select<4>(nks, wsf, bias, T, E, k, topk_idx, topk_w, pp, s);
  } else if (!bf16) {
    const int grid = (T + 15) / 16;
    hipLaunchKernelGGL(route_f32_kernel, dim3(grid), dim3(kThreads), 0, s,
                       static_cast<const float*>(x), static_cast<const float*>(wg), bias, T, H, E,
                       k, topk_idx, topk_w, pp);
    err = hipGetLastError();
  } else {
    switch (bf16_tokens_per_block(T)) {
      case 64: err = launch_bf16_bt<64>(x, wg, bias, T, H, E, k, topk_idx, topk_w, pp, s); break;
      case 32: err = launch_bf16_bt<32>(x, wg, bias, T, H, E, k, topk_idx, topk_w, pp, s); break;
      default: err = launch_bf16_bt<16>(x, wg, bias, T, H, E, k, topk_idx, topk_w, pp, s); break;
    }
  }
  if (err != hipSuccess || prob_mean == nullptr) return err;
  hipLaunchKernelGGL(prob_mean_kernel, dim3(1), dim3(kThreads), 0, s, pp, topk_blocks(T, E, bf16), T,
                     E, prob_mean);
  return hipGetLastError();
}

}  // namespace moe
