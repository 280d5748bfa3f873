// Grouped routing: sigmoid or softmax scores, a balance bias that moves the
// choice and not the weights, experts limited to the best groups, top-k,
// renormalised and scaled weights. The choice by biased scores with unbiased
// weights is the other reading of the balance bias of "Kimi K3
// 专家路由不均衡诊断" section 4.2 (moe_route has it inside the softmax); top-k and the
// renormalisation are those of the "hncyxsy.com Kimi K3 fine-grained MoE"
// article's router listing.
//
//   s = x . Wg^T                      p = sigmoid(s) or softmax(s)
//   v = p + b (b = -inf or NaN, or a NaN score: the expert is off)
//   group score = sum of the group's 1 or 2 largest v (experts that are on)
//   chosen: the topk_groups best groups, in them the k largest v
//   w_j = scale * p_j / (renorm ? sum_j' p_j' : 1)
//
// Without a bias the experts of the chosen groups are ordered by s itself
// (both score functions are monotone), so scores past the point where p rounds
// to 1 or 0 keep their order. Renormalised weights are taken relative to the
// largest chosen score, so they do not underflow together.
//
// The scores come from the score tiles of route_tile.hpp (MFMA, fp32
// accumulation); selection works on the fp32 scores in LDS.
#include "kernels.hpp"
#include "route_tile.hpp"

namespace moe {
namespace {

constexpr int kMaxGroups = 64;  // one bit each of a token's 64-bit group mask

struct GroupArgs {
  const float* bias;  // [E] or null
  int groups, per, topk_groups, group_top;
  uint32_t magic;     // e / per == (e * magic) >> 16 for e < 256
  int softmax, renorm;
  float scale;
};

__device__ __forceinline__ float sigmoidf(float s) { return 1.0f / (1.0f + expf(-s)); }

// exp by the hardware's exp2 (relative error about |x| * 6e-8 and an ulp): the choice
// evaluates all E experts of a token, and its values carry the scores' own error of
// that size. The k weights take expf.
__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }

template <int L, int G>
__device__ __forceinline__ float group_max(float v) {
  if constexpr ((1 << L) < G) return group_max<L + 1, G>(fmaxf(v, __uint_as_float(partner<L>(__float_as_uint(v)))));
  return v;
}

// LDS writes of this wave are seen by its later reads (the LDS serves a wave in order;
// this keeps the compiler from moving them).
__device__ __forceinline__ void wave_lds_fence() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// LDS of the group stage of BT tokens: the values v and the group scores.
template <int BT, int NW>
struct GroupLds {
  float v[BT * tile_stride<BT, NW>()];
  float gs[BT][kMaxGroups + 1];
};

// Chooses for the BT tokens whose scores are in the LDS tile sc (row stride
// tile_stride<BT, NW>(), no bias in them). Lanes as in topk_tokens: G = 64 * NW / BT
// lanes a token, all in one wave, so nothing here needs a barrier; lane g has the
// experts g, g + G, ... A token's time is instructions: its E values p + b are worked
// out once, by the hardware's exp2 and reciprocal, and kept in LDS for the group
// scores (one lane a group reads its group). Work on scores in place of values, and a
// workgroup's barriers between the stages, took 31 us for 4096 tokens of 256 experts.
template <int BT, int KP, int EPX, int NW>
__device__ __forceinline__ void grouped_tokens(const float* sc, GroupLds<BT, NW>& L,
                                               const GroupArgs& a, int t0, int T, int E, int k,
                                               int32_t* __restrict__ topk_idx,
                                               float* __restrict__ topk_w) {
  constexpr int NT = NW * 64, G = NT / BT, S = tile_stride<BT, NW>();
  static_assert(G >= 1 && G <= 64 && BT * G == NT, "one group of lanes per token");
  constexpr int NSUB = (EPX + G - 1) / G;
  constexpr int NBLK = (NSUB + KP - 1) / KP;
  const int t = threadIdx.x / G, g = threadIdx.x % G;
  const int tok = t0 + t;
  const float* row = sc + t * S;
  const bool limit = a.topk_groups < a.groups;

  float x[NBLK * KP];  // scores, then the keys' values
#pragma unroll
  for (int i = 0; i < NBLK * KP; ++i) x[i] = i < NSUB ? row[min(g + G * i, E - 1)] : 0.0f;
  float top = 0.0f, rz = 1.0f;
  if (a.softmax) {
    float m = -INFINITY, z = 0.0f;
#pragma unroll
    for (int i = 0; i < NSUB; ++i) m = fmaxf(m, x[i]);  // fmaxf drops a NaN
    top = group_max<0, G>(m);
#pragma unroll
    for (int i = 0; i < NSUB; ++i) {
      const float d = x[i] - top;
      z += d == d && g + G * i < E ? exp_fast(d) : 0.0f;
    }
    rz = 1.0f / group_sum<0, G>(z);
  }
  if (a.bias != nullptr || limit) {
    // branch free in the experts (a load or a write under a branch would wait for each in
    // turn); columns from E up hold values that nobody reads
    float v[NSUB], b[NSUB];
#pragma unroll
    for (int i = 0; i < NSUB; ++i) b[i] = 0.0f;
    if (a.bias != nullptr) {
#pragma unroll
      for (int i = 0; i < NSUB; ++i) b[i] = a.bias[min(g + G * i, E - 1)];
    }
    if (a.softmax) {
#pragma unroll
      for (int i = 0; i < NSUB; ++i) v[i] = fmaf(exp_fast(x[i] - top), rz, b[i]);
    } else {
#pragma unroll
      for (int i = 0; i < NSUB; ++i) v[i] = __builtin_amdgcn_rcpf(1.0f + exp_fast(-x[i])) + b[i];
    }
    if (limit) {
#pragma unroll
      for (int i = 0; i < NSUB; ++i) L.v[t * S + g + G * i] = v[i];
    }
    if (a.bias != nullptr) {
#pragma unroll
      for (int i = 0; i < NSUB; ++i) x[i] = v[i];
    }
  }
  unsigned long long mask = ~0ull;
  if (limit) {
    wave_lds_fence();
    // one lane a group; each starts at another expert of its group, which spreads the
    // LDS banks when groups are a power of two wide
    for (int gb = 0; gb < a.groups; gb += G) {
      const int q = gb + g;
      if (q < a.groups) {
        const float* r = L.v + t * S + q * a.per;
        float b1 = -INFINITY, b2 = -INFINITY;
        int i = q % a.per;
        for (int n = 0; n < a.per; n += 4) {
          float v[4];  // past the end: nothing
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            v[u] = n + u < a.per ? fmaxf(r[i], -INFINITY) : -INFINITY;
            i = i + 1 == a.per ? 0 : i + 1;
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            b2 = fmaxf(b2, fminf(b1, v[u]));
            b1 = fmaxf(b1, v[u]);
          }
        }
        // the second counts only if it is on
        L.gs[t][q] = a.group_top == 2 && b2 > -INFINITY ? b1 + b2 : b1;
      }
    }
    wave_lds_fence();
    mask = 0;
    for (int gb = 0; gb < a.groups; gb += G) {
      const int q = gb + g;
      bool in = false;
      if (q < a.groups) {
        const float own = L.gs[t][q];
        int rank = 0;
        for (int o = 0; o < a.groups; ++o) {
          const float v = L.gs[t][o];
          rank += v > own || (v == own && o < q);
        }
        in = rank < a.topk_groups;
      }
      unsigned long long bits = __ballot(in);
      if constexpr (G < 64) bits = (bits >> ((threadIdx.x & 63) / G * G)) & ((1ull << (G & 63)) - 1);
      mask |= bits << gb;
    }
  }

  uint64_t list[KP];
#pragma unroll
  for (int b = 0; b < NBLK; ++b) {
    uint64_t blk[KP];
#pragma unroll
    for (int i = 0; i < KP; ++i) {
      const int e = g + G * (b * KP + i);
      const bool in = e < E && ((mask >> ((min(e, E - 1) * a.magic) >> 16)) & 1);
      blk[i] = topk_key(x[b * KP + i], e) & (uint64_t)(-(int64_t)in);
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

  // the chosen scores; an expert that is off (chosen only when fewer than k
  // are on) weighs nothing
  float sj[KP], m = -INFINITY;
#pragma unroll
  for (int j = 0; j < KP; ++j) {
    sj[j] = -INFINITY;
    if (j < k && key_score(list[j]) > -INFINITY) sj[j] = row[key_expert(list[j])];
    m = fmaxf(m, sj[j]);
  }
  // renormalised: p_j times a factor that all j share (softmax: Z * exp(top - m);
  // sigmoid: exp(-min(m, 0)))
  if (!a.softmax) m = fminf(m, 0.0f);
  float p[KP], sum = 0.0f;
#pragma unroll
  for (int j = 0; j < KP; ++j) {
    p[j] = 0.0f;
    if (j < k && sj[j] > -INFINITY) {
      if (a.softmax) p[j] = a.renorm ? expf(sj[j] - m) : expf(sj[j] - top) * rz;
      else if (!a.renorm || sj[j] > 0.0f) p[j] = sigmoidf(sj[j]);
      else p[j] = expf(sj[j] - m) / (1.0f + expf(sj[j]));
    }
    sum += p[j];
  }
  const float f = a.renorm ? (sum > 0.0f ? a.scale / sum : sum * 0.0f) : a.scale;
  if (tok < T) {
#pragma unroll
    for (int j = 0; j < KP; ++j)
      if (j < k && j % G == g) {
        topk_idx[(size_t)tok * k + j] = key_expert(list[j]);
        topk_w[(size_t)tok * k + j] = p[j] * f;
      }
  }
}

template <int BT, int EPX, int NW = 4>
__device__ __forceinline__ void grouped_phase(const float* sc, GroupLds<BT, NW>& L,
                                              const GroupArgs& a, int t0, int T, int E, int k,
                                              int32_t* __restrict__ idx, float* __restrict__ w) {
  if (k <= 1) grouped_tokens<BT, 1, EPX, NW>(sc, L, a, t0, T, E, k, idx, w);
  else if (k <= 2) grouped_tokens<BT, 2, EPX, NW>(sc, L, a, t0, T, E, k, idx, w);
  else if (k <= 4) grouped_tokens<BT, 4, EPX, NW>(sc, L, a, t0, T, E, k, idx, w);
  else grouped_tokens<BT, 8, EPX, NW>(sc, L, a, t0, T, E, k, idx, w);
}

// One launch: BT tokens x all E experts (EP >= E) over all of H, then the choice.
template <int BT, int EP, int NW>
__global__ __launch_bounds__(NW * 64) void grouped_bf16_kernel(
    const uint16_t* __restrict__ x, const uint16_t* __restrict__ wg, GroupArgs a, int T, int H,
    int E, int k, int32_t* __restrict__ topk_idx, float* __restrict__ topk_w) {
  using C = RouteTile<BT, EP, NW>;
  constexpr int NEED = C::SC_BYTES + (int)sizeof(GroupLds<BT, NW>);
  constexpr int LDS = C::LDS > NEED ? C::LDS : NEED;
  static_assert(LDS <= 160 * 1024 && C::SC_BYTES % 8 == 0, "score tile and group stage in LDS");
  __shared__ __align__(16) uint8_t smem[LDS];
  const int t0 = blockIdx.x * BT;
  f32x4_t acc[C::MC][C::NC];
  score_tile<BT, EP, NW, uint16_t, true>(smem, x, wg, t0, T, 0, E, H, 0, H / 64, acc);
  scores_to_lds<BT, EP, NW>(smem, E, nullptr, acc);
  grouped_phase<BT, EP, NW>(reinterpret_cast<float*>(smem),
                            *reinterpret_cast<GroupLds<BT, NW>*>(smem + C::SC_BYTES), a, t0, T, E, k,
                            topk_idx, topk_w);
}

// Second launch of the two-launch paths: the K slices of each score are summed
// in slice order, then the choice.
template <int NKS, int BT, int EPX>
__global__ __launch_bounds__(kThreads) void grouped_select_kernel(const float* __restrict__ ws,
                                                                  GroupArgs a, int T, int E, int k,
                                                                  int32_t* __restrict__ topk_idx,
                                                                  float* __restrict__ topk_w) {
  constexpr int S = tile_stride<BT>(), G = kThreads / BT, NSUB = (EPX + G - 1) / G;
  __shared__ float sc[BT * S];
  __shared__ GroupLds<BT, 4> L;
  const int t0 = blockIdx.x * BT;
  // each lane sums the experts that it will choose from; about 32 loads in flight, from
  // addresses clamped into the buffer
  constexpr int PER = NKS >= 16 ? 2 : 32 / NKS < NSUB ? 32 / NKS : NSUB;
  const int t = threadIdx.x / G, g = threadIdx.x % G;
  const float* src = ws + (size_t)min(t0 + t, T - 1) * E;
#pragma unroll
  for (int i0 = 0; i0 < NSUB; i0 += PER) {
    float v[PER][NKS];
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
      for (int q = 0; q < NKS; ++q) v[i][q] = src[(size_t)q * T * E + min(g + G * (i0 + i), E - 1)];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      float s = 0.0f;
#pragma unroll
      for (int q = 0; q < NKS; ++q) s += v[i][q];
      sc[t * S + g + G * (i0 + i)] = s;  // columns from E up: read by nobody
    }
  }
  wave_lds_fence();
  grouped_phase<BT, EPX>(sc, L, a, t0, T, E, k, topk_idx, topk_w);
}

template <int BT, int EPX>
hipError_t launch_select_e(int nks, const float* ws, const GroupArgs& a, int T, int E, int k,
                           int32_t* idx, float* w, hipStream_t s) {
  const dim3 grid((T + BT - 1) / BT), block(kThreads);
  switch (nks) {
    case 1: hipLaunchKernelGGL((grouped_select_kernel<1, BT, EPX>), grid, block, 0, s, ws, a, T, E, k, idx, w); break;
    case 2: hipLaunchKernelGGL((grouped_select_kernel<2, BT, EPX>), grid, block, 0, s, ws, a, T, E, k, idx, w); break;
    case 4: hipLaunchKernelGGL((grouped_select_kernel<4, BT, EPX>), grid, block, 0, s, ws, a, T, E, k, idx, w); break;
    case 8: hipLaunchKernelGGL((grouped_select_kernel<8, BT, EPX>), grid, block, 0, s, ws, a, T, E, k, idx, w); break;
    case 16: hipLaunchKernelGGL((grouped_select_kernel<16, BT, EPX>), grid, block, 0, s, ws, a, T, E, k, idx, w); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

template <int BT>
hipError_t launch_select(int nks, const float* ws, const GroupArgs& a, int T, int E, int k,
                         int32_t* idx, float* w, hipStream_t s) {
  if (E <= 64) return launch_select_e<BT, 64>(nks, ws, a, T, E, k, idx, w, s);
  if (E <= 128) return launch_select_e<BT, 128>(nks, ws, a, T, E, k, idx, w, s);
  return launch_select_e<BT, kMaxE>(nks, ws, a, T, E, k, idx, w, s);
}

template <int BT, int EP, int NW = 4>
hipError_t launch_bf16(const void* x, const void* wg, const GroupArgs& a, int T, int H, int E,
                       int k, int32_t* idx, float* w, hipStream_t s) {
  hipLaunchKernelGGL((grouped_bf16_kernel<BT, EP, NW>), dim3((T + BT - 1) / BT), dim3(NW * 64), 0,
                     s, static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(wg), a, T, H,
                     E, k, idx, w);
  return hipGetLastError();
}

template <int BT>
hipError_t launch_bf16_bt(const void* x, const void* wg, const GroupArgs& a, int T, int H, int E,
                          int k, int32_t* idx, float* w, hipStream_t s) {
  if (E <= 16) return launch_bf16<BT, 16>(x, wg, a, T, H, E, k, idx, w, s);
  if (E <= 32) return launch_bf16<BT, 32>(x, wg, a, T, H, E, k, idx, w, s);
  if (E <= 64) return launch_bf16<BT, 64>(x, wg, a, T, H, E, k, idx, w, s);
  if constexpr (BT != 32) {  // 8192 to 16383 tokens and E > 64 take two launches
    if (E <= 128) return launch_bf16<BT, 128, route_waves<BT, 128>()>(x, wg, a, T, H, E, k, idx, w, s);
    return launch_bf16<BT, 256, route_waves<BT, 256>()>(x, wg, a, T, H, E, k, idx, w, s);
  }
  return hipErrorInvalidValue;
}

// bf16 calls take the paths of moe_route, except that few tokens with a small Wg (256 KB)
// take one launch too: a workgroup of 16 tokens reads all of it at about 60 GB/s, which
// costs the GPU 0 to 3 us more than two launches (H 2048, E 60, T 16: 12.6 against 9.4;
// T 1777: 12.9 against 11.6; H 1024, E 16: 5.1 against 7.3) and saves the host the second
// one and the workspace (5 us). At 512 KB one launch takes up to twice as long.
bool one_launch(int T, int H, int E, bool bf16) {
  return bf16 && (route_mode(T, E, true) == kOneLaunch ||
                  (T < 2048 && (long long)E * H <= 128 * 1024));
}

// fp32 scores always take two launches: 16 x 64 tiles for few tokens, else 64 x 128.
bool f32_big(int T) { return T >= 512; }

// K slices of the fp32 paths: a power of two that divides the panels (32 k), about 512
// workgroups, at least 4 panels each.
int f32_kslices(int T, int H, int E) {
  const bool big = f32_big(T);
  const int tiles = big ? ((T + 63) / 64) * ((E + 127) / 128) : ((T + 15) / 16) * ((E + 63) / 64);
  int ks = 1;
  while (ks * 2 * tiles <= 512 && (H / 32) % (ks * 8) == 0 && ks * 2 <= kMaxSlices) ks *= 2;
  return ks;
}

hipError_t launch_partial_f32(const void* x, const void* wg, int T, int H, int E, float* sp,
                              hipStream_t s) {
  const int nks = f32_kslices(T, H, E), kps = H / 32 / nks;
  const float* xp = static_cast<const float*>(x);
  const float* wp = static_cast<const float*>(wg);
  if (f32_big(T))
    hipLaunchKernelGGL((route_partial_kernel<64, 128, 4, float, true>), dim3((T + 63) / 64, (E + 127) / 128, nks),
                       dim3(256), 0, s, xp, wp, T, H, E, kps, sp);
  else
    hipLaunchKernelGGL((route_partial_kernel<kPartBT, kPartEP, 4, float, true>),
                       dim3((T + kPartBT - 1) / kPartBT, (E + kPartEP - 1) / kPartEP, nks), dim3(256), 0,
                       s, xp, wp, T, H, E, kps, sp);
  return hipGetLastError();
}

}  // namespace

size_t route_grouped_ws_bytes(int T, int H, int E, bool bf16) {
  if (one_launch(T, H, E, bf16)) return 0;
  return bf16 ? scores_ws_bytes(T, H, E, true)
              : align256((size_t)f32_kslices(T, H, E) * T * E * sizeof(float));
}

hipError_t launch_route_grouped(const void* x, const void* wg, const float* bias, int T, int H,
                                int E, int k, bool softmax, int groups, int topk_groups,
                                int group_top, bool renorm, float scale, bool bf16,
                                int32_t* topk_idx, float* topk_w, void* ws, hipStream_t s) {
  GroupArgs a{};
  a.bias = bias;
  a.groups = groups;
  a.per = E / groups;
  a.topk_groups = topk_groups;
  a.group_top = group_top;
  a.magic = (65536u + a.per - 1) / a.per;
  a.softmax = softmax;
  a.renorm = renorm;
  a.scale = scale;
  if (!one_launch(T, H, E, bf16)) {
    float* sp = static_cast<float*>(ws);
    const int nks = bf16 ? route_kslices(T, H, E) : f32_kslices(T, H, E);
    const hipError_t err = bf16 ? launch_partial<true>(x, wg, T, H, E, sp, s)
                                : launch_partial_f32(x, wg, T, H, E, sp, s);
    if (err != hipSuccess) return err;
    return select_tokens_per_block(T) == 16
               ? launch_select<16>(nks, sp, a, T, E, k, topk_idx, topk_w, s)
               : launch_select<4>(nks, sp, a, T, E, k, topk_idx, topk_w, s);
  }
  switch (bf16_tokens_per_block(T)) {
    case 64: return launch_bf16_bt<64>(x, wg, a, T, H, E, k, topk_idx, topk_w, s);
    case 32: return launch_bf16_bt<32>(x, wg, a, T, H, E, k, topk_idx, topk_w, s);
    default: return launch_bf16_bt<16>(x, wg, a, T, H, E, k, topk_idx, topk_w, s);
  }
}

}  // namespace moe
