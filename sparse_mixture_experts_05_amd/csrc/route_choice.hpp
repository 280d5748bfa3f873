// The choice of grouped routing, from fp32 scores in LDS: shared by the grouped route and
// the few-token layer. Included by the .hip files that choose; everything is local to the
// including file. The formulas are at the head of route_grouped.hip.
#pragma once

#include <type_traits>

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

// The largest u of the wave, in every lane: DPP steps within 16 lanes, then their last
// lanes broadcast to the next 16 and 32 (row_bcast), lane 63 has it.
__device__ __forceinline__ uint32_t wave_max(uint32_t u) {
  auto step = [&](auto ctrl) {
    u = max(u, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, decltype(ctrl)::value, 0xF, 0xF, true));
  };
  step(std::integral_constant<int, 0x111>{});  // row_shr 1, 2, 4, 8
  step(std::integral_constant<int, 0x112>{});
  step(std::integral_constant<int, 0x114>{});
  step(std::integral_constant<int, 0x118>{});
  step(std::integral_constant<int, 0x142>{});  // row_bcast 15, 31
  step(std::integral_constant<int, 0x143>{});
  return (uint32_t)__builtin_amdgcn_readlane((int)u, 63);
}

// list[0 .. k-1] <- the k largest keys of a token that has a whole wave: lane g holds the
// high halves (scores) of the keys of experts g, g + 64, ... (0: none). k times the largest
// score, then its lowest expert from the lanes' masks, in scalar registers: 20 instructions
// a round, where merging sorted lists of 8 over 64 lanes takes 700 (grouped route, k 8, 16
// tokens of 128 experts 12.0 -> 10.2 us, 1000 of 256 26.5 -> 24.8; k 1 and 2 the same).
template <int KP, int NSUB>
__device__ __forceinline__ void pop_top(uint32_t (&o)[NSUB], int k, uint64_t (&list)[KP]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int j = 0; j < KP; ++j) {
    list[j] = 0;
    if (j >= k) continue;
    uint32_t m = o[0];
#pragma unroll
    for (int i = 1; i < NSUB; ++i) m = max(m, o[i]);
    m = wave_max(m);
    int e = -1;
#pragma unroll
    for (int i = NSUB - 1; i >= 0; --i) {
      const unsigned long long at = __ballot(o[i] == m);
      if (at != 0) e = 64 * i + __ffsll(at) - 1;
    }
#pragma unroll
    for (int i = 0; i < NSUB; ++i)
      if (e == 64 * i + lane) o[i] = 0;
    list[j] = ((uint64_t)m << 32) | (uint32_t)(~(uint32_t)e);
  }
}

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
  if constexpr (G == 64) {
    uint32_t o[NSUB];
#pragma unroll
    for (int i = 0; i < NSUB; ++i) {
      const int e = g + G * i;
      const bool in = e < E && ((mask >> ((min(e, E - 1) * a.magic) >> 16)) & 1);
      o[i] = in ? (uint32_t)(topk_key(x[i], e) >> 32) : 0u;
    }
    pop_top<KP, NSUB>(o, k, list);
  } else {
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
  }

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

GroupArgs group_args(const float* bias, int E, bool softmax, int groups, int topk_groups,
                     int group_top, bool renorm, float scale) {
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
  return a;
}

}  // namespace
}  // namespace moe
