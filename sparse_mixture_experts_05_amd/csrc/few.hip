// A whole MoE layer for a few tokens (T <= 64) in two launches: scores, then choice,
// experts, shared expert and combine. A decode step is a stream of the chosen experts'
// weights; what the layer's separate launches cost there is their drains and starts.
//
//   s[t,e]  = x[t] . wg[e] (+ bias[e])                    top-k as moe_route_grouped
//   h[t,j]  = act(x[t] . up[e_j]^T + b_up[e_j])           rounded to the layer's type
//   out[t]  = sum_j w[t,j] (h[t,j] . down[e_j]^T + b_down[e_j])  + shared expert(x[t])
//
// The second launch is one queue of tasks, taken by ticket in this order:
//   up tasks    (expert, 32 weight rows of up: 32 columns of h, or 16 of a gated act)
//   down tasks  (K slice, 32 columns of out), over all chosen experts of the slice
// A down task waits until the up tasks of its experts are done. It waits only for lower
// tickets, and whoever holds a lower ticket is running and waits for nothing (an up task)
// or for lower tickets still: the queue empties whatever number of workgroups is resident
// and whatever else the GPU runs. (The wait ends after a second in any case: a workspace
// that another call is using gives wrong results, no hang.)
//
// MFMA columns are tokens, in order: an expert's product is made for all of them and kept
// for those that chose it, so nothing is sorted or gathered, and a token's sum stays in
// one lane. Weights go straight to registers (nothing else on the chip reads them).
#include <algorithm>

#include "kernels.hpp"
#include "linear.hpp"
#include "route_choice.hpp"

namespace moe {
namespace {

using namespace lin;

constexpr int kWaves = 8, kFewThreads = kWaves * 64;
constexpr int kFewT = 64, kSlots = 8;     // tokens, experts of a token
constexpr int kCols = 32;                 // weight rows of a task: two MFMA row tiles
constexpr int kMaxDown = 8;               // K slices of the down tasks
constexpr int kBT = 16;                   // tokens of a pass of the choice

struct FewArgs {
  const void *x, *up, *down, *b_up, *b_down, *s_up, *s_down;
  const float* bias;  // inside the scores, or null
  GroupArgs g;
  int T, H, E, k, F, Fs, act;
  float* scores;       // [T, E]
  void* h;             // [T * k, F], then [T, Fs]
  float* part;         // [H / 32, D, 2, column tiles, 64, 4]: partial columns of out
  unsigned* counters;  // ticket | done [E + 1] | arrived [H / 32, column tiles]
  int D;
  int32_t* idx;
  float* w;
  void* out;
};

__host__ __device__ inline int counter_ints(int E, int H, int nt) { return 1 + E + 1 + H / kCols * nt; }

// ----------------------------------------------------------------- scores

// 16 experts x 16 tokens a workgroup of 16 waves, which share H (64 bytes of a row a step)
// and add their sums in wave order. Clears the second launch's counters.
constexpr int kScoreWaves = 16;

template <typename T>
__global__ __launch_bounds__(kScoreWaves * 64) void few_scores_kernel(const T* __restrict__ x,
                                                                     const T* __restrict__ wg, int nT,
                                                                     int H, int E, float* __restrict__ scores,
                                                                     unsigned* __restrict__ counters,
                                                                     int ncount) {
  constexpr int U = 8;
  __shared__ f32x4_t red[kScoreWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int id = blockIdx.y * gridDim.x + blockIdx.x;
  for (int i = id * (kScoreWaves * 64) + threadIdx.x; i < ncount; i += gridDim.x * gridDim.y * kScoreWaves * 64)
    counters[i] = 0;
  const int e0 = blockIdx.x * 16, t0 = blockIdx.y * 16;
  const uint8_t* a = reinterpret_cast<const uint8_t*>(wg + (size_t)min(e0 + (lane & 15), E - 1) * H) + (lane >> 4) * 16;
  const uint8_t* b = reinterpret_cast<const uint8_t*>(x + (size_t)min(t0 + (lane & 15), nT - 1) * H) + (lane >> 4) * 16;
  const int S = H * (int)sizeof(T) / 64;
  const int s1 = (wave + 1) * S / kScoreWaves;
  f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
  int s = wave * S / kScoreWaves;
  for (; s + U <= s1; s += U) {
    u32x4_t av[U], bv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) av[u] = ld16(a + (size_t)(s + u) * 64), bv[u] = ld16(b + (size_t)(s + u) * 64);
#pragma unroll
    for (int u = 0; u < U; ++u) acc = mma16<T>(av[u], bv[u], acc);
  }
  for (; s < s1; ++s) acc = mma16<T>(ld16(a + (size_t)s * 64), ld16(b + (size_t)s * 64), acc);
  red[wave][lane] = acc;
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int q = 1; q < kScoreWaves; ++q) acc += red[q][lane];
  const int t = t0 + (lane & 15);
  if (t >= nT) return;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int e = e0 + (lane >> 4) * 4 + v;
    if (e < E) scores[(size_t)t * E + e] = acc[v];
  }
}

// ----------------------------------------------------------------- the queue

// acc[r][c] += rows of w[r] . rows of col[c] over the steps [s0, s1) of 64 bytes. The
// pointers are the lane's: row lane % 16 of its tile, 16 bytes at lane / 16. U steps are
// in flight while U are multiplied.
template <typename T, int NT, int U>
__device__ __forceinline__ void stream(const uint8_t* const (&w)[2], const uint8_t* const (&col)[NT],
                                       int s0, int s1, f32x4_t (&acc)[2][NT]) {
  u32x4_t wa[U][2], ca[U][NT], wb[U][2], cb[U][NT];
  auto load = [&](u32x4_t (&wv)[U][2], u32x4_t (&cv)[U][NT], int s) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int r = 0; r < 2; ++r) wv[u][r] = ld16(w[r] + (size_t)(s + u) * 64);
#pragma unroll
      for (int c = 0; c < NT; ++c) cv[u][c] = ld16(col[c] + (size_t)(s + u) * 64);
    }
  };
  auto mma = [&](const u32x4_t (&wv)[U][2], const u32x4_t (&cv)[U][NT]) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int c = 0; c < NT; ++c) acc[r][c] = mma16<T>(wv[u][r], cv[u][c], acc[r][c]);
  };
  int s = s0;
  if (s + U <= s1) {
    load(wa, ca, s);
    for (;;) {
      s += U;
      const bool more = s + U <= s1;
      if (more) load(wb, cb, s);
      mma(wa, ca);
      if (!more) break;
      s += U;
      const bool again = s + U <= s1;
      if (again) load(wa, ca, s);
      mma(wb, cb);
      if (!again) break;
    }
  }
  for (; s < s1; ++s) {
    u32x4_t cv[NT];
#pragma unroll
    for (int c = 0; c < NT; ++c) cv[c] = ld16(col[c] + (size_t)s * 64);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const u32x4_t wv = ld16(w[r] + (size_t)s * 64);
#pragma unroll
      for (int c = 0; c < NT; ++c) acc[r][c] = mma16<T>(wv, cv[c], acc[r][c]);
    }
  }
}

// Waits until *p has reached n, a second at most (100 ticks of this clock a microsecond).
__device__ __forceinline__ void wait_count(const unsigned* p, unsigned n) {
  const unsigned long long start = wall_clock64();
  while (__hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) < n) {
    __builtin_amdgcn_s_sleep(2);
    if (wall_clock64() - start > 100000000ull) break;
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
}

template <typename T, int NT, int EPX>
struct FewLds {
  static constexpr int S = tile_stride<kBT, kWaves>();
  union {
    struct {
      float sc[kBT * S];
      GroupLds<kBT, kWaves> g;
    } choice;
    f32x4_t red[kWaves][2][NT][64];
  };
  int idx[NT * 16][kSlots];  // -1 past k
  float w[NT * 16][kSlots];
  int mark[kMaxE];           // a pair of the expert, or -1
  int segs[kMaxE];           // the chosen experts, ascending
  int nseg, ticket;
};

// The pair (token, slot) of expert e among token t's, or -1; its weight in wt.
__device__ __forceinline__ int pair_of(const int (&idx)[kSlots], const float (&w)[kSlots], int t, int e,
                                       int k, float& wt) {
  int p = -1;
  wt = 0.0f;
#pragma unroll
  for (int j = 0; j < kSlots; ++j)
    if (idx[j] == e) p = t * k + j, wt = w[j];
  return p;
}

template <typename T, int NT, int EPX>
__global__ __launch_bounds__(kFewThreads, NT == 1 ? 4 : 2) void few_kernel(FewArgs a) {
  constexpr int U = NT == 4 ? 1 : 2;
  constexpr int ES = (int)sizeof(T);
  __shared__ FewLds<T, NT, EPX> L;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const bool gt = gated(a.act);

  // the choice, in every workgroup: it costs less than handing it round
  for (int i = tid; i < kMaxE; i += kFewThreads) L.mark[i] = -1;
  for (int i = tid; i < NT * 16 * kSlots; i += kFewThreads) {
    L.idx[i / kSlots][i % kSlots] = -1;
    L.w[i / kSlots][i % kSlots] = 0.0f;
  }
  for (int t0 = 0; t0 < a.T; t0 += kBT) {
    __syncthreads();
    for (int i = tid; i < kBT * EPX; i += kFewThreads) {
      const int e = min(i % EPX, a.E - 1);
      const float s = a.scores[(size_t)min(t0 + i / EPX, a.T - 1) * a.E + e];
      L.choice.sc[i / EPX * L.S + i % EPX] = a.bias != nullptr ? s + a.bias[e] : s;
    }
    __syncthreads();
    // rows of k: spread to rows of kSlots below
    int32_t* idx = &L.idx[0][0] + t0 * a.k;
    float* w = &L.w[0][0] + t0 * a.k;
    grouped_phase<kBT, EPX, kWaves>(L.choice.sc, L.choice.g, a.g, 0, min(kBT, a.T - t0), a.E, a.k, idx, w);
  }
  __syncthreads();
  int pi = -1;
  float pw = 0.0f;
  static_assert(NT * 16 * kSlots <= kFewThreads, "one thread a slot");
  if (tid < NT * 16 * kSlots && tid / kSlots < a.T && tid % kSlots < a.k) {
    pi = (&L.idx[0][0])[tid / kSlots * a.k + tid % kSlots];
    pw = (&L.w[0][0])[tid / kSlots * a.k + tid % kSlots];
    if (blockIdx.x == 0) {
      a.idx[tid / kSlots * a.k + tid % kSlots] = pi;
      a.w[tid / kSlots * a.k + tid % kSlots] = pw;
    }
  }
  __syncthreads();
  if (tid < NT * 16 * kSlots) {
    L.idx[tid / kSlots][tid % kSlots] = pi;
    L.w[tid / kSlots][tid % kSlots] = pw;
    if (pi >= 0) atomicMax(&L.mark[pi], tid / kSlots * a.k + tid % kSlots);
  }
  __syncthreads();
  if (wave == 0) {
    int n = 0;
    for (int e0 = 0; e0 < kMaxE; e0 += 64) {
      const bool in = L.mark[e0 + lane] >= 0;
      const unsigned long long m = __ballot(in);
      if (in) L.segs[n + __popcll(m & ((1ull << lane) - 1))] = e0 + lane;
      n += __popcll(m);
    }
    if (lane == 0) L.nseg = n;
  }
  __syncthreads();
  const int nseg = L.nseg;

  const int H = a.H, F = a.F, Fs = a.Fs;
  const int chunk = gt ? kCols / 2 : kCols;  // columns of h of an up task
  const int CS = Fs / chunk, CF = F / chunk;
  const int nup = CS + nseg * CF, ntile = H / kCols;
  const int total = nup + ntile * a.D;
  const int two = gt ? 2 : 1;
  T* h = static_cast<T*>(a.h);
  T* hs = h + (size_t)a.T * a.k * F;
  unsigned* done = a.counters + 1;  // [0]: shared expert, [1 + e]
  unsigned* arrived = done + a.E + 1;
  const int l16 = lane & 15, kq = lane >> 4;
  int tok[NT];  // the lane's token of each column tile
#pragma unroll
  for (int c = 0; c < NT; ++c) tok[c] = min(c * 16 + l16, a.T - 1);

  for (;;) {
    if (tid == 0) L.ticket = (int)__hip_atomic_fetch_add(a.counters, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    const int task = __builtin_amdgcn_readfirstlane(L.ticket);
    if (task >= total) return;
    f32x4_t acc[2][NT];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int c = 0; c < NT; ++c) acc[r][c] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

    if (task < nup) {
      const bool sh = task < CS;
      const int e = sh ? -1 : L.segs[(task - CS) / CF];
      const int f0 = (sh ? task : (task - CS) % CF) * chunk, N = sh ? Fs : F;
      const uint8_t* base = static_cast<const uint8_t*>(sh ? a.s_up : a.up) +
                            (sh ? 0 : (size_t)e * two * F * H * ES) + kq * 16;
      const uint8_t* wp[2] = {base + (size_t)(f0 + l16) * H * ES,
                              base + ((size_t)(gt ? N : 16) + f0 + l16) * H * ES};
      const uint8_t* cp[NT];
#pragma unroll
      for (int c = 0; c < NT; ++c) cp[c] = static_cast<const uint8_t*>(a.x) + (size_t)tok[c] * H * ES + kq * 16;
      const int S = H * ES / 64;
      stream<T, NT, U>(wp, cp, wave * S / kWaves, (wave + 1) * S / kWaves, acc);
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int c = 0; c < NT; ++c) L.red[wave][r][c][lane] = acc[r][c];
      __syncthreads();
      if (wave < NT) {
        // column tile `wave`
        f32x4_t v[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          v[r] = L.red[0][r][wave][lane];
#pragma unroll
          for (int q = 1; q < kWaves; ++q) v[r] += L.red[q][r][wave][lane];
        }
        const int t = wave * 16 + l16;
        float wt;
        const int p = t < a.T ? (sh ? t : pair_of(L.idx[t], L.w[t], t, e, a.k, wt)) : -1;
        if (p >= 0) {
          T* row = (sh ? hs + (size_t)p * Fs : h + (size_t)p * F) + f0 + kq * 4;
          const T* b = sh || a.b_up == nullptr ? nullptr
                                               : static_cast<const T*>(a.b_up) + (size_t)e * two * F + f0 + kq * 4;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            if (gt && r == 1) continue;
            Out4 bg{}, bu{}, none{};
            if (b != nullptr) {
              bg = load4(b + r * 16);
              if (gt) bu = load4(b + F);
            }
            const Out4 o = finish4<ES == 2>(a.act, v[r], v[1], bg, bu, false, none);
            if constexpr (ES == 2) *reinterpret_cast<uint2*>(row + r * 16) = pack4(o);
            else *reinterpret_cast<f32x4_t*>(row + r * 16) = f32x4_t{o.v[0], o.v[1], o.v[2], o.v[3]};
          }
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
        if (lane == 0)
          __hip_atomic_fetch_add(done + 1 + e, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    } else {
      // K slice d of all chosen experts' (the shared one's first) rows n0 .. n0 + 31 of down
      const int d = (task - nup) / ntile, nt = (task - nup) % ntile, n0 = nt * kCols;
      const int SS = Fs * ES / 64, SF = F * ES / 64;
      const long long all = SS + (long long)nseg * SF;
      const int lo = (int)(all * d / a.D), hi = (int)(all * (d + 1) / a.D);
      int s = lo + (int)((long long)(hi - lo) * wave / kWaves);
      const int end = lo + (int)((long long)(hi - lo) * (wave + 1) / kWaves);
      while (s < end) {
        const bool sh = s < SS;
        const int seg = sh ? 0 : (s - SS) / SF, e = sh ? -1 : __builtin_amdgcn_readfirstlane(L.segs[seg]);
        const int first = sh ? 0 : SS + seg * SF, K = sh ? Fs : F;
        const int stop = min(end, first + (sh ? SS : SF));
        const uint8_t* base = static_cast<const uint8_t*>(sh ? a.s_down : a.down) +
                              (sh ? 0 : (size_t)e * H * F * ES) + kq * 16;
        const uint8_t* wp[2] = {base + (size_t)(n0 + l16) * K * ES, base + (size_t)(n0 + 16 + l16) * K * ES};
        const uint8_t* cp[NT];
        float wt[NT];
        bool in[NT];
#pragma unroll
        for (int c = 0; c < NT; ++c) {
          // a token that did not choose the expert reads the row of one that did, and drops
          // the result
          int p = tok[c];
          wt[c] = 1.0f;
          if (!sh) p = pair_of(L.idx[tok[c]], L.w[tok[c]], tok[c], e, a.k, wt[c]);
          in[c] = p >= 0;
          if (p < 0) p = L.mark[e];
          cp[c] = reinterpret_cast<const uint8_t*>((sh ? hs : h) + (size_t)p * K) + kq * 16;
        }
        f32x4_t part[2][NT];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int c = 0; c < NT; ++c) part[r][c] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        wait_count(done + 1 + e, (unsigned)((sh ? CS : CF) * NT));
        stream<T, NT, U>(wp, cp, s - first, stop - first, part);
        if (!sh && s == first && a.b_down != nullptr) {  // the bias once, with the first part
          const T* b = static_cast<const T*>(a.b_down) + (size_t)e * H + n0 + kq * 4;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const Out4 bv = load4(b + r * 16);
#pragma unroll
            for (int c = 0; c < NT; ++c)
#pragma unroll
              for (int v = 0; v < 4; ++v) part[r][c][v] += bv.v[v];
          }
        }
#pragma unroll
        for (int c = 0; c < NT; ++c) {
          if (!in[c]) continue;
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[r][c][v] = fmaf(wt[c], part[r][c][v], acc[r][c][v]);
        }
        s = stop;
      }
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int c = 0; c < NT; ++c) L.red[wave][r][c][lane] = acc[r][c];
      __syncthreads();
      if (wave < NT) {
        f32x4_t v[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          v[r] = L.red[0][r][wave][lane];
#pragma unroll
          for (int q = 1; q < kWaves; ++q) v[r] += L.red[q][r][wave][lane];
        }
        bool last = true;
        if (a.D > 1) {
          // the slice that arrives last adds all of them up, in slice order
          float* P = a.part + ((size_t)nt * a.D * 2 * NT + wave) * 256 + lane * 4;
#pragma unroll
          for (int r = 0; r < 2; ++r)
            *reinterpret_cast<f32x4_t*>(P + (size_t)((d * 2 + r) * NT) * 256) = v[r];
          __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
          unsigned before = 0;
          if (lane == 0)
            before = __hip_atomic_fetch_add(arrived + nt * NT + wave, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          last = __builtin_amdgcn_readfirstlane(before) == (unsigned)(a.D - 1);
          if (last) {
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              f32x4_t q[kMaxDown];
#pragma unroll
              for (int i = 0; i < kMaxDown; ++i)  // all loads first, from clamped slices
                q[i] = *reinterpret_cast<const f32x4_t*>(P + (size_t)((min(i, a.D - 1) * 2 + r) * NT) * 256);
              v[r] = q[0];
#pragma unroll
              for (int i = 1; i < kMaxDown; ++i)
                if (i < a.D) v[r] += q[i];
            }
          }
        }
        const int t = wave * 16 + l16;
        if (last && t < a.T) {
          T* row = static_cast<T*>(a.out) + (size_t)t * H + n0 + kq * 4;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            if constexpr (ES == 2)
              *reinterpret_cast<uint2*>(row + r * 16) = make_uint2(cvt_bf16x2(v[r][0], v[r][1]), cvt_bf16x2(v[r][2], v[r][3]));
            else
              *reinterpret_cast<f32x4_t*>(row + r * 16) = v[r];
          }
        }
      }
    }
    __syncthreads();  // red and ticket are free
  }
}

// ----------------------------------------------------------------- host side

int col_tiles(int T) { return T <= 16 ? 1 : T <= 32 ? 2 : 4; }

// K slices of the down tasks: two tasks a CU, each wave of a task with 4 steps or more.
int down_slices(int H, int F, int Fs, int k, bool bf16) {
  const int steps = (int)(((long long)k * F + Fs) * (bf16 ? 2 : 4) / 64);
  int d = 1;
  while (d < kMaxDown && H / kCols * d * 2 <= 512 && steps / (d * 2) >= 4 * kWaves) d *= 2;
  return d;
}

struct FewLayout {
  size_t scores, h, part, counters, bytes;
};
FewLayout layout(int T, int H, int E, int k, int F, int Fs, bool bf16) {
  FewLayout l{};
  const int nt = col_tiles(T), D = down_slices(H, F, Fs, k, bf16);
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t p = at;
    at += align256(n);
    return p;
  };
  l.scores = take((size_t)T * E * 4);
  l.h = take(((size_t)T * k * F + (size_t)T * Fs) * (bf16 ? 2 : 4));
  l.part = take(D > 1 ? (size_t)(H / kCols) * D * 2 * nt * 1024 : 0);
  l.counters = take((size_t)counter_ints(E, H, nt) * 4);
  l.bytes = at;
  return l;
}

template <typename T, int NT>
hipError_t launch_queue(const FewArgs& a, int grid, hipStream_t s) {
  if (a.E <= 64) hipLaunchKernelGGL((few_kernel<T, NT, 64>), dim3(grid), dim3(kFewThreads), 0, s, a);
  else hipLaunchKernelGGL((few_kernel<T, NT, kMaxE>), dim3(grid), dim3(kFewThreads), 0, s, a);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_few_t(const FewArgs& a, const void* wg, hipStream_t s) {
  const int nt = col_tiles(a.T);
  hipLaunchKernelGGL((few_scores_kernel<T>), dim3((a.E + 15) / 16, (a.T + 15) / 16), dim3(kScoreWaves * 64),
                     0, s, static_cast<const T*>(a.x), static_cast<const T*>(wg), a.T, a.H, a.E, a.scores,
                     a.counters, counter_ints(a.E, a.H, nt));
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  // two workgroups a CU, no more than there are tasks
  const int chunk = a.act == kActGeglu || a.act == kActSwiglu ? kCols / 2 : kCols;
  const long long tasks = (long long)std::min(a.E, a.T * a.k) * (a.F / chunk) + a.Fs / chunk +
                          (long long)(a.H / kCols) * a.D;
  const int grid = (int)std::min(tasks, 512LL);
  switch (nt) {
    case 1: return launch_queue<T, 1>(a, grid, s);
    case 2: return launch_queue<T, 2>(a, grid, s);
    default: return launch_queue<T, 4>(a, grid, s);
  }
}

}  // namespace

int few_max_tokens() { return kFewT; }

size_t few_ws_bytes(int T, int H, int E, int k, int F, int Fs, bool bf16) {
  return layout(T, H, E, k, F, Fs, bf16).bytes;
}

hipError_t launch_few(const FewCall& c, hipStream_t s) {
  const FewLayout l = layout(c.T, c.H, c.E, c.k, c.F, c.Fs, c.bf16);
  uint8_t* ws = static_cast<uint8_t*>(c.ws);
  FewArgs a{};
  a.x = c.x, a.up = c.up, a.down = c.down, a.b_up = c.b_up, a.b_down = c.b_down;
  a.s_up = c.s_up, a.s_down = c.s_down;
  a.bias = c.bias_in_score ? c.bias : nullptr;
  a.g = group_args(c.bias_in_score ? nullptr : c.bias, c.E, c.softmax, c.groups, c.topk_groups,
                   c.group_top, c.renorm, c.scale);
  a.T = c.T, a.H = c.H, a.E = c.E, a.k = c.k, a.F = c.F, a.Fs = c.Fs, a.act = c.act;
  a.scores = reinterpret_cast<float*>(ws + l.scores);
  a.h = ws + l.h;
  a.part = reinterpret_cast<float*>(ws + l.part);
  a.counters = reinterpret_cast<unsigned*>(ws + l.counters);
  a.D = down_slices(c.H, c.F, c.Fs, c.k, c.bf16);
  a.idx = c.idx, a.w = c.w, a.out = c.out;
  return c.bf16 ? launch_few_t<uint16_t>(a, c.wg, s) : launch_few_t<float>(a, c.wg, s);
}

}  // namespace moe
