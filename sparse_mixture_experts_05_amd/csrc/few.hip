// A whole MoE layer for a few tokens (T <= 64): a launch for the scores, from 9 tokens on
// one for the choice, and one for choice (up to 8 tokens), experts, shared expert and
// combine. A decode step is a stream of the chosen experts' weights; what the layer's
// separate launches cost there is their drains and starts.
//
//   s[t,e]  = x[t] . wg[e] (+ bias[e])                    top-k as moe_route_grouped
//   h[t,j]  = act(x[t] . up[e_j]^T + b_up[e_j])           rounded to the layer's type
//   out[t]  = sum_j w[t,j] (h[t,j] . down[e_j]^T + b_down[e_j])  + shared expert(x[t])
//
// In the last launch every workgroup chooses for itself or loads the choice, and then has
// two kinds of tasks:
//   up    (unit, 16 weight rows of up: 16 columns of h, or 8 of a gated act), by ticket
//   down  (K slice, 16 columns of out) over all units, dealt out by workgroup
// A down task waits until every up task is done. A workgroup starts on its down tasks only
// when it has drawn a ticket past the last up task, so by then every up task is held by a
// workgroup that runs, and that waits for nothing before it is through with its tickets:
// the wait ends whatever number of workgroups is resident and whatever else the GPU runs.
// (It gives up after some seconds and writes NaN, few_rules.hpp: so a workspace that
// another call is using at the same time, which clears the counters, does not hang the GPU.
// That, and that no access leaves the operands, is all that is ensured then: what both calls
// write is undefined.)
//
// h is rounded to bf16 because the matrix instruction takes no wider operand (the separate
// calls do the same): out is 2.3e-3 of its norm from float64 with it and would be 1.7e-3, its
// own rounding, with h in two bf16 parts, at twice the MFMAs and twice h's way through memory.
//
// The pairs (token, chosen expert) are sorted by expert in every workgroup's LDS; up to 16
// pairs of an expert make a unit, the columns of one MFMA tile, and the shared expert has
// units of 16 tokens. Weights go straight to registers (nothing else on the chip reads
// them); the first steps of a task are loaded while the task before it is summed up and
// stored, those of the down weights while the last up tasks are waited for.
//
// Bound by HBM (T = 64 reads 5.8 TB/s of weights) and, for a token or two, by the launches'
// starts, the choice and the wait between up and down (18 of 1 token's 55 us). bf16, in a
// graph of 20 calls (eager the same within 2 %), against the separate calls (route, dispatch,
// products, combine), eager and in such a graph:
//   1 token, 128 experts of 4096 x 1536 swiglu, 8 chosen, one shared   75 us (111, 111)
//   16 tokens, 128 experts of 4096 x 1024 gelu, 8 chosen              224 us (253, 251)
//   64 tokens, 128 experts of 4096 x 1024 swiglu, 8 chosen            545 us (558, 557)
//   64 tokens, 64 experts of 256 x 512 swiglu, 8 chosen                55 us (62, 39)
// The separate calls are bound by the host when eager (62 us and more), not in a graph. Of
// their time in a graph, over 168 shapes with cold weights, this layer takes
//   experts of 3 MB (1024 x 512 gated) or more: 0.66 to 1.04 with up to 2 pairs an expert
//     (T k / E), 0.8 to 1.17 with 4, 0.9 to 1.17 with 8, 1.15 to 1.5 with 16 (an expert's
//     second unit is a second pass over its weights);
//   smaller ones: 0.9 to 1.06 with 1 token, 1 to 1.7 with 4 tokens or more (its steps wait
//     for each other, and launches of that size cost no more than the wait).
// 4 steps in flight a wave (R): 2, 3, 5, 6, 8, 12 and 16 are slower by 1 to 20 % (1 token of
// gelu 58.3 us; 62.7, 62.0, 64.9, 60.1, 61.6, 70.6, 69.0), as are two workgroups a CU (70.7).
#include <algorithm>

#include "few_rules.hpp"
#include "kernels.hpp"
#include "linear.hpp"
#include "route_choice.hpp"

namespace moe {
namespace {

using namespace lin;

constexpr int kWaves = 8;                 // streaming waves of a workgroup
constexpr int kFewT = 64, kPairs = kFewT * 8;  // tokens; pairs of a token and its expert
constexpr int kUnits = kMaxE + kPairs / 16 + kFewT / 16;  // at most
constexpr int kCols = 16;                 // weight rows of a task
constexpr int kMaxDown = 8;               // K slices of the down tasks
constexpr int kMaxScore = 8;              // K slices of the scores

struct FewArgs {
  const void *x, *up, *down, *b_up, *b_down, *s_up, *s_down;
  const float* bias;  // inside the scores, or null
  GroupArgs g;
  int T, H, E, k, F, Fs, act;
  float* scores;       // [KS, T, E]
  void* h;             // [T * k, F] in the order of the experts, then [T, Fs]
  float* part;         // [H / 16, D, T, 16]: partial columns of out
  unsigned* counters;  // tickets | up tasks done | go [kGo] | arrived [H / 16]
  int KS, D, batch;
  int32_t* idx;
  float* w;
  void* out;
};

// Tickets, done and every go have 512 bytes of their own: workgroups that wait would slow
// down those that count, and they look at one of kGo places, which the last up task sets.
constexpr int kLine = 128, kGo = 16;
constexpr int kArrived = (2 + kGo) * kLine;
static_assert((unsigned long long)kUnits * (1 << 20) / (kCols / 2) < few::kNoTicket, "tickets of all up tasks");
inline int counter_ints(int H) { return kArrived + H / kCols; }

// ----------------------------------------------------------------- scores

// 16 experts x 16 tokens x a slice of H a workgroup of 4 waves, which share the slice (64
// bytes of a row a step) and add their sums in wave order. Clears the counters of the
// last launch. The slices spread Wg over the CUs: one CU reads about 55 GB/s.
template <typename T>
__global__ __launch_bounds__(256) void few_scores_kernel(const T* __restrict__ x, const T* __restrict__ wg,
                                                        int nT, int H, int E, float* __restrict__ scores,
                                                        unsigned* __restrict__ counters, int ncount) {
  constexpr int U = 4, NW = 4;
  __shared__ f32x4_t red[NW][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int id = (blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
  for (int i = id * 256 + threadIdx.x; i < ncount; i += gridDim.x * gridDim.y * gridDim.z * 256) counters[i] = 0;
  const int e0 = blockIdx.x * 16, t0 = blockIdx.y * 16;
  const uint8_t* a = reinterpret_cast<const uint8_t*>(wg + (size_t)min(e0 + (lane & 15), E - 1) * H) + (lane >> 4) * 16;
  const uint8_t* b = reinterpret_cast<const uint8_t*>(x + (size_t)min(t0 + (lane & 15), nT - 1) * H) + (lane >> 4) * 16;
  const int S = H * (int)sizeof(T) / 64, parts = gridDim.z * NW, part = blockIdx.z * NW + wave;
  const int s1 = (int)((long long)(part + 1) * S / parts);
  f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
  int s = (int)((long long)part * S / parts);
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
  for (int q = 1; q < NW; ++q) acc += red[q][lane];
  const int t = t0 + (lane & 15);
  if (t >= nT) return;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int e = e0 + (lane >> 4) * 4 + v;
    if (e < E) scores[((size_t)blockIdx.z * nT + t) * E + e] = acc[v];
  }
}

// ----------------------------------------------------------------- handing over

// What workgroups hand to each other within the launch (h and the partial columns of out)
// goes past the caches that they do not share: stores at agent scope, which are complete
// at memory once vmcnt says so, and 16-byte loads with sc1, the same scope. Fences would do
// as well and write back and invalidate a whole XCD's L2 each (1 token of 128 experts
// 173 us, 113 this way).
__device__ __forceinline__ void put8(void* p, uint2 v) {
  __hip_atomic_store(static_cast<uint64_t*>(p), (uint64_t)v.y << 32 | v.x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void put16(void* p, const f32x4_t& v) {
  put8(p, make_uint2(__float_as_uint(v[0]), __float_as_uint(v[1])));
  put8(static_cast<uint8_t*>(p) + 8, make_uint2(__float_as_uint(v[2]), __float_as_uint(v[3])));
}
typedef __amdgpu_buffer_rsrc_t Shared;  // a buffer and its bytes: loads past it give zeros
__device__ __forceinline__ Shared shared_buffer(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00020000);
}
__device__ __forceinline__ u32x4_t get16(Shared b, uint32_t at, uint32_t uniform) {
  return __builtin_amdgcn_raw_buffer_load_b128(b, at, uniform, 16);  // sc1
}

// Everything that this wave stored is at memory; then *p counts n more.
__device__ __forceinline__ unsigned announce(unsigned* p, unsigned n = 1) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  unsigned before = 0;
  if ((threadIdx.x & 63) == 0) before = __hip_atomic_fetch_add(p, n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return __builtin_amdgcn_readfirstlane(before);
}

// Waits until *p is set; false if it has not been after kLooks looks, of about a
// microsecond each. Looks and not time: a workgroup that the GPU has put aside for
// another process does not look.
constexpr int kLooks = 1 << 22;
__device__ __forceinline__ bool wait_set(const unsigned* p) {
  for (int i = 0; i < kLooks; ++i) {
    if (__hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != 0) return true;
    __builtin_amdgcn_s_sleep(4);
  }
  return false;
}

// ----------------------------------------------------------------- the stream

// 16 rows of weights: their uniform base at the wave's first step, and the lane's offset
// (row lane % 16, 16 bytes at lane / 16).
struct Rows {
  const uint8_t* w;
  uint32_t lane;
  int steps;   // of 64 bytes a row
  int stride;  // bytes from one to the next
  __device__ __forceinline__ const uint8_t* at(int s) const { return w + (size_t)s * stride; }
};

// R steps of the weights and of the columns, in flight or landed.
template <int R>
struct Ring {
  u32x4_t w[R], c[R];
};

// The first steps of a stream. Steps past its end repeat the last one (and a stream
// without steps reads the row's start), which nobody multiplies.
template <int R, typename Col>
__device__ __forceinline__ void first_steps(Ring<R>& g, const Rows& w, Col col) {
#pragma unroll
  for (int u = 0; u < R; ++u) {  // in the order of their use
    const int s = min(u, max(w.steps - 1, 0));
    g.w[u] = ld16(w.at(s) + w.lane);
    g.c[u] = col(s);
    __builtin_amdgcn_sched_barrier(0);
  }
}
template <int R>
__device__ __forceinline__ void first_rows(Ring<R>& g, const Rows& w) {
#pragma unroll
  for (int u = 0; u < R; ++u) g.w[u] = ld16(w.at(min(u, max(w.steps - 1, 0))) + w.lane);
}
template <int R, typename Col>
__device__ __forceinline__ void first_cols(Ring<R>& g, int steps, Col col) {
#pragma unroll
  for (int u = 0; u < R; ++u) g.c[u] = col(min(u, max(steps - 1, 0)));
}

// Rows of w . columns over w's steps, the first R of which are in the ring. A step's place
// is refilled with the step R further on, or from there on with the first steps of the next
// stream, so that R steps are in flight at any time: the barrier between two tasks does not
// drain them. col(s, next): step s of the columns of this stream, or of the next one.
template <typename T, int R, typename Col>
__device__ __forceinline__ f32x4_t stream(Ring<R>& g, const Rows& w, const Rows& next, Col col) {
  const int S = w.steps, last = max(next.steps - 1, 0);
  f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
  int b = 0;
  do {  // one round at least, which fetches the next stream's
#pragma unroll
    for (int u = 0; u < R; ++u) {
      const bool live = b + u < S;  // a last, partial round multiplies zeros
      const u32x4_t zero = {0, 0, 0, 0};
      acc = mma16<T>(live ? g.w[u] : zero, live ? g.c[u] : zero, acc);
      const bool more = b + u + R < S;
      const int s = more ? b + u + R : min(u, last);
      const uint8_t* base = more ? w.at(s) : next.at(s);
      g.w[u] = ld16(base + (more ? w.lane : next.lane));
      g.c[u] = col(s, !more);
      __builtin_amdgcn_sched_barrier(0);  // loads stay in the order of their use
    }
    b += R;
  } while (b < S);
  return acc;
}

// ----------------------------------------------------------------- the queue

struct FewLds {
  static constexpr int S = tile_stride<kWaves, kWaves>();
  union {
    struct {
      float sc[kWaves * S];
      GroupLds<kWaves, kWaves> g;
      int idx[kPairs];
      float w[kPairs];
      int count[kWaves][kMaxE];  // pairs of each expert by wave; then [0]: its first place
    } choice;
    f32x4_t red[2][kWaves][64];               // up: the waves' sums of two tasks in turn
    float out[2][kWaves][kFewT][kCols];       // down: each wave's part of the columns of out
  };
  int tok[kPairs];     // by place in the experts' order: the pair's token
  float w[kPairs];     // and weight
  // a unit: its expert (-1: the shared one), first place (the shared one's: token) and pairs
  int expert[kUnits], first[kUnits], pairs[kUnits];
  int units, start[2], ticket[2];  // a workgroup's first tickets, then every next one in turn
};

// The scores of token t, expert i * 64 + lane, summed in slice order.
template <int EPX>
__device__ __forceinline__ void sum_scores(const FewArgs& a, int t, float* row) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < EPX / 64; ++i) {
    const int e = min(i * 64 + lane, a.E - 1);
    float v[kMaxScore];
#pragma unroll
    for (int q = 0; q < kMaxScore; ++q) v[q] = a.scores[((size_t)min(q, a.KS - 1) * a.T + t) * a.E + e];
    float s = v[0];
#pragma unroll
    for (int q = 1; q < kMaxScore; ++q)
      if (q < a.KS) s += v[q];
    row[i * 64 + lane] = a.bias != nullptr ? s + a.bias[e] : s;
  }
}

// The choice as a launch of its own, a token a workgroup of one wave, for more than kOwn
// tokens: the workgroups of the last launch choose up to kOwn, a token a wave, in what
// the launch costs (6 us), but take a wave's tokens one after another (5.5 us a token:
// 16 tokens 17 us, 64 49).
constexpr int kOwn = kWaves;
template <int EPX>
__global__ __launch_bounds__(64) void few_choice_kernel(FewArgs a) {
  __shared__ float sc[tile_stride<1, 1>()];
  __shared__ GroupLds<1, 1> g;
  const int t = blockIdx.x;
  sum_scores<EPX>(a, t, sc);
  wave_lds_fence();
  grouped_phase<1, EPX, 1>(sc, g, a.g, t, a.T, a.E, a.k, a.idx, a.w);
}

// The choice of every token, or its loads; the pairs in the experts' order, and the units:
// the shared expert's, then each expert's. One wave a token, for itself, then one thread a
// pair. The wave that finishes tasks draws the workgroup's first ticket meanwhile, and where a
// ticket is one task the second, when every workgroup has its first.
__device__ __forceinline__ int draw_ticket(const FewArgs& a) {
  return few::ticket_number(__hip_atomic_fetch_add(a.counters, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
}

template <int EPX>
__device__ __forceinline__ void choose(const FewArgs& a, FewLds& L) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const bool drawer = tid == kWaves * 64;
  if (drawer) L.start[0] = draw_ticket(a);
  const bool own = a.T <= kOwn;
  if (own && wave < a.T) {
    sum_scores<EPX>(a, wave, L.choice.sc + wave * L.S);
    wave_lds_fence();
    grouped_phase<kWaves, EPX, kWaves>(L.choice.sc, L.choice.g, a.g, 0, a.T, a.E, a.k, L.choice.idx, L.choice.w);
  }
  for (int i = tid; i < kWaves * kMaxE; i += kWaves * 64) (&L.choice.count[0][0])[i] = 0;
  lds_barrier();
  if (drawer && a.batch == 1) L.start[1] = draw_ticket(a);
  // Places have to be the same in every workgroup: pairs of an expert keep their order.
  // Pairs of this wave with the lane's expert: by the 8 bits of its number.
  const bool pair = tid < a.T * a.k;  // the streams' threads
  static_assert(kPairs <= kWaves * 64 && kMaxE <= 256, "one thread a pair");
  int e = 0, rank = 0;
  float w = 0.0f;
  if (pair) {
    e = own ? L.choice.idx[tid] : a.idx[tid];
    w = own ? L.choice.w[tid] : a.w[tid];
    if (own && blockIdx.x == 0) a.idx[tid] = e, a.w[tid] = w;
    unsigned long long same = __ballot(true);
#pragma unroll
    for (int bit = 0; bit < 8; ++bit) {
      const unsigned long long on = __ballot((e >> bit) & 1);
      same &= (e >> bit) & 1 ? on : ~on;
    }
    rank = __popcll(same & ((1ull << lane) - 1));
    if (rank == 0) L.choice.count[wave][e] = __popcll(same);
  }
  lds_barrier();
  if (pair)
    for (int q = 0; q < wave; ++q) rank += L.choice.count[q][e];
  lds_barrier();
  if (wave == 0) {
    // places and units before each of this lane's 4 experts
    int c[4], places = 0, units = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = 0;
#pragma unroll
      for (int q = 0; q < kWaves; ++q) c[i] += L.choice.count[q][lane * 4 + i];
      places += c[i];
      units += (c[i] + 15) / 16;
    }
    int p = places, u = units;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int vp = __shfl_up(p, d), vu = __shfl_up(u, d);
      if (lane >= d) p += vp, u += vu;
    }
    const int su = a.Fs > 0 ? (a.T + 15) / 16 : 0;
    if (lane == 63) L.units = su + u;
    p -= places;
    u += su - units;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      L.choice.count[0][lane * 4 + i] = p;
      for (int q = 0; q < c[i]; q += 16, ++u) {
        L.expert[u] = lane * 4 + i;
        L.first[u] = p + q;
        L.pairs[u] = min(16, c[i] - q);
      }
      p += c[i];
    }
    if (lane < su) {
      L.expert[lane] = -1;
      L.first[lane] = lane * 16;
      L.pairs[lane] = min(16, a.T - lane * 16);
    }
  }
  lds_barrier();
  if (pair) {
    const int at = L.choice.count[0][e] + rank;
    L.tok[at] = tid / a.k;
    L.w[at] = w;
  }
  lds_barrier();
}

template <typename T>
__device__ __forceinline__ void store4(T* row, const f32x4_t& v) {
  if constexpr (sizeof(T) == 2)
    *reinterpret_cast<uint2*>(row) = make_uint2(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]));
  else
    *reinterpret_cast<f32x4_t*>(row) = v;
}

// kWaves waves stream weights; one more sums up what those made of a task, finishes it and
// draws the tickets while the streams go on with the next task.
template <typename T, int EPX>
__global__ __launch_bounds__((kWaves + 1) * 64, 3) void few_kernel(FewArgs a) {
  constexpr int R = 4;
  constexpr int ES = (int)sizeof(T);
  __shared__ FewLds L;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  choose<EPX>(a, L);
  auto uni = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
  const bool gt = gated(a.act);
  const int H = a.H, F = a.F, Fs = a.Fs, units = uni(L.units);
  const int su = Fs > 0 ? (a.T + 15) / 16 : 0;  // the shared expert's units
  const int chunk = gt ? kCols / 2 : kCols;     // columns of h of an up task
  const int CS = Fs / chunk, CF = F / chunk;
  const int nup = su * CS + (units - su) * CF, ntile = H / kCols, ndown = ntile * a.D;
  T* h = static_cast<T*>(a.h);
  const size_t shared_at = (size_t)a.T * a.k * F;  // the shared expert's rows (elements)
  const int l16 = lane & 15, kq = lane >> 4;
  struct Task {
    int unit, f0;  // first column of h
  };
  auto up_task = [&](int t) {
    const int r = t - su * CS;
    return r < 0 ? Task{t / CS, t % CS * chunk} : Task{su + r / CF, r % CF * chunk};
  };
  // A ticket is `batch` tasks one behind the other (a power of two).
  int t0 = uni(L.start[0]) * a.batch, t1 = a.batch == 1 ? uni(L.start[1]) : t0 + 1;
  auto draws = [&](int t) { return ((t + 1) & (a.batch - 1)) == 0; };  // behind task t
  int task = blockIdx.x;

  if (wave == kWaves) {
    int turn = 0;
    unsigned finished = 0;
    for (; t0 < nup; ++finished) {
      if (lane == 0 && draws(t1)) L.ticket[turn] = draw_ticket(a);
      lds_barrier();
      // sums in wave order; with a gate, the up half is in the lanes 32 further on
      f32x4_t v = L.red[turn][0][lane], u = L.red[turn][0][lane ^ 32];
#pragma unroll
      for (int q = 1; q < kWaves; ++q) v += L.red[turn][q][lane], u += L.red[turn][q][lane ^ 32];
      const Task k = up_task(t0);
      const int e = uni(L.expert[k.unit]);
      if (l16 < L.pairs[k.unit] && (!gt || kq < 2)) {
        const size_t r = L.first[k.unit] + l16;
        T* row = (e < 0 ? h + shared_at + r * Fs : h + r * F) + k.f0 + kq * 4;
        Out4 bg{}, bu{}, none{};
        if (e >= 0 && a.b_up != nullptr) {
          const T* b = static_cast<const T*>(a.b_up) + (size_t)e * (gt ? 2 : 1) * F + k.f0 + kq * 4;
          bg = load4(b);
          if (gt) bu = load4(b + F);
        }
        const Out4 o = finish4<ES == 2>(a.act, v, u, bg, bu, false, none);
        if constexpr (ES == 2) put8(row, pack4(o));
        else put16(row, f32x4_t{o.v[0], o.v[1], o.v[2], o.v[3]});
      }
      t0 = t1;
      t1 = draws(t1) ? uni(L.ticket[turn]) * a.batch : t1 + 1;
      turn ^= 1;
    }
    // all of them at once: a wait for the stores and the count after every task is in the way
    // of the next one (64 tokens of 64 experts 2048 x 1024 223 -> 203 us)
    if (finished > 0 && announce(a.counters + kLine, finished) + finished == (unsigned)nup && lane < kGo)
      __hip_atomic_store(a.counters + (2 + lane) * kLine, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (task >= ndown) return;
    const bool done = wait_set(a.counters + (2 + blockIdx.x % kGo) * kLine);
    lds_barrier();
    const few::Slice what = few::slice_step(done, a.D);
    for (turn = 0; task < ndown; task += gridDim.x, turn ^= 1) {
      lds_barrier();
      const int d = task / ntile, nt = task % ntile;
      // lane l has columns 4 (l % 4) .. + 3 of token l / 4 and every 16th after it
      const int n = (a.T + 15) / 16, c = (lane & 3) * 4;
      f32x4_t v[kFewT / 16];
#pragma unroll
      for (int i = 0; i < kFewT / 16; ++i) {
        if (i >= n) continue;
        const int t = min(i * 16 + (lane >> 2), a.T - 1);
        v[i] = *reinterpret_cast<const f32x4_t*>(&L.out[turn][0][t][c]);
#pragma unroll
        for (int q = 1; q < kWaves; ++q) v[i] += *reinterpret_cast<const f32x4_t*>(&L.out[turn][q][t][c]);
        if (what == few::kGiveUp) v[i] = f32x4_t{NAN, NAN, NAN, NAN};
      }
      if (what == few::kHandOver) {
        // the slice that arrives last adds all of them up, in slice order
        const uint32_t tile = (uint32_t)a.T * kCols * 4, at = (uint32_t)(nt * a.D) * tile + lane * 16;
        uint8_t* P = reinterpret_cast<uint8_t*>(a.part) + at + d * tile;
#pragma unroll
        for (int i = 0; i < kFewT / 16; ++i)
          if (i < n && i * 16 + (lane >> 2) < a.T) put16(P + i * 1024, v[i]);
        if (!few::adds_up(announce(a.counters + kArrived + nt), a.D)) continue;
        const Shared pb = shared_buffer(a.part, (uint32_t)ndown * tile);
#pragma unroll
        for (int i = 0; i < kFewT / 16; ++i) {
          if (i >= n) continue;
          u32x4_t q[kMaxDown];
#pragma unroll
          for (int j = 0; j < kMaxDown; ++j)  // all loads first, from clamped slices
            q[j] = get16(pb, at + i * 1024, (uint32_t)min(j, a.D - 1) * tile);
          v[i] = __builtin_bit_cast(f32x4_t, q[0]);
#pragma unroll
          for (int j = 1; j < kMaxDown; ++j)
            if (j < a.D) v[i] += __builtin_bit_cast(f32x4_t, q[j]);
        }
      }
#pragma unroll
      for (int i = 0; i < kFewT / 16; ++i) {
        const int t = i * 16 + (lane >> 2);
        if (t < a.T) store4(static_cast<T*>(a.out) + (size_t)t * H + nt * kCols + c, v[i]);
      }
    }
    return;
  }

  // the streams
  // The steps of an up task go round the waves, so that what the workgroups read at one
  // time lies anywhere in the rows: with a slice of a row each (1 KiB of 4096 bf16), all
  // were at addresses with the same bits 6 to 9, which some of the HBM channels hold (64
  // tokens of 128 experts 645 -> 587 us, 1 token 78.5 -> 75.3; 128 bytes at a time 640).
  const int SH = H * ES / 64, lo = min(wave, SH - 1), mine = (SH - wave + kWaves - 1) / kWaves;
  auto x_step = [&](int s) { return (lo + s * kWaves) * 64; };
  struct Up {
    Rows rows;
    uint32_t col;  // the lane's row of x
  };
  auto up = [&](int t) {
    const Task k = up_task(t);
    const int e = uni(L.expert[k.unit]), N = e < 0 ? Fs : F;
    Up u;
    u.rows.w = static_cast<const uint8_t*>(e < 0 ? a.s_up : a.up) +
               (e < 0 ? 0 : (size_t)e * (gt ? 2 : 1) * F * H * ES) + (size_t)k.f0 * H * ES + lo * 64;
    // with a gate, 8 gate rows and the 8 up rows of the same columns
    const uint32_t row = gt ? (l16 & 7) + (l16 >> 3) * N : l16;
    u.rows.lane = row * (uint32_t)(H * ES) + kq * 16;
    u.rows.steps = mine;  // none if the row is that short
    u.rows.stride = kWaves * 64;
    const int p = L.first[k.unit] + min(l16, L.pairs[k.unit] - 1);
    u.col = (uint32_t)((e < 0 ? p : L.tok[p]) * H * ES + kq * 16);
    return u;
  };
  const Shared xb = shared_buffer(a.x, (uint32_t)a.T * H * ES);

  // A piece of a down task: steps of one unit in this wave's part of the task's K slice.
  struct Piece {
    Rows rows;
    uint32_t col, at;   // the lane's row of h and the first byte of it
    int unit, s, n0;    // first step among all units', first column of the task
    bool first;         // has the unit's first step
  };
  const Shared hb = shared_buffer(h, (uint32_t)((shared_at + (size_t)a.T * Fs) * ES));
  const int SS = Fs * ES / 64, SF = F * ES / 64, all = su * SS + (units - su) * SF;
  auto piece = [&](int n0, int s0, int end) {
    Piece p;
    const int s = min(s0, all - 1), r = s - su * SS;  // an empty piece points at something
    const bool sh = r < 0;
    p.unit = sh ? s / SS : su + r / SF;
    const int first = sh ? p.unit * SS : su * SS + (p.unit - su) * SF, K = sh ? Fs : F;
    const int e = uni(L.expert[p.unit]);
    p.s = s0, p.n0 = n0;
    p.rows.stride = 64;
    p.rows.steps = max(0, min(end, first + (sh ? SS : SF)) - s0);
    p.first = s == first;
    p.at = (uint32_t)(s - first) * 64;
    p.rows.w = static_cast<const uint8_t*>(sh ? a.s_down : a.down) + (sh ? 0 : (size_t)e * H * F * ES) +
               (size_t)n0 * K * ES + p.at;
    p.rows.lane = (uint32_t)(l16 * K * ES + kq * 16);
    const size_t row = L.first[p.unit] + min(l16, L.pairs[p.unit] - 1);
    p.col = (uint32_t)(((sh ? shared_at : 0) + row * K) * ES) + kq * 16;
    return p;
  };
  auto wave_end = [&](int t, int w) {  // step at which the part of wave w - 1 ends
    const int d = t / ntile;
    const int from = (int)((long long)all * d / a.D), to = (int)((long long)all * (d + 1) / a.D);
    return from + (int)((long long)(to - from) * w / kWaves);
  };
  auto first_piece = [&](int t) { return piece(t % ntile * kCols, wave_end(t, wave), wave_end(t, wave + 1)); };

  Piece p = first_piece(min(task, ndown - 1));
  Ring<R> ring;
  int turn = 0;
  if (t0 < nup) {
    Up u = up(t0);
    first_steps(ring, u.rows, [&](int s) { return __builtin_amdgcn_raw_buffer_load_b128(xb, u.col, x_step(s), 0); });
    while (t0 < nup) {
      const bool more = t1 < nup;  // else the down weights, whose rows of h are not there yet
      Up n;
      n.rows = p.rows, n.col = 0;
      if (more) n = up(t1);
      L.red[turn][wave][lane] = stream<T>(ring, u.rows, n.rows, [&](int s, bool next) {
        return __builtin_amdgcn_raw_buffer_load_b128(xb, next ? n.col : u.col, next && !more ? 0 : x_step(s), 0);
      });
      lds_barrier();
      t0 = t1;
      t1 = draws(t1) ? uni(L.ticket[turn]) * a.batch : t1 + 1;
      turn ^= 1;
      u = n;
    }
  } else if (task < ndown) {
    first_rows(ring, p.rows);
  }
  if (task >= ndown) return;
  lds_barrier();  // every up task is done: no load from h before this, and red is read
  first_cols(ring, p.rows.steps, [&](int s) { return get16(hb, p.col, p.at + s * 64); });
  for (turn = 0; task < ndown; task += gridDim.x, turn ^= 1) {
    float (*out)[kCols] = L.out[turn][wave];
    for (int i = lane; i < a.T * (kCols / 4); i += 64)
      *reinterpret_cast<f32x4_t*>(&out[i >> 2][(i & 3) * 4]) = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    const int end = wave_end(task, wave + 1);
    for (bool more = true; more;) {
      more = p.s + p.rows.steps < end;
      const Piece q = more ? piece(p.n0, p.s + p.rows.steps, end)
                           : first_piece(task + (int)gridDim.x < ndown ? task + (int)gridDim.x : task);
      f32x4_t part = stream<T>(ring, p.rows, q.rows, [&](int s, bool next) {
        return get16(hb, next ? q.col : p.col, (next ? q.at : p.at) + s * 64);
      });
      if (p.rows.steps > 0 && l16 < L.pairs[p.unit]) {
        const int e = L.expert[p.unit], place = L.first[p.unit] + l16;
        if (p.first && e >= 0 && a.b_down != nullptr) {  // the bias once, with the first part
          const Out4 b = load4(static_cast<const T*>(a.b_down) + (size_t)e * H + p.n0 + kq * 4);
#pragma unroll
          for (int v = 0; v < 4; ++v) part[v] += b.v[v];
        }
        const int t = e < 0 ? place : L.tok[place];
        const float w = e < 0 ? 1.0f : L.w[place];
        f32x4_t* at = reinterpret_cast<f32x4_t*>(&out[t][kq * 4]);
        f32x4_t o = *at;
#pragma unroll
        for (int v = 0; v < 4; ++v) o[v] = fmaf(w, part[v], o[v]);
        *at = o;
      }
      p = q;
    }
    lds_barrier();
  }
}

// ----------------------------------------------------------------- host side

// K slices of the down tasks: a task a CU, each wave of a task with 4 steps or more.
int down_slices(int T, int H, int E, int k, int F, int Fs, bool bf16) {
  const long long cols = (long long)std::min(E, T * k) * F + (long long)(T + 15) / 16 * Fs;
  const long long steps = cols * (bf16 ? 2 : 4) / 64;
  int d = 1;
  while (d < kMaxDown && H / kCols * d * 2 <= 256 && steps / (d * 2) >= 4 * kWaves) d *= 2;
  return d;
}

// Tasks of a ticket: up to 8 and 128 KiB of weights, with two tickets a CU. The workgroups'
// draws from one counter are 10 ns apart, 2.7 us a round of 256, in which a CU reads 55 KB:
// 64 tokens of 64 experts 256 x 512 75 us with a task a ticket, 54 so; 2048 x 1024 204 and
// 188; 32 tokens of 200 experts 128 x 1024 242 and 145 (16 or 32 tasks: 153, 173).
int batch_tasks(int T, int H, int E, int k, int F, int act, bool bf16) {
  const int chunk = act == kActGeglu || act == kActSwiglu ? kCols / 2 : kCols;
  const long long tasks = (long long)std::min(E, T * k) * (F / chunk), bytes = (long long)kCols * H * (bf16 ? 2 : 4);
  int n = 1;
  while (n < 8 && bytes * n * 2 <= 131072 && tasks >= 512LL * n * 2) n *= 2;
  return n;
}

// K slices of the scores: up to 128 workgroups, each wave of one with a step or more.
int score_slices(int T, int H, int E, bool bf16) {
  const int tiles = ((E + 15) / 16) * ((T + 15) / 16), steps = H * (bf16 ? 2 : 4) / 64;
  int n = 1;
  while (n < kMaxScore && tiles * n * 2 <= 128 && steps >= 8 * n) n *= 2;
  return n;
}

struct FewLayout {
  size_t scores, h, part, counters, bytes;
};
FewLayout layout(int T, int H, int E, int k, int F, int Fs, bool bf16) {
  FewLayout l{};
  const int D = down_slices(T, H, E, k, F, Fs, bf16);
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t p = at;
    at += align256(n);
    return p;
  };
  l.scores = take((size_t)score_slices(T, H, E, bf16) * T * E * 4);
  l.h = take(((size_t)T * k * F + (size_t)T * Fs) * (bf16 ? 2 : 4));
  l.part = take(D > 1 ? (size_t)(H / kCols) * D * T * kCols * 4 : 0);
  l.counters = take((size_t)counter_ints(H) * 4);
  l.bytes = at;
  return l;
}

template <typename T>
hipError_t launch_few_t(const FewArgs& a, const void* wg, hipStream_t s) {
  hipLaunchKernelGGL((few_scores_kernel<T>), dim3((a.E + 15) / 16, (a.T + 15) / 16, a.KS), dim3(256), 0, s,
                     static_cast<const T*>(a.x), static_cast<const T*>(wg), a.T, a.H, a.E, a.scores,
                     a.counters, counter_ints(a.H));
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  // a workgroup a CU, no more than there are tasks
  const int chunk = a.act == kActGeglu || a.act == kActSwiglu ? kCols / 2 : kCols;
  const long long tasks = (long long)std::min(a.E, a.T * a.k) * (a.F / chunk) + a.Fs / chunk +
                          (long long)(a.H / kCols) * a.D;
  const dim3 grid((unsigned)std::min(tasks, 256LL)), block((kWaves + 1) * 64);
  auto choose_and_run = [&](auto epx) {
    constexpr int EPX = decltype(epx)::value;
    if (a.T > kOwn) {
      hipLaunchKernelGGL((few_choice_kernel<EPX>), dim3(a.T), dim3(64), 0, s, a);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((few_kernel<T, EPX>), grid, block, 0, s, a);
    return hipGetLastError();
  };
  if (a.E <= 64) return choose_and_run(std::integral_constant<int, 64>{});
  if (a.E <= 128) return choose_and_run(std::integral_constant<int, 128>{});
  return choose_and_run(std::integral_constant<int, kMaxE>{});
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
  a.KS = score_slices(c.T, c.H, c.E, c.bf16);
  a.D = down_slices(c.T, c.H, c.E, c.k, c.F, c.Fs, c.bf16);
  a.batch = batch_tasks(c.T, c.H, c.E, c.k, c.F, c.act, c.bf16);
  a.idx = c.idx, a.w = c.w, a.out = c.out;
  return c.bf16 ? launch_few_t<uint16_t>(a, c.wg, s) : launch_few_t<float>(a, c.wg, s);
}

}  // namespace moe
