// Pieces shared by the routing kernels: the sorted key lists of the top-k,
// the MFMA score tile, and the score launch of the two-launch paths with the
// rules that choose a path. Included by the .hip files that route; everything
// is local to the including file.
#pragma once

#include "common.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxE = 256;

// Row stride (floats) of a score tile of BT tokens in a workgroup of NW
// waves. The top-k gives each token G = 64*NW/BT consecutive lanes; lane g of
// a token reads the columns g, g + G, ..., so a stride of G (mod 64) puts the
// 64 lanes of a wave on 64 distinct banks.
template <int BT, int NW = 4>
constexpr int tile_stride() { return kMaxE + NW * 64 / BT; }

// ---------------------------------------------------------------- top-k
// Every (score, expert) pair is one 64-bit key: the score's bits mapped to an
// order-preserving unsigned integer in the high half, the complement of the
// expert id in the low half. A larger key is a better entry: a higher score,
// or an equal score with a lower id. A NaN score reads as -inf and -0 as +0
// (they compare equal). Key 0 is below every real entry and marks an empty
// slot, so the k chosen ids are always real, distinct and < E.
// Written with arithmetic only (max with -inf drops a NaN, adding +0 turns
// -0 into +0, the sign mask flips the order of negatives): as selects the
// compiler turned the mapping into three nested branches per key.
__device__ __forceinline__ uint64_t topk_key(float s, int e) {
  const uint32_t u = __float_as_uint(fmaxf(s, -INFINITY) + 0.0f);
  const uint32_t o = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
  return ((uint64_t)o << 32) | (uint32_t)(~(uint32_t)e);
}
__device__ __forceinline__ float key_score(uint64_t key) {
  const uint32_t o = (uint32_t)(key >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ int key_expert(uint64_t key) { return (int)(~(uint32_t)key); }

__device__ __forceinline__ void cswap(uint64_t& a, uint64_t& b) {  // a <- max, b <- min
  const bool gt = a > b;
  const uint64_t hi = gt ? a : b, lo = gt ? b : a;
  a = hi;
  b = lo;
}

// Sorts a bitonic sequence of N keys into descending order (half-cleaners).
template <int N>
__device__ __forceinline__ void bitonic_clean(uint64_t (&c)[N]) {
#pragma unroll
  for (int st = N / 2; st > 0; st >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((i & st) == 0) cswap(c[i], c[i + st]);
}

// Sorts N keys into descending order (bitonic sorting network).
template <int N>
__device__ __forceinline__ void bitonic_sort(uint64_t (&c)[N]) {
#pragma unroll
  for (int size = 2; size <= N; size <<= 1)
#pragma unroll
    for (int st = size / 2; st > 0; st >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i)
        if ((i & st) == 0) {
          if ((i & size) == 0) cswap(c[i], c[i + st]);
          else cswap(c[i + st], c[i]);
        }
}

// list <- the N largest of list and blk (both sorted descending): the
// elementwise max of list and reversed blk is bitonic and holds them.
template <int N>
__device__ __forceinline__ void merge_top(uint64_t (&list)[N], const uint64_t (&blk)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) list[i] = list[i] > blk[N - 1 - i] ? list[i] : blk[N - 1 - i];
  bitonic_clean<N>(list);
}

// Merge the lists of the G lanes of a token, levels 0 .. log2(G)-1; every
// lane ends with the same list.
template <int L, int G, int N>
__device__ __forceinline__ void group_merge(uint64_t (&list)[N]) {
  if constexpr ((1 << L) < G) {
    uint64_t other[N];
#pragma unroll
    for (int i = 0; i < N; ++i) other[i] = partner64<L>(list[i]);
    merge_top<N>(list, other);
    group_merge<L + 1, G, N>(list);
  }
}

// Sum over the G lanes of a token: each level adds a lane's value and its
// partner's, and fp addition is commutative, so every lane gets the same bits.
template <int L, int G>
__device__ __forceinline__ float group_sum(float v) {
  if constexpr ((1 << L) < G) return group_sum<L + 1, G>(v + __uint_as_float(partner<L>(__float_as_uint(v))));
  return v;
}

// bf16 scores on MFMA 16x16x32 with operands staged in LDS. One workgroup
// (4 waves) computes a BT x EP tile of scores: BT tokens and EP experts
// starting at expert e0, over the K panels [kp0, kp1) of 64 elements.
// A panel holds the BT token rows, then the EP expert rows (R rows in all, a
// multiple of 32; rows past the data repeat a valid row and are never used),
// 128 bytes each. Rows are copied global -> LDS with global_load_lds: one
// instruction moves 8 rows, 8 consecutive lanes reading one whole 128-byte
// line. NS stages of PPS panels rotate through LDS, so two stages are in
// flight while one is multiplied. Chunk c (16 bytes) of LDS row r sits at
// slot c ^ ((r >> 1) & 7): a 128-bit read by 16 lanes (16 consecutive rows,
// one chunk) then touches 16 distinct 4-bank groups.
// Work split over the NW waves: EP >= 64, wave w computes experts
// [w*EP/NW, (w+1)*EP/NW) over all panels; EP < 64, wave w takes the panels
// p = w (mod NW) of every stage for the whole tile and the NW partial tiles
// are summed in wave order.
template <int BT, int EP, int NW = 4>
struct RouteTile {
  static constexpr int R = (BT + EP + 31) / 32 * 32;  // rows per panel
  static constexpr int PB = R * 128;                  // panel bytes
  static constexpr bool KSPLIT = EP < 64;
  static constexpr int PPS_RAW = (40 * 1024) / PB < 1 ? 1 : (40 * 1024) / PB;
  // panels per stage: a multiple of 4 when the waves split them, else <= 2
  static constexpr int PPS = KSPLIT ? (PPS_RAW >= 8 ? 8 : 4) : (PPS_RAW > 2 ? 2 : PPS_RAW);
  static constexpr int SB = PPS * PB;                 // stage bytes
  static constexpr int NS = 3;                        // stages
  static constexpr int NI = PPS * R / 8 / NW;         // DMA instructions per wave per stage
  static constexpr int MC = BT / 16;                  // 16-row tiles per wave
  static constexpr int NC = KSPLIT ? EP / 16 : EP / 16 / NW;  // 16-column tiles per wave
  static constexpr int SC_BYTES = BT * tile_stride<BT, NW>() * 4;
  static constexpr int PART_BYTES = KSPLIT ? NW * BT * EP * 4 : 0;
  static constexpr int LDS = NS * SB > SC_BYTES + PART_BYTES ? NS * SB : SC_BYTES + PART_BYTES;
  static_assert(PPS * R % (8 * NW) == 0, "whole DMA instructions per wave");
  static_assert(!KSPLIT || PPS % NW == 0, "the waves split each stage's panels evenly");
  static_assert(KSPLIT || NC >= 1, "whole 16-column tiles per wave");
  static_assert(NI < 32, "vmcnt range");
  static_assert(LDS <= 160 * 1024, "LDS budget");
};

// The K loop of one tile (T: bf16 bits or fp32; a panel is 128 bytes of a row, the
// K range in panels); returns with every wave's accumulators complete and
// the LDS free for reuse (after a barrier).
//
// SUMS: several partial sums per score, one for each half panel of a stage (fp32: two,
// over every other MFMA), added up behind the loop. In one chain over K every addition
// rounds a partial sum that grows to the score itself; n sums are n times smaller, and the
// rounding error falls to about a half with 2, a third with 4, a fifth with 8. Error of
// softmax weights against float64 where nothing slices K, in u = 2^-24: 64 tokens, E 256,
// fp32, H 2112 28.9 -> 5.9, H 4032 40.1 -> 8.9 (8 sums); 1024 tokens, E 128, fp32, H 4032
// 39.0 -> 12.5 (4); 64 tokens, bf16, H 4032 15.4 -> 4.9 (4); 16384 tokens 15.9 -> 8.5 (2).
// Held in registers that the tiles leave free; times within 3 % of one chain either way.
template <int BT, int EP, int NW = 4, typename T_ = uint16_t, bool SUMS = false>
__device__ __forceinline__ void score_tile(uint8_t* smem, const T_* __restrict__ x,
                                           const T_* __restrict__ wg, int t0, int T, int e0,
                                           int E, int H, int kp0, int kp1,
                                           f32x4_t (&acc)[RouteTile<BT, EP, NW>::MC][RouteTile<BT, EP, NW>::NC]) {
  using C = RouteTile<BT, EP, NW>;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int NST = (kp1 - kp0 + C::PPS - 1) / C::PPS;  // stages

  // DMA plan of this lane: instruction q copies rows [8g, 8g+8) of panel pq[q].
  const T_* src[C::NI];
  int pq[C::NI], dst[C::NI];
#pragma unroll
  for (int q = 0; q < C::NI; ++q) {
    const int j = wave * C::NI + q;
    const int p = j / (C::R / 8), g = j % (C::R / 8);
    const int r = 8 * g + (lane >> 3);
    const int chunk = (lane & 7) ^ ((r >> 1) & 7);
    const T_* row = r < BT ? x + (size_t)min(t0 + r, T - 1) * H
                                 : wg + (size_t)min(e0 + r - BT, E - 1) * H;
    src[q] = row + chunk * (int)(16 / sizeof(T_));
    pq[q] = p;
    dst[q] = p * C::PB + g * 1024;
  }
  auto issue = [&](int st) {
    uint8_t* base = smem + (st % C::NS) * C::SB;
#pragma unroll
    for (int q = 0; q < C::NI; ++q)
      lds_dma16(src[q] + (size_t)min(kp0 + st * C::PPS + pq[q], kp1 - 1) * (128 / sizeof(T_)), base + dst[q]);
  };

  // the sums besides acc, by panel of a stage, k step and MFMA
  constexpr int PS = SUMS && !C::KSPLIT ? C::PPS : 1;
  constexpr int JS = sizeof(T_) == 4 ? 2 : 1, NSUM = SUMS ? PS * 2 * JS : 1;
  f32x4_t sum[NSUM][C::MC][C::NC];
#pragma unroll
  for (int m = 0; m < C::MC; ++m)
#pragma unroll
    for (int n = 0; n < C::NC; ++n) {
      acc[m][n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int q = 0; q < NSUM; ++q) sum[q][m][n] = acc[m][n];
    }

  // fragment of a 16-row tile: row lane%16, chunk ks*4 + lane/16 (a 32-deep k step)
  const int fr = (lane & 15) * 128;
  const int sw = (lane >> 1) & 7;
  const int c0 = C::KSPLIT ? 0 : wave * (EP / NW);

#pragma unroll
  for (int st = 0; st < C::NS - 1; ++st)
    if (st < NST) issue(st);
  for (int st = 0; st < NST; ++st) {
    if (st + C::NS - 2 < NST) wait_vmcnt<(C::NS - 2) * C::NI>();
    else wait_vmcnt<0>();
    lds_barrier();  // stage st landed for every wave; stage st-1 is no longer read
    if (st + C::NS - 1 < NST) issue(st + C::NS - 1);
    const uint8_t* base = smem + (st % C::NS) * C::SB;
#pragma unroll
    for (int p = 0; p < C::PPS; ++p) {
      if (C::KSPLIT && p % NW != wave) continue;
      if (kp0 + st * C::PPS + p >= kp1) continue;
      const uint8_t* pan = base + p * C::PB;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const int slot = ((ks * 4 + (lane >> 4)) ^ sw) * 16;
        u32x4_t a[C::MC], b[C::NC];
#pragma unroll
        for (int m = 0; m < C::MC; ++m)
          a[m] = *reinterpret_cast<const u32x4_t*>(pan + m * 16 * 128 + fr + slot);
#pragma unroll
        for (int n = 0; n < C::NC; ++n)
          b[n] = *reinterpret_cast<const u32x4_t*>(pan + (BT + c0 + n * 16) * 128 + fr + slot);
#pragma unroll
        for (int m = 0; m < C::MC; ++m)
#pragma unroll
          for (int n = 0; n < C::NC; ++n) {
            const int q = (p % PS * 2 + ks) * JS;
            if constexpr (!SUMS) {
              acc[m][n] = mma16<T_>(a[m], b[n], acc[m][n]);
            } else if constexpr (JS == 1) {
              sum[q][m][n] = mma16<T_>(a[m], b[n], sum[q][m][n]);
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                sum[q + j % JS][m][n] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                    __uint_as_float(a[m][j]), __uint_as_float(b[n][j]), sum[q + j % JS][m][n], 0, 0, 0);
            }
          }
      }
    }
    if constexpr (SUMS) {
      // held in accumulation registers from stage to stage
#pragma unroll
      for (int q = 0; q < NSUM; ++q)
#pragma unroll
        for (int m = 0; m < C::MC; ++m)
#pragma unroll
          for (int n = 0; n < C::NC; ++n) asm volatile("" : "+a"(sum[q][m][n]));
    }
  }
  if constexpr (SUMS) {
#pragma unroll
    for (int h = NSUM / 2; h > 0; h /= 2)
#pragma unroll
      for (int q = 0; q < h; ++q)
#pragma unroll
        for (int m = 0; m < C::MC; ++m)
#pragma unroll
          for (int n = 0; n < C::NC; ++n) sum[q][m][n] += sum[q + h][m][n];
#pragma unroll
    for (int m = 0; m < C::MC; ++m)
#pragma unroll
      for (int n = 0; n < C::NC; ++n) acc[m][n] = sum[0][m][n];
  }
  __syncthreads();  // every wave is done with the stages
}

// Scores of the tile plus the bias into LDS (row-major, tile_stride<BT>()),
// columns < ncol. D layout of 16x16: lane holds column lane%16, rows
// (lane/16)*4 + v.
template <int BT, int EP, int NW = 4>
__device__ __forceinline__ void scores_to_lds(uint8_t* smem, int ncol, const float* __restrict__ bias,
                                              const f32x4_t (&acc)[RouteTile<BT, EP, NW>::MC][RouteTile<BT, EP, NW>::NC]) {
  using C = RouteTile<BT, EP, NW>;
  constexpr int S = tile_stride<BT, NW>();
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float* sc = reinterpret_cast<float*>(smem);
  if (!C::KSPLIT) {
    const int c0 = wave * (EP / NW);
#pragma unroll
    for (int m = 0; m < C::MC; ++m)
#pragma unroll
      for (int n = 0; n < C::NC; ++n) {
        const int col = c0 + n * 16 + (lane & 15);
        const float b = (bias != nullptr && col < ncol) ? bias[col] : 0.0f;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int row = m * 16 + (lane >> 4) * 4 + v;
          if (col < ncol) sc[row * S + col] = bias != nullptr ? acc[m][n][v] + b : acc[m][n][v];
        }
      }
  } else {
    float* part = reinterpret_cast<float*>(smem + C::SC_BYTES);
#pragma unroll
    for (int m = 0; m < C::MC; ++m)
#pragma unroll
      for (int n = 0; n < C::NC; ++n)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int row = m * 16 + (lane >> 4) * 4 + v;
          part[(wave * BT + row) * EP + n * 16 + (lane & 15)] = acc[m][n][v];
        }
    __syncthreads();
    for (int q = threadIdx.x; q < BT * ncol; q += NW * 64) {
      const int row = q / ncol, col = q % ncol;
      float v = part[(0 * BT + row) * EP + col];
#pragma unroll
      for (int w = 1; w < NW; ++w) v += part[(w * BT + row) * EP + col];  // waves in order
      sc[row * S + col] = bias != nullptr ? v + bias[col] : v;
    }
  }
  __syncthreads();
}

// Partial score tiles of the two-launch paths: workgroup (token block, expert
// block, K slice) stores its BT x EP tile to ws[ks][t][e] (no bias).
constexpr int kPartBT = 16, kPartEP = 64, kMaxSlices = 16;

template <int BT, int EP, int NW = 4, typename T_ = uint16_t, bool SUMS = false>
__global__ __launch_bounds__(NW * 64, SUMS ? 2 : 1)  // two workgroups a CU: at most 256 registers
void route_partial_kernel(const T_* __restrict__ x, const T_* __restrict__ wg, int T, int H, int E,
                          int kps, float* __restrict__ ws) {
  using C = RouteTile<BT, EP, NW>;
  static_assert(!C::KSPLIT, "each wave owns EP / NW experts");
  __shared__ __align__(16) uint8_t smem[C::NS * C::SB];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t0 = blockIdx.x * BT, e0 = blockIdx.y * EP, ks = blockIdx.z;
  f32x4_t acc[C::MC][C::NC];
  score_tile<BT, EP, NW, T_, SUMS>(smem, x, wg, t0, T, e0, E, H, ks * kps, (ks + 1) * kps, acc);
  // D layout of 16x16: lane holds column lane%16, rows (lane/16)*4 + v
#pragma unroll
  for (int m = 0; m < C::MC; ++m)
#pragma unroll
    for (int n = 0; n < C::NC; ++n) {
      const int e = e0 + wave * (EP / NW) + n * 16 + (lane & 15);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int t = t0 + m * 16 + (lane >> 4) * 4 + v;
        if (t < T && e < E) ws[((size_t)ks * T + t) * E + e] = acc[m][n][v];
      }
    }
}

// Waves of a workgroup of the bf16 score kernels: 8 for tiles of 128 or more
// experts whose panels split into whole copy instructions over 8 waves, else
// 4. With 8, a CU keeps twice the waves issuing the L2 -> LDS copies of Wg
// (the same bytes in flight stream faster: a microbenchmark read 75 against
// 49 GB/s per CU with 32 KiB in flight) and the top-k has twice the lanes per
// token.
template <int BT, int EP>
constexpr int route_waves() {
  using C = RouteTile<BT, EP>;  // its panel rows and panels per stage do not depend on the waves
  // panel-split tiles (E <= 32) stay at 4: with 8 (one panel of each stage per
  // wave) the Mixtral-shaped route took 12.4 against 12.0 us
  if (C::KSPLIT) return 4;
  return EP >= 128 && (C::PPS * C::R) % 64 == 0 ? 8 : 4;
}

enum RouteMode { kOneLaunch, kTwoSmall, kTwoBig };
RouteMode route_mode(int T, int E, bool bf16) {
  if (!bf16) return kOneLaunch;
  if (T < 2048) return kTwoSmall;
  return E > 64 && T < 16384 ? kTwoBig : kOneLaunch;
}
bool route_two_phase(int T, int E, bool bf16) { return route_mode(T, E, bf16) != kOneLaunch; }

// Tile of the big-tile path.
int big_bt(int E) { return E > 128 ? 128 : 64; }
int big_ep(int E) { return E > 128 ? 256 : 128; }

// K slices of a two-launch path: about 256 workgroups in phase 1, a power of
// two (at most kMaxSlices) that divides the H/64 panels.
int route_kslices(int T, int H, int E) {
  const bool big = route_mode(T, E, true) == kTwoBig;
  const int bt = big ? big_bt(E) : kPartBT, ep = big ? big_ep(E) : kPartEP;
  const int tiles = ((T + bt - 1) / bt) * ((E + ep - 1) / ep);
  int ks = 1;
  while (ks * 2 * tiles <= 256 && (H / 64) % (ks * 2) == 0 && ks * 2 <= kMaxSlices) ks *= 2;
  return ks;
}

// Tokens per workgroup of the one-launch bf16 path: as many as keep >= 256
// workgroups (one per CU).
int bf16_tokens_per_block(int T) { return T >= 64 * 256 ? 64 : T >= 32 * 256 ? 32 : 16; }

// Tokens per workgroup of the two-launch select: 16 from T = 1024 up (at
// least 64 workgroups), else 4. Measured on the whole route of the
// fine-grained layer (T = 4096, H = 4096, E = 128, k = 8): 34.5 -> 33.2 us.
// Up to 4 tokens there is one workgroup either way, and 16 lanes per token
// merge over fewer levels than 64.
int select_tokens_per_block(int T) { return T >= 1024 || T <= 4 ? 16 : 4; }

// Score launch of the two-launch paths (route_mode != kOneLaunch).
template <bool SUMS = false>
hipError_t launch_partial(const void* x, const void* wg, int T, int H, int E, float* sp,
                          hipStream_t s) {
  const int nks = route_kslices(T, H, E);
  const int kps = (H / 64) / nks;
  const uint16_t* xp = static_cast<const uint16_t*>(x);
  const uint16_t* wp = static_cast<const uint16_t*>(wg);
  if (route_mode(T, E, true) == kTwoSmall) {
    const dim3 grid((T + kPartBT - 1) / kPartBT, (E + kPartEP - 1) / kPartEP, nks);
    hipLaunchKernelGGL((route_partial_kernel<kPartBT, kPartEP, 4, uint16_t, SUMS>), grid, dim3(kThreads), 0, s, xp,
                       wp, T, H, E, kps, sp);
  } else if (E > 128) {
    const dim3 grid((T + 127) / 128, (E + 255) / 256, nks);
    hipLaunchKernelGGL((route_partial_kernel<128, 256, route_waves<128, 256>(), uint16_t, SUMS>), grid,
                       dim3(route_waves<128, 256>() * 64), 0, s, xp, wp, T,
                       H, E, kps, sp);
  } else {
    const dim3 grid((T + 63) / 64, (E + 127) / 128, nks);
    hipLaunchKernelGGL((route_partial_kernel<64, 128, route_waves<64, 128>(), uint16_t, SUMS>), grid,
                       dim3(route_waves<64, 128>() * 64), 0, s, xp, wp, T, H,
                       E, kps, sp);
  }
  return hipGetLastError();
}

size_t align256(size_t b) { return (b + 255) & ~size_t(255); }

size_t scores_ws_bytes(int T, int H, int E, bool bf16) {
  if (!route_two_phase(T, E, bf16)) return 0;
  return align256((size_t)route_kslices(T, H, E) * T * E * sizeof(float));
}

}  // namespace
}  // namespace moe
