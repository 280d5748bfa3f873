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
#include <cmath>

#include "common.hpp"
#include "kernels.hpp"
#include "linear.hpp"
#include "plan.hpp"

namespace moe {
namespace {

using namespace lin;

constexpr int kThreads = 256;

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

// The tile of this workgroup, BM rows x bnc output columns. Tiles are numbered
// segment by segment, column tile by column tile, row tile by row tile, and XCD
// x (workgroups x, x + 8, ...) takes a contiguous run of them: the tiles that
// share a weight panel run on one XCD at about one time. M = 0: no work.
template <int BM>
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
    t.row0 = t.q % nm * BM;
    t.n0 = t.q / nm * bnc;
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
  const int local = (int)(q - (long long)base * ntn);
  const int m = local % nb;
  t.e = e;
  t.q = (int)q;
  t.row0 = off + m * BM;
  const int left = cnt - m * BM;
  t.M = left < BM ? left : BM;
  t.n0 = local / nb * bnc;
  return t;
}

// ----------------------------------------------------------------- 64 x 64 tiles

// Tiles of BM rows x 64 weight rows (64 output columns, or 32 of a gated
// product) by 4 waves in a 2 x 2 grid, bf16 or fp32. Operand rows are copied
// global -> LDS with global_load_lds (8 rows of 128 bytes an instruction) into a
// ring of NS stages of 128 bytes of K; 16-byte chunk c of row r sits at slot
// c ^ ((r >> 1) & 7), so the 16 lanes of a fragment read (16 consecutive rows, one
// chunk) touch 16 distinct 4-bank groups. The weights are the MFMA's A and the rows
// its B: lane l ends with 4 consecutive weight rows of row l % 16 of x. In a gated
// product the first half of a wave's weight sub-tiles holds gate rows, the second the up rows
// of the same columns.
//
// blockIdx.y of gridDim.y: a K slice. With several, a slice writes its
// accumulators to a.part and lin_tile_reduce_kernel finishes the tile.
template <int BM_>
struct TileShape {
  static constexpr int BM = BM_, BN = 64, NS = 3;
  static constexpr int TM = BM / 2 / 16, TN = BN / 2 / 16;  // sub-tiles of a wave
  static constexpr int STAGE = (BM + BN) * 128;
  static constexpr int NI = (BM + BN) / 8 / 4;  // copies per wave per stage
};

__device__ __forceinline__ int tile_col(int wn, int j, bool gt) {  // first column of a sub-tile
  constexpr int W = 64 / 2;
  return gt ? wn * (W / 2) + j * 16 : wn * W + j * 16;
}

// Epilogue of a wave's accumulators, straight to memory.
template <typename T, typename Sh>
__device__ __forceinline__ void tile_store(const LinArgs& a, const LinTile& t,
                                           const f32x4_t (&acc)[Sh::TM][Sh::TN]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave >> 1, wn = wave & 1;
  const bool gt = gated(a.act);
#pragma unroll
  for (int i = 0; i < Sh::TM; ++i) {
    const int r = wm * (Sh::BM / 2) + i * 16 + (lane & 15);
    if (r >= t.M) continue;
#pragma unroll
    for (int j = 0; j < Sh::TN; ++j) {
      if (gt && j >= Sh::TN / 2) continue;
      const int c = t.n0 + tile_col(wn, j, gt) + (lane >> 4) * 4;
      if (c < a.N) store4<T>(a, t.e, (size_t)(t.row0 + r), c, acc[i][j], acc[i][(j + Sh::TN / 2) % Sh::TN]);
    }
  }
}

// Accumulator (i, j) of this thread in slice ks of a tile's partials.
template <typename Sh>
__device__ __forceinline__ float* tile_part(const LinArgs& a, const LinTile& t, int ks, int nks,
                                            int i, int j) {
  return a.part + ((size_t)t.q * nks + ks) * Sh::BM * Sh::BN +
         ((size_t)(i * Sh::TN + j) * kThreads + threadIdx.x) * 4;
}

template <typename Sh>
__device__ __forceinline__ LinTile find(const LinArgs& a) {
  return lin_tile<Sh::BM>(a, gated(a.act) ? Sh::BN / 2 : Sh::BN);
}

template <typename T, int BM_>
__global__ __launch_bounds__(kThreads) void lin_tile_kernel(LinArgs a) {
  using Sh = TileShape<BM_>;
  constexpr int BM = Sh::BM, BN = Sh::BN, NS = Sh::NS, STAGE = Sh::STAGE, NI = Sh::NI;
  constexpr int TM = Sh::TM, TN = Sh::TN;
  __shared__ __attribute__((aligned(16))) uint8_t smem[NS * STAGE];
  const LinTile t = find<Sh>(a);
  if (t.M == 0) return;
  const bool gt = gated(a.act);
  const int N = a.N, K = a.K;
  const T* x = static_cast<const T*>(a.x);
  const T* w = static_cast<const T*>(a.w) + (size_t)t.e * (gt ? 2 : 1) * N * K;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave >> 1, wn = wave & 1;
  constexpr int BK = 128 / sizeof(T), EC = 16 / sizeof(T);  // elements of a stage, of a chunk
  const int KT0 = K / BK;
  const int kbase = (int)((long long)blockIdx.y * KT0 / gridDim.y);
  const int KT = (int)((long long)(blockIdx.y + 1) * KT0 / gridDim.y) - kbase;

  const T* src[NI];
#pragma unroll
  for (int q = 0; q < NI; ++q) {
    const int r = 8 * (wave * NI + q) + (lane >> 3);
    const int chunk = (lane & 7) ^ ((r >> 1) & 7);
    const T* row;
    if (r < BM) {
      row = x + x_row(a, t.row0 + min(r, t.M - 1)) * K;  // rows past the end: its last
    } else {
      const int b = r - BM, j = b / 16 % TN;
      const int half = gt && j >= TN / 2 ? 1 : 0;
      const int c = t.n0 + tile_col(b / (BN / 2), j - half * (TN / 2), gt) + b % 16;
      row = w + ((size_t)half * N + min(c, N - 1)) * K;  // columns past the end: its last
    }
    src[q] = row + (size_t)kbase * BK + chunk * EC;
  }
  auto issue = [&](int kt) {
    uint8_t* base = smem + (kt % NS) * STAGE;
#pragma unroll
    for (int q = 0; q < NI; ++q) lds_dma16(src[q] + (size_t)kt * BK, base + (wave * NI + q) * 1024);
  };
  // fp32: 4 sums per output, for each half of a stage and every other MFMA, added up
  // behind the loop. One chain over K rounds partial sums as large as the result; 4 are
  // off by half as much (512 x 4096 x 4096 against float64, u = 2^-24: 19.2 -> 9.6 u, with
  // a gate 29.3 -> 14.1; 154.6 and 155.4 us)
  constexpr int NSUM = sizeof(T) == 4 ? 4 : 1;
  f32x4_t sum[NSUM][TM][TN];
#pragma unroll
  for (int s = 0; s < NSUM; ++s)
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) sum[s][i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const int fx = (wm * (BM / 2) + (lane & 15)) * 128;
  const int fw = (BM + wn * (BN / 2) + (lane & 15)) * 128;
  const int sw = (lane >> 1) & 7;  // (row >> 1) & 7 of every fragment row of this lane

#pragma unroll
  for (int st = 0; st < NS - 1; ++st)
    if (st < KT) issue(st);
  for (int kt = 0; kt < KT; ++kt) {
    // stage kt landed: at most the copies of the stages after it are in flight
    if (kt + NS - 2 < KT) wait_vmcnt<(NS - 2) * NI>();
    else wait_vmcnt<0>();
    lds_barrier();  // for every wave; stage kt-1 is no longer read
    if (kt + NS - 1 < KT) issue(kt + NS - 1);
    const uint8_t* cur = smem + (kt % NS) * STAGE;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const int slot = ((ks * 4 + (lane >> 4)) ^ sw) * 16;
      u32x4_t xf[TM], wf[TN];
#pragma unroll
      for (int j = 0; j < TN; ++j) wf[j] = ld16(cur + fw + j * 16 * 128 + slot);
#pragma unroll
      for (int i = 0; i < TM; ++i) xf[i] = ld16(cur + fx + i * 16 * 128 + slot);
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          if constexpr (NSUM == 1) {
            sum[0][i][j] = mma16<T>(wf[j], xf[i], sum[0][i][j]);
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              sum[ks * 2 + q % 2][i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                  __uint_as_float(wf[j][q]), __uint_as_float(xf[i][q]), sum[ks * 2 + q % 2][i][j], 0, 0, 0);
          }
        }
    }
    if constexpr (NSUM > 1) {  // held in accumulation registers from stage to stage
#pragma unroll
      for (int s = 0; s < NSUM; ++s)
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j) asm volatile("" : "+a"(sum[s][i][j]));
    }
  }
  f32x4_t acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      acc[i][j] = sum[0][i][j];
      if constexpr (NSUM > 1) acc[i][j] = (acc[i][j] + sum[1][i][j]) + (sum[2][i][j] + sum[3][i][j]);
    }
  if (gridDim.y == 1) {
    tile_store<T, Sh>(a, t, acc);
    return;
  }
#pragma unroll
  for (int i = 0; i < TM; ++i)
    if (wm * (BM / 2) + i * 16 < t.M)
#pragma unroll
      for (int j = 0; j < TN; ++j)
        *reinterpret_cast<f32x4_t*>(tile_part<Sh>(a, t, blockIdx.y, gridDim.y, i, j)) = acc[i][j];
}

// Sums the nks K slices of each tile in slice order, then the epilogue. One
// workgroup per row sub-tile i of a tile (blockIdx.y), so that a launch with few
// tiles still has many.
constexpr int kMaxSlices = 16;

template <typename T, int BM_>
__global__ __launch_bounds__(kThreads) void lin_tile_reduce_kernel(LinArgs a, int nks) {
  using Sh = TileShape<BM_>;
  const LinTile t = find<Sh>(a);
  if (t.M == 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const bool gt = gated(a.act);
  const int i = blockIdx.y;
  const int r = (wave >> 1) * (Sh::BM / 2) + i * 16 + (lane & 15);
  f32x4_t acc[Sh::TN];
  if ((wave >> 1) * (Sh::BM / 2) + i * 16 >= t.M) return;
#pragma unroll
  for (int j = 0; j < Sh::TN; ++j) {
    f32x4_t v[kMaxSlices];
#pragma unroll
    for (int s = 0; s < kMaxSlices; ++s)  // all loads first, from clamped slices
      v[s] = *reinterpret_cast<const f32x4_t*>(tile_part<Sh>(a, t, min(s, nks - 1), nks, i, j));
    acc[j] = v[0];
#pragma unroll
    for (int s = 1; s < kMaxSlices; ++s)
      if (s < nks) acc[j] += v[s];
  }
  if (r >= t.M) return;
#pragma unroll
  for (int j = 0; j < Sh::TN; ++j) {
    if (gt && j >= Sh::TN / 2) continue;
    const int c = t.n0 + tile_col(wave & 1, j, gt) + (lane >> 4) * 4;
    if (c < a.N) store4<T>(a, t.e, (size_t)(t.row0 + r), c, acc[j], acc[(j + Sh::TN / 2) % Sh::TN]);
  }
}

// ----------------------------------------------------------------- bf16, few rows

// Decode: a few rows per segment, so a launch is a stream of the weights. A
// workgroup takes up to 16 rows of one segment and 16 output columns; its 4
// waves share K in 32-deep steps (8 or 16 waves were no faster, 1 x 4096 x 4096
// to 16 x 512 x 4096: 7.3-11.4 us either way). Weights go from memory straight to registers
// (no other wave reads them): one 16-byte load per lane per 16 weight rows x 32 k,
// in chunks of U steps with the next chunk in flight while one is multiplied.
// v_mfma_f32_16x16x32_bf16 takes the weights as A and the rows as B, lane l
// loads weight row l % 16 and x row l % 16 at k = 8 (l / 16) of each step. Rows
// past the block's end read its last row and are not stored. The waves' sums are
// added in wave order through LDS.
template <bool GT>
__global__ __launch_bounds__(kThreads) void lin_rows_kernel(LinArgs a) {
  constexpr int KQ = 4, U = 4, H = GT ? 2 : 1;
  __shared__ f32x4_t red[KQ][H][64];
  const LinTile t = lin_tile<16>(a, 16);
  if (t.M == 0) return;
  const int N = a.N, K = a.K;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int S = K / 32;
  const int s0 = wave * S / KQ, s1 = (wave + 1) * S / KQ;
  const uint16_t* wp[H];
#pragma unroll
  for (int h = 0; h < H; ++h)
    wp[h] = static_cast<const uint16_t*>(a.w) +
            ((size_t)(t.e * H + h) * N + t.n0 + (lane & 15)) * K + (lane >> 4) * 8;
  const uint16_t* xp = static_cast<const uint16_t*>(a.x) +
                       x_row(a, t.row0 + min(lane & 15, t.M - 1)) * K + (lane >> 4) * 8;
  f32x4_t acc[H];
#pragma unroll
  for (int h = 0; h < H; ++h) acc[h] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  u32x4_t wa[U][H], xa[U], wb[U][H], xb[U];
  auto load = [&](u32x4_t (&w)[U][H], u32x4_t (&x)[U], int s) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int h = 0; h < H; ++h) w[u][h] = ld16(wp[h] + (size_t)(s + u) * 32);
      x[u] = ld16(xp + (size_t)(s + u) * 32);
    }
  };
  auto mma = [&](const u32x4_t (&w)[U][H], const u32x4_t (&x)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < H; ++h)
        acc[h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(w[u][h]), as_bf16x8(x[u]), acc[h], 0, 0, 0);
  };
  int s = s0;
  if (s + U <= s1) {
    load(wa, xa, s);
    for (;;) {
      s += U;
      const bool more = s + U <= s1;
      if (more) load(wb, xb, s);
      mma(wa, xa);
      if (!more) break;
      s += U;
      const bool again = s + U <= s1;
      if (again) load(wa, xa, s);
      mma(wb, xb);
      if (!again) break;
    }
  }
  for (; s < s1; ++s) {
    const u32x4_t x1 = ld16(xp + (size_t)s * 32);
#pragma unroll
    for (int h = 0; h < H; ++h)
      acc[h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(ld16(wp[h] + (size_t)s * 32)),
                                                       as_bf16x8(x1), acc[h], 0, 0, 0);
  }
  if (wave != 0) {
#pragma unroll
    for (int h = 0; h < H; ++h) red[wave][h][lane] = acc[h];
  }
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int q = 1; q < KQ; ++q)
#pragma unroll
    for (int h = 0; h < H; ++h) acc[h] += red[q][h][lane];
  const int r = lane & 15;
  if (r < t.M) store4<uint16_t>(a, t.e, (size_t)(t.row0 + r), t.n0 + (lane >> 4) * 4, acc[0], acc[H - 1]);
}

// ----------------------------------------------------------------- host side

// Tiles of a launch, at most: sum_e ceil(c_e / BM) <= M / BM + #{e : c_e > 0} row
// tiles, each with all column tiles.
long long lin_tiles(const LinArgs& a, int BM, int bnc) {
  const long long mt = a.offsets ? (long long)a.M / BM + std::min(a.E, a.M)
                                 : ((long long)a.M + BM - 1) / BM;
  return mt * ((a.N + bnc - 1) / bnc);
}
unsigned lin_grid(const LinArgs& a, int BM, int bnc) {  // whole rounds of the 8 XCDs
  return (unsigned)((lin_tiles(a, BM, bnc) + 7) / 8 * 8);
}

enum LinPath { kRows, kTile64, kBigHalf, kBig };  // moe_path
struct LinPlan {
  LinPath path;
  int nks;  // K slices (64 x 64 tiles)
};

bool host_gated(int act) { return act == kActGeglu || act == kActSwiglu; }

// fp32 products always take these tiles, bound by the fp32 MFMA rate (a sixteenth of
// bf16's): of 32 rows where 64 would leave CUs without one (64 x 512 x 256: 9.8 to 6.8
// us), and as many K slices as fill the chip with about two workgroups a CU and
// leave each 8 stages or more.
int f32_rows(const LinArgs& a) {
  return lin_tiles(a, 64, host_gated(a.act) ? 32 : 64) < 256 ? 32 : 64;
}
int f32_slices(const LinArgs& a) {
  const double tiles = (double)lin_tiles(a, f32_rows(a), host_gated(a.act) ? 32 : 64);
  int nks = 1;
  while (nks < kMaxSlices && tiles * nks * 2 <= 512 && a.K / 32 >= 16 * nks) nks *= 2;
  return nks;
}

// Path of a bf16 product: the least of the four paths' estimated times, in us. The
// estimates hold what was measured (graph replay, no act; M x N x K dense, then E
// experts with evenly drawn rows):
//                        rows    64x64 (slices)   256x128   256x256
//   1 x 4096 x 4096       8.7     11.7 (8)           41        44
//   64 x 4096 x 4096              14.0 (4)           43        51
//   256 x 4096 x 4096             23.7 (2)           44        73
//   512 x 4096 x 4096             33.9 (1)           45        73
//   1024 x 4096 x 4096            61.7 (1)           47        73
//   2048 x 4096 x 4096           140   (1)           58        75
//   3000 x 4096 x 4096           219   (1)           97        81
//   4096 x 4096 x 4096           305   (1)          114        96
//   64 x 1024 x 1024      5.0      8.1 (8)           15        19
//   2048 x 512 x 4096             26.4 (1)           44        73
//   1 x 64 x 8192        11.7      9.1 (16)          20        27
//   64 x 1024 x 8192               10.7 (16)          28        34
//   256 x 4096 x 8192             38.0 (4)           36        52
//   512 x 4096 x 8192             62.3 (1)           47        57
//   2048 x 4096 x 8192           297   (1)          106       117
//   128 x 512 x 14336             14.9 (16)          31        47
//   256 x 4096 x 28672           104   (2)           71        85
//   E 8, 64 rows, 1024 x 1024    7.1     10.0 (1)    15        18
//   E 8, 512 rows, 4096 x 4096           61.4 (1)    68        77
//   E 8, 1024 rows, 4096 x 4096          93   (1)    72        88
//   E 8, 8192 rows, 4096 x 4096         525   (1)   273       257
//   E 128, 1024 rows, 1024 x 4096       184   (1)   246       191
//   E 64, 16384 rows, 1024 x 1024        81   (1)    65        57
// A stage is 64 k. Few-row kernel: every block of 16 rows x 16 columns reads both
// operands from the caches (8.5 TB/s), and a wave walks a quarter of K (1 us per
// 1000). 64x64 tiles: 0.36 us a stage while fewer than 1.75 workgroups share a CU,
// then in proportion, and a third of the time in which every column tile reads its rows
// from L2 (8 TB/s) does not hide; slices add a launch (3 us) and their partials' round trip. The large tiles run one
// workgroup a CU: 0.56 or 1 us a stage on an idle chip, 0.83 or 1.38 when every CU
// runs one (power and cache traffic); the last round's K slices are plan.hpp's, and the
// launch that adds them up takes 3 us and their bytes at 3.3 TB/s. Of the lesser of work
// and weight stream a tenth does not hide behind the other.
LinPlan lin_plan(const LinArgs& a) {
  const double h = host_gated(a.act) ? 2.0 : 1.0, cols = h * a.N;  // weight rows of an expert
  // experts with rows, as if each row drew its expert
  const double live = a.offsets ? a.E * (1.0 - std::exp(-(double)a.M / a.E)) : 1.0;
  const double stages = a.K / 64;
  // row tiles of a segmented launch: each segment's last one is half full on average
  auto row_tiles = [&](int bm) {
    return a.offsets ? std::max(live, (double)a.M / bm + live / 2) : std::ceil((double)a.M / bm);
  };
  struct Large {
    double us;
    bool split;  // K slices in the last round, and a launch that adds them up
  };
  auto big = [&](int bn, double idle, double full) {
    const double tiles = row_tiles(256) * std::ceil(cols / bn);
    const double start = 8.0 + (a.offsets ? 2.0 : 0.0);
    if (a.K >= plan::kSplitMinK) {
      const long long each = (long long)std::ceil(tiles / plan::kXcds);  // tiles of an XCD
      const long long rounds = each / plan::kSlots;
      const int tail = (int)(each % plan::kSlots);
      const int spl = plan::tail_slices(tail, a.K / plan::kStageK);
      if (spl > 1) {
        const double last = tiles - 256.0 * rounds;
        return Large{start + stages * rounds * full +
                         std::ceil(stages / spl) * std::max(idle, full * tail * spl / plan::kSlots) +
                         3.0 + last * spl * 256 * bn * 4 / 3.3e6,
                     true};
      }
    }
    const double whole = std::floor(tiles / 256), rest = tiles - 256 * whole;
    return Large{start + stages * (whole * full + (rest <= 0 ? 0.0 : std::max(idle, full * rest / 256))),
                 false};
  };
  const double hbm = 2.0 * ((double)a.M * a.K + live * cols * a.K) / 5.3e6;
  // What a call costs its caller: the GPU's time, but in a run of calls no less than the
  // host's for its launches (9 us for one, 13 for two and a workspace); a tenth of the
  // GPU's own time decides between equals.
  auto cost = [](double us, bool two) { return std::max(us, two ? 13.0 : 9.0) + 0.1 * us; };
  LinPlan best{kRows, 1};
  double t = cost(3.2 + std::max({1.1 * hbm, a.K / 1000.0,
                             row_tiles(16) * (a.N / 16) * (16 * h + std::min(16.0, a.M / live)) * a.K * 2 / 8.5e6}), false);
  auto take = [&](LinPath path, int nks, double us, bool two) {
    const double c = cost(us, two);
    if (c < t) t = c, best = LinPlan{path, nks};
  };
  const double tiles = row_tiles(64) * std::ceil(cols / 64);
  const double rows_l2 = 0.3 * 2.0 * a.M * a.K * std::ceil(cols / 64) / 8e6;
  for (int nks = 1; nks <= 16; nks *= 2) {
    if (nks > 1 && (a.K / 64 < 2 * nks || tiles * nks > 2048)) break;
    double us = 4.4 + std::ceil(stages / nks) * 0.36 * std::max(1.0, tiles * nks / 448);
    if (nks > 1) us += 3.0 + 8.0 * a.M * cols * nks / 5e6;
    take(kTile64, nks, std::max(us, 3.0 + hbm) + 0.1 * std::min(us, hbm) + rows_l2, nks > 1);
  }
  if (big_ok(a)) {
    const Large half = big(128, 0.56, 0.83), whole = big(256, 1.0, 1.38);
    const bool table = a.offsets != nullptr;  // written by a launch of its own
    take(kBigHalf, 1, std::max(half.us, 8.0 + 1.1 * hbm) + 0.1 * std::min(half.us, hbm), table || half.split);
    take(kBig, 1, std::max(whole.us, 8.0 + hbm) + 0.1 * std::min(whole.us, hbm), table || whole.split);
  }
  return best;
}

size_t tile_ws_bytes(const LinArgs& a, int bm, int nks) {
  if (nks <= 1) return 0;
  return (size_t)lin_tiles(a, bm, host_gated(a.act) ? 32 : 64) * nks * bm * 64 * sizeof(float);
}

template <typename T, int BM>
hipError_t run_tile(LinArgs a, int nks, void* ws, hipStream_t s) {
  const int bnc = host_gated(a.act) ? 32 : 64;
  const unsigned grid = lin_grid(a, BM, bnc);
  a.tiles = (int)lin_tiles(a, BM, bnc);
  a.part = static_cast<float*>(ws);
  hipLaunchKernelGGL((lin_tile_kernel<T, BM>), dim3(grid, nks), dim3(kThreads), 0, s, a);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || nks <= 1) return err;
  hipLaunchKernelGGL((lin_tile_reduce_kernel<T, BM>), dim3(grid, TileShape<BM>::TM), dim3(kThreads), 0,
                     s, a, nks);
  return hipGetLastError();
}

LinArgs lin_args(const void* x, const int32_t* gather, int gk, int gT, const int32_t* offsets,
                 int E, int M, int N, int K, int act) {
  LinArgs a{};
  a.x = x, a.offsets = offsets, a.gather = gather, a.gk = gk, a.gT = gT;
  a.E = E, a.M = M, a.N = N, a.K = K, a.act = act;
  return a;
}

}  // namespace

bool linear_fits(int E, int M, int N, int K, int act, bool grouped, bool bf16) {
  const int32_t some = 0;  // only tested for null
  const LinArgs a = lin_args(nullptr, nullptr, 1, M, grouped ? &some : nullptr, E, M, N, K, act);
  // a grid dimension holds less than 2^32 threads; every path but the few-row one has at
  // most the workgroups of the 64 x 64 tiles
  // (fp32 tiles of 32 rows are a few hundred at most)
  const int bnc = host_gated(act) ? 32 : 64;
  const bool rows = bf16 && lin_plan(a).path == kRows;
  return lin_tiles(a, rows ? 16 : 64, rows ? 16 : bnc) + 8 < (1LL << 32) / kThreads;
}

size_t linear_ws_bytes(int E, int M, int N, int K, int act, bool grouped, bool bf16) {
  const int32_t some = 0;
  const LinArgs a = lin_args(nullptr, nullptr, 1, M, grouped ? &some : nullptr, E, M, N, K, act);
  if (!bf16) return tile_ws_bytes(a, f32_rows(a), f32_slices(a));
  const LinPlan p = lin_plan(a);
  if (p.path >= kBigHalf) return big_ws_bytes(a, p.path == kBigHalf);
  return p.path == kTile64 ? tile_ws_bytes(a, 64, p.nks) : 0;
}

int linear_path(int E, int M, int N, int K, int act, bool grouped, bool bf16, int* slices) {
  const int32_t some = 0;
  const LinArgs a = lin_args(nullptr, nullptr, 1, M, grouped ? &some : nullptr, E, M, N, K, act);
  const LinPlan p = bf16 ? lin_plan(a) : LinPlan{kTile64, f32_slices(a)};
  *slices = p.path >= kBigHalf ? big_slices(a, p.path == kBigHalf) : p.nks;
  return p.path;
}

hipError_t launch_linear(const void* x, const int32_t* gather, int gk, int gT,
                         const int32_t* offsets, int E, int M, int N, int K, const void* w,
                         const void* bias, int act, const void* res, bool bf16, void* y, void* ws,
                         hipStream_t s) {
  LinArgs a = lin_args(x, gather, gk, gT, offsets, E, M, N, K, act);
  a.w = w, a.bias = bias, a.res = res, a.y = y;
  const bool gt = host_gated(act);
  if (!bf16)
    return f32_rows(a) == 32 ? run_tile<float, 32>(a, f32_slices(a), ws, s)
                             : run_tile<float, 64>(a, f32_slices(a), ws, s);
  LinPlan p = lin_plan(a);
  // gathered rows past the large tiles' 32-bit offsets: no workspace needed either
  if (p.path >= kBigHalf && gather && !big_gather_ok(a)) p = LinPlan{kTile64, 1};
  switch (p.path) {
    case kRows: {
      const dim3 grid(lin_grid(a, 16, 16));
      a.tiles = (int)lin_tiles(a, 16, 16);
      if (gt) hipLaunchKernelGGL((lin_rows_kernel<true>), grid, dim3(kThreads), 0, s, a);
      else hipLaunchKernelGGL((lin_rows_kernel<false>), grid, dim3(kThreads), 0, s, a);
      return hipGetLastError();
    }
    case kTile64: return run_tile<uint16_t, 64>(a, p.nks, ws, s);
    default: return launch_big(a, p.path == kBigHalf, ws, s);
  }
}

}  // namespace moe
