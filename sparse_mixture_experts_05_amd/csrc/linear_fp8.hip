// Products of 8-bit floating-point operands (e4m3) with block scales, and the epilogue of
// moe_linear (linear.hip), dense and over the experts' ragged segments.
//
//   a[m,n] = sum_b sx[b,m] sw[n / 128, b] sum_{k in block b} x[m,k] w[n,k]  + bias[n]
//   y[m,n] = act(a) + residual, or act(a_0) * a_1 + residual (gated acts), in bf16
//
// with blocks b of 128 along K. v_mfma_f32_16x16x128_f8f6f4 takes a whole block in one
// instruction; its fp32 sums are then scaled into the accumulators by FMAs (the scales have
// any mantissa, so the matrix core cannot chain blocks). Both operands are read in the same
// order of k, the only thing that the instruction's layout along K asks for.
//
// The instruction adds 8 neighbours of K at a time, cut toward zero at 2^-13 of the power
// of two of their largest product (measured; the 16x16x32 form does the same), and those
// sums in fp32. On Gaussian operands that is 1.5e-5 of the result, without a bias, a
// hundredth of the output's bf16 rounding; products on bf16 MFMAs would not cut, at half
// the rate.
#include <algorithm>
#include <cmath>

#include "common.hpp"
#include "kernels.hpp"
#include "linear_fp8.hpp"

namespace moe {
namespace {

using namespace lin;

// ----------------------------------------------------------------- tiles

// Tiles of BM rows x BN weight rows (BN output columns, or BN / 2 of a gated product) by
// WM x WN waves. A stage is a block of 128 k: operand rows of 128 bytes, copied global ->
// LDS (8 rows an instruction) into a ring of NS stages, chunk c of row r at slot
// c ^ ((r >> 1) & 7) as in the bf16 tiles. Each wave also copies the scales of its own
// rows. The weights are the MFMA's A and the rows its B: lane l ends with 4 consecutive
// weight rows of row l % 16 of x. In a gated product the first half of a wave's weight
// sub-tiles holds gate rows, the second the up rows of the same columns.
//
// blockIdx.y of gridDim.y: a K slice. With several, a slice writes its accumulators to
// a.part and fp8_reduce_kernel finishes the tile.
template <int BM_, int BN_, int WM_, int WN_, int NS_>
struct Shape8 {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NS = NS_;
  static constexpr int NW = WM * WN, NT = NW * 64;
  static constexpr int TM = BM / WM / 16, TN = BN / WN / 16;  // sub-tiles of a wave
  static constexpr int NI = (BM + BN) / 8 / NW;               // row copies per wave per stage
  static constexpr int SI = (TM * 16 + 63) / 64;              // scale copies
  static constexpr int ROWS = (BM + BN) * 128;
  static constexpr int STAGE = ROWS + NW * SI * 256;
  static constexpr int GN = BN >= 128 ? 1024 / BN : 1;        // column tiles of an n-block
  static_assert(NS * STAGE <= 160 * 1024, "LDS of one workgroup");
};

template <typename Sh>
__device__ __forceinline__ int col8(int wn, int j, bool gt) {  // first column of a sub-tile
  constexpr int W = Sh::BN / Sh::WN;
  return gt ? wn * (W / 2) + j * 16 : wn * W + j * 16;
}

template <typename Sh>
__device__ __forceinline__ LinTile find8(const LinArgs& a) {
  return lin_tile<Sh::BM, Sh::GN>(a, gated(a.act) ? Sh::BN / 2 : Sh::BN);
}

template <typename Sh>
__device__ __forceinline__ float* part8(const LinArgs& a, const LinTile& t, int ks, int nks, int i, int j) {
  return a.part + ((size_t)t.q * nks + ks) * Sh::BM * Sh::BN +
         ((size_t)(i * Sh::TN + j) * Sh::NT + threadIdx.x) * 4;
}

// global_load_lds_dword: lane i copies 4 bytes from its address g to LDS at M0 + 4 * i.
__device__ __forceinline__ void lds_dma4(const void* g, void* lds_uniform) {
  const uint32_t m0 = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)(lds_uniform))));
  asm volatile(
      "s_mov_b32 m0, %1\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dword %0, off"
      :
      : "v"(g), "s"(m0)
      : "memory");
}

template <typename Sh, bool GT>
__global__ __launch_bounds__(Sh::NT) void fp8_tile_kernel(Fp8Args f) {
  constexpr int BM = Sh::BM, BN = Sh::BN, NS = Sh::NS, NI = Sh::NI, SI = Sh::SI;
  constexpr int TM = Sh::TM, TN = Sh::TN, H = GT ? 2 : 1;
  __shared__ __attribute__((aligned(16))) uint8_t smem[NS * Sh::STAGE];
  const LinArgs& a = f.a;
  const LinTile t = find8<Sh>(a);
  if (t.M == 0) return;
  const int N = a.N, K = a.K;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / Sh::WN, wn = wave % Sh::WN;
  const int KT0 = K / kBlock8;
  const int kbase = (int)((long long)blockIdx.y * KT0 / gridDim.y);
  const int KT = (int)((long long)(blockIdx.y + 1) * KT0 / gridDim.y) - kbase;

  const uint8_t* x = static_cast<const uint8_t*>(a.x);
  const uint8_t* w = static_cast<const uint8_t*>(a.w) + (size_t)t.e * H * N * K;
  const uint8_t* src[NI];
#pragma unroll
  for (int q = 0; q < NI; ++q) {
    const int r = 8 * (wave * NI + q) + (lane >> 3);
    const int chunk = (lane & 7) ^ ((r >> 1) & 7);
    const uint8_t* row;
    if (r < BM) {
      row = x + x_row(a, t.row0 + min(r, t.M - 1)) * K;  // rows past the end: its last
    } else {
      const int b = r - BM, j = b / 16 % TN;
      const int half = GT && j >= TN / 2 ? 1 : 0;
      const int c = t.n0 + col8<Sh>(b / (BN / Sh::WN), j - half * (TN / 2), GT) + b % 16;
      row = w + ((size_t)half * N + min(c, N - 1)) * K;  // columns past the end: its last
    }
    src[q] = row + (size_t)kbase * kBlock8 + chunk * 16;
  }
  const float* ssrc[SI];
#pragma unroll
  for (int q = 0; q < SI; ++q) {
    const int r = wm * (BM / Sh::WM) + min(q * 64 + lane, TM * 16 - 1);
    ssrc[q] = f.xs + x_row(a, t.row0 + min(r, t.M - 1)) + (size_t)kbase * f.xrows;
  }
  auto issue = [&](int kt) {
    uint8_t* base = smem + (kt % NS) * Sh::STAGE;
#pragma unroll
    for (int q = 0; q < NI; ++q) lds_dma16(src[q] + (size_t)kt * kBlock8, base + (wave * NI + q) * 1024);
#pragma unroll
    for (int q = 0; q < SI; ++q)
      lds_dma4(ssrc[q] + (size_t)kt * f.xrows, base + Sh::ROWS + (wave * SI + q) * 256);
  };
  // the weights' scales of this wave's columns, which lie in one block: lane l holds
  // those of the stages l, l + 64, ...
  const float* wsp[H];
  float wsv[H];
#pragma unroll
  for (int h = 0; h < H; ++h) wsp[h] = w_scales(f, t.e, h, GT, t.n0 + col8<Sh>(wn, 0, GT)) + kbase;

  f32x4_t acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const int fx = (wm * (BM / Sh::WM) + (lane & 15)) * 128;
  const int fw = (BM + wn * (BN / Sh::WN) + (lane & 15)) * 128;
  const int sw = (lane >> 1) & 7;  // (row >> 1) & 7 of every fragment row of this lane
  const int slot0 = ((lane >> 4) ^ sw) * 16, slot1 = ((4 + (lane >> 4)) ^ sw) * 16;
  const int sfx = Sh::ROWS + wave * SI * 256 + (lane & 15) * 4;

#pragma unroll
  for (int st = 0; st < NS - 1; ++st)
    if (st < KT) issue(st);
  for (int kt = 0; kt < KT; ++kt) {
    if ((kt & 63) == 0) {
#pragma unroll
      for (int h = 0; h < H; ++h) wsv[h] = wsp[h][min(kt + lane, KT - 1)];
    }
    // stage kt landed: at most the copies of the stages after it are in flight
    if (kt + NS - 2 < KT) wait_vmcnt<(NS - 2) * (NI + SI)>();
    else wait_vmcnt<0>();
    lds_barrier();  // for every wave; stage kt-1 is no longer read
    if (kt + NS - 1 < KT) issue(kt + NS - 1);
    const uint8_t* cur = smem + (kt % NS) * Sh::STAGE;
    float sws[H];
#pragma unroll
    for (int h = 0; h < H; ++h)
      sws[h] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wsv[h]), kt & 63));
    u32x4_t wf[TN][2];
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      wf[j][0] = ld16(cur + fw + j * 16 * 128 + slot0);
      wf[j][1] = ld16(cur + fw + j * 16 * 128 + slot1);
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const u32x4_t x0 = ld16(cur + fx + i * 16 * 128 + slot0);
      const u32x4_t x1 = ld16(cur + fx + i * 16 * 128 + slot1);
      const float sx = *reinterpret_cast<const float*>(cur + sfx + i * 64);
      float s[H];
#pragma unroll
      for (int h = 0; h < H; ++h) s[h] = sx * sws[h];
#pragma unroll
      for (int j = 0; j < TN; ++j)
        fma4(acc[i][j], s[GT && j >= TN / 2 ? H - 1 : 0], mma_block(wf[j][0], wf[j][1], x0, x1));
    }
  }
  if (gridDim.y == 1) {
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int r = wm * (BM / Sh::WM) + i * 16 + (lane & 15);
      if (r >= t.M) continue;
#pragma unroll
      for (int j = 0; j < (GT ? TN / 2 : TN); ++j) {
        const int c = t.n0 + col8<Sh>(wn, j, GT) + (lane >> 4) * 4;
        if (c < N) store4<uint16_t>(a, t.e, (size_t)(t.row0 + r), c, acc[i][j], acc[i][GT ? j + TN / 2 : j]);
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < TM; ++i)
    if (wm * (BM / Sh::WM) + i * 16 < t.M)
#pragma unroll
      for (int j = 0; j < TN; ++j)
        *reinterpret_cast<f32x4_t*>(part8<Sh>(a, t, blockIdx.y, gridDim.y, i, j)) = acc[i][j];
}

// Sums the nks K slices of each tile in slice order, then the epilogue. One workgroup per
// row sub-tile i of a tile (blockIdx.y), so that a launch with few tiles still has many.
constexpr int kMaxSlices = 16;

template <typename Sh, bool GT>
__global__ __launch_bounds__(Sh::NT) void fp8_reduce_kernel(Fp8Args f, int nks) {
  constexpr int TN = Sh::TN;
  const LinArgs& a = f.a;
  const LinTile t = find8<Sh>(a);
  if (t.M == 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / Sh::WN, wn = wave % Sh::WN;
  const int i = blockIdx.y;
  const int r = wm * (Sh::BM / Sh::WM) + i * 16 + (lane & 15);
  if (wm * (Sh::BM / Sh::WM) + i * 16 >= t.M) return;
  f32x4_t acc[TN];
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    f32x4_t v[kMaxSlices];
#pragma unroll
    for (int s = 0; s < kMaxSlices; ++s)  // all loads first, from clamped slices
      v[s] = *reinterpret_cast<const f32x4_t*>(part8<Sh>(a, t, min(s, nks - 1), nks, i, j));
    acc[j] = v[0];
#pragma unroll
    for (int s = 1; s < kMaxSlices; ++s)
      if (s < nks) acc[j] += v[s];
  }
  if (r >= t.M) return;
#pragma unroll
  for (int j = 0; j < (GT ? TN / 2 : TN); ++j) {
    const int c = t.n0 + col8<Sh>(wn, j, GT) + (lane >> 4) * 4;
    if (c < a.N) store4<uint16_t>(a, t.e, (size_t)(t.row0 + r), c, acc[j], acc[GT ? j + TN / 2 : j]);
  }
}

// ----------------------------------------------------------------- few rows

// Decode: up to 16 rows of one segment and 16 output columns a workgroup, the weights
// straight from memory to registers; as lin_rows_kernel (linear.hip), with a block of K a
// step: lane l loads 32 bytes of weight row l % 16 and of x row l % 16. The 4 waves share
// the blocks of K in turn; their sums are added in wave order through LDS.
template <bool GT>
__global__ __launch_bounds__(256) void fp8_rows_kernel(Fp8Args f) {
  constexpr int KQ = 4, U = 2, H = GT ? 2 : 1;
  __shared__ f32x4_t red[KQ][H][64];
  const LinArgs& a = f.a;
  const LinTile t = lin_tile<16>(a, 16);
  if (t.M == 0) return;
  const int N = a.N, K = a.K;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int S = K / kBlock8;
  const int s0 = wave * S / KQ, s1 = (wave + 1) * S / KQ;
  const uint8_t* wp[H];
  const float* wsp[H];
#pragma unroll
  for (int h = 0; h < H; ++h) {
    wp[h] = static_cast<const uint8_t*>(a.w) +
            ((size_t)(t.e * H + h) * N + t.n0 + (lane & 15)) * K + (lane >> 4) * 16;
    wsp[h] = w_scales(f, t.e, h, GT, t.n0);
  }
  const size_t xr = x_row(a, t.row0 + min(lane & 15, t.M - 1));
  const uint8_t* xp = static_cast<const uint8_t*>(a.x) + xr * K + (lane >> 4) * 16;
  const float* xsp = f.xs + xr;
  f32x4_t acc[H];
#pragma unroll
  for (int h = 0; h < H; ++h) acc[h] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  struct Step {
    u32x4_t w[H][2], x[2];
    float ws[H], xs;
  };
  Step p[U], q[U];
  auto load = [&](Step (&d)[U], int s) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int h = 0; h < H; ++h) {
        d[u].w[h][0] = ld16(wp[h] + (size_t)(s + u) * kBlock8);
        d[u].w[h][1] = ld16(wp[h] + (size_t)(s + u) * kBlock8 + 64);
        d[u].ws[h] = wsp[h][s + u];
      }
      d[u].x[0] = ld16(xp + (size_t)(s + u) * kBlock8);
      d[u].x[1] = ld16(xp + (size_t)(s + u) * kBlock8 + 64);
      d[u].xs = xsp[(size_t)(s + u) * f.xrows];
    }
  };
  auto one = [&](const Step& d) {
#pragma unroll
    for (int h = 0; h < H; ++h)
      fma4(acc[h], d.ws[h] * d.xs, mma_block(d.w[h][0], d.w[h][1], d.x[0], d.x[1]));
  };
  auto mma = [&](const Step (&d)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) one(d[u]);
  };
  int s = s0;
  if (s + U <= s1) {
    load(p, s);
    for (;;) {
      s += U;
      const bool more = s + U <= s1;
      if (more) load(q, s);
      mma(p);
      if (!more) break;
      s += U;
      const bool again = s + U <= s1;
      if (again) load(p, s);
      mma(q);
      if (!again) break;
    }
  }
  if (s < s1) {  // one block is left (U = 2)
    static_assert(U == 2, "the rest is one block");
    Step d;
#pragma unroll
    for (int h = 0; h < H; ++h) {
      d.w[h][0] = ld16(wp[h] + (size_t)s * kBlock8);
      d.w[h][1] = ld16(wp[h] + (size_t)s * kBlock8 + 64);
      d.ws[h] = wsp[h][s];
    }
    d.x[0] = ld16(xp + (size_t)s * kBlock8);
    d.x[1] = ld16(xp + (size_t)s * kBlock8 + 64);
    d.xs = xsp[(size_t)s * f.xrows];
    one(d);
  }
  if (wave != 0) {
#pragma unroll
    for (int h = 0; h < H; ++h) red[wave][h][lane] = acc[h];
  }
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int q2 = 1; q2 < KQ; ++q2)
#pragma unroll
    for (int h = 0; h < H; ++h) acc[h] += red[q2][h][lane];
  const int r = lane & 15;
  if (r < t.M) store4<uint16_t>(a, t.e, (size_t)(t.row0 + r), t.n0 + (lane >> 4) * 4, acc[0], acc[H - 1]);
}

// ----------------------------------------------------------------- host side

bool host_gated(int act) { return act == kActGeglu || act == kActSwiglu; }

using Small = Shape8<64, 64, 2, 2, 3>;
using Mid = Shape8<128, 128, 2, 2, 2>;

// Tiles of a launch, at most: sum_e ceil(c_e / BM) <= M / BM + #{e : c_e > 0} row tiles,
// each with all column tiles.
long long tiles8(const LinArgs& a, int BM, int bnc) {
  const long long mt = a.offsets ? (long long)a.M / BM + std::min(a.E, a.M)
                                 : ((long long)a.M + BM - 1) / BM;
  return mt * ((a.N + bnc - 1) / bnc);
}
template <typename Sh>
long long tiles8(const LinArgs& a) {
  return tiles8(a, Sh::BM, host_gated(a.act) ? Sh::BN / 2 : Sh::BN);
}
unsigned rounds8(long long tiles) { return (unsigned)((tiles + 7) / 8 * 8); }  // of the 8 XCDs

long long big_tiles8(const LinArgs& a) { return tiles8(a, 256, host_gated(a.act) ? 128 : 256); }

enum Fp8Path { kRows8, kSmall8, kMid8, kLarge8 };  // moe_fp8_path
struct Fp8Plan {
  Fp8Path path;
  int nks;
};

Fp8Plan plan8(const LinArgs& a) {
  const double live = a.offsets ? a.E * (1.0 - std::exp(-(double)a.M / a.E)) : 1.0;
  const double per = a.M / live;
  if (per <= 16) return {kRows8, 1};
  if (fp8_big_ok(a) && big_tiles8(a) >= 200) return {kLarge8, 1};
  if (tiles8<Mid>(a) >= 200) return {kMid8, 1};
  int nks = 1;
  while (nks < kMaxSlices && tiles8<Small>(a) * nks * 2 <= 512 && a.K / kBlock8 >= 8 * nks) nks *= 2;
  return {kSmall8, nks};
}

template <typename Sh>
size_t part_bytes8(const LinArgs& a, int nks) {
  return nks <= 1 ? 0 : (size_t)tiles8<Sh>(a) * nks * Sh::BM * Sh::BN * sizeof(float);
}

template <typename Sh, bool GT>
hipError_t run_tiles8(Fp8Args f, int nks, void* ws, hipStream_t s) {
  f.a.tiles = (int)tiles8<Sh>(f.a);
  f.a.part = static_cast<float*>(ws);
  const unsigned grid = rounds8(f.a.tiles);
  hipLaunchKernelGGL((fp8_tile_kernel<Sh, GT>), dim3(grid, nks), dim3(Sh::NT), 0, s, f);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || nks <= 1) return err;
  hipLaunchKernelGGL((fp8_reduce_kernel<Sh, GT>), dim3(grid, Sh::TM), dim3(Sh::NT), 0, s, f, nks);
  return hipGetLastError();
}

template <bool GT>
hipError_t run8(Fp8Args f, const Fp8Plan& p, void* ws, hipStream_t s) {
  switch (p.path) {
    case kRows8: {
      f.a.tiles = (int)tiles8(f.a, 16, 16);
      hipLaunchKernelGGL((fp8_rows_kernel<GT>), dim3(rounds8(f.a.tiles)), dim3(256), 0, s, f);
      return hipGetLastError();
    }
    case kSmall8: return run_tiles8<Small, GT>(f, p.nks, ws, s);
    case kMid8: return run_tiles8<Mid, GT>(f, p.nks, ws, s);
    default: f.a.tiles = (int)big_tiles8(f.a); return launch_fp8_big(f, rounds8(f.a.tiles), s);
  }
}

LinArgs args8(const void* x, const int32_t* gather, int gk, int gT, const int32_t* offsets, int E,
              int M, int N, int K, int act) {
  LinArgs a{};
  a.x = x, a.offsets = offsets, a.gather = gather, a.gk = gk, a.gT = gT;
  a.E = E, a.M = M, a.N = N, a.K = K, a.act = act;
  return a;
}
LinArgs shape_args8(int E, int M, int N, int K, int act, bool grouped) {
  static const int32_t some = 0;  // only tested for null
  return args8(nullptr, nullptr, 1, M, grouped ? &some : nullptr, E, M, N, K, act);
}

}  // namespace

bool linear_fp8_fits(int E, int M, int N, int K, int act, bool grouped) {
  const LinArgs a = shape_args8(E, M, N, K, act, grouped);
  // a grid dimension holds less than 2^32 threads, and tile numbers are ints
  switch (plan8(a).path) {
    case kRows8: return tiles8(a, 16, 16) + 8 < (1LL << 32) / 256;
    case kSmall8: return tiles8<Small>(a) + 8 < (1LL << 32) / Small::NT;
    case kMid8: return tiles8<Mid>(a) + 8 < (1LL << 32) / Mid::NT;
    default:  // or, for gathered rows past 4 GiB, the 128 x 128 tiles
      return big_tiles8(a) + 8 < (1LL << 32) / 512 && tiles8<Mid>(a) + 8 < (1LL << 32) / Mid::NT;
  }
}

size_t linear_fp8_ws_bytes(int E, int M, int N, int K, int act, bool grouped) {
  const LinArgs a = shape_args8(E, M, N, K, act, grouped);
  const Fp8Plan p = plan8(a);
  switch (p.path) {
    case kRows8: return 0;
    case kSmall8: return part_bytes8<Small>(a, p.nks);
    case kMid8: return part_bytes8<Mid>(a, p.nks);
    default: return 0;
  }
}

int linear_fp8_path(int E, int M, int N, int K, int act, bool grouped, int* slices) {
  const Fp8Plan p = plan8(shape_args8(E, M, N, K, act, grouped));
  *slices = p.nks;
  return p.path;
}

hipError_t launch_linear_fp8(const void* x, const float* x_scale, const int32_t* gather, int gk,
                             int gT, const int32_t* offsets, int E, int M, int N, int K,
                             const void* w, const float* w_scale, const void* bias, int act,
                             const void* res, void* y, void* ws, hipStream_t s) {
  Fp8Args f{};
  f.a = args8(x, gather, gk, gT, offsets, E, M, N, K, act);
  f.a.w = w, f.a.bias = bias, f.a.res = res, f.a.y = y;
  f.xs = x_scale, f.ws = w_scale, f.xrows = gather ? gT : M;
  Fp8Plan p = plan8(f.a);
  // gathered rows past the large tiles' 32-bit offsets: no workspace needed either
  if (p.path == kLarge8 && !fp8_big_ok(f.a)) p = Fp8Plan{kMid8, 1};
  return host_gated(act) ? run8<true>(f, p, ws, s) : run8<false>(f, p, ws, s);
}

}  // namespace moe
