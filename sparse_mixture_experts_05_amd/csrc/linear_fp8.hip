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
//
// Here: the few-row kernel and the choice of a path; the tiles are in linear_fp8_tiles.hip.
#include <algorithm>
#include <cmath>

#include "common.hpp"
#include "kernels.hpp"
#include "linear_fp8.hpp"

namespace moe {
namespace {

using namespace lin;

// ----------------------------------------------------------------- few rows

// Decode: up to 16 rows of one segment and 16 output columns a workgroup, the weights
// straight from memory to registers; as lin_rows_kernel (linear.hip), with a block of K a
// step: lane l loads 32 bytes of weight row l % 16 and of x row l % 16. The blocks of K go
// round the 4 waves (with a slice of K a wave, the workgroups read more often from the same
// HBM channels at one time: 81 of 128 experts 2048 x 4096 126 -> 121 us); their sums are
// added in wave order through LDS. Bound by HBM: 5.6 TB/s of weights there, and by a
// launch's start below some 50 MB (8 x 4096 x 4096: 7.3 us, of which its bytes take 3).
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
  const int mine = (S - wave + KQ - 1) / KQ;  // blocks wave, wave + KQ, ...
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
  auto one_load = [&](Step& d, int s) {
    const size_t b = (size_t)s * KQ + wave;
#pragma unroll
    for (int h = 0; h < H; ++h) {
      d.w[h][0] = ld16(wp[h] + b * kBlock8);
      d.w[h][1] = ld16(wp[h] + b * kBlock8 + 64);
      d.ws[h] = wsp[h][b];
    }
    d.x[0] = ld16(xp + b * kBlock8);
    d.x[1] = ld16(xp + b * kBlock8 + 64);
    d.xs = xsp[b * f.xrows];
  };
  auto load = [&](Step (&d)[U], int s) {
#pragma unroll
    for (int u = 0; u < U; ++u) one_load(d[u], s + u);
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
  int s = 0;
  if (s + U <= mine) {
    load(p, s);
    for (;;) {
      s += U;
      const bool more = s + U <= mine;
      if (more) load(q, s);
      mma(p);
      if (!more) break;
      s += U;
      const bool again = s + U <= mine;
      if (again) load(p, s);
      mma(q);
      if (!again) break;
    }
  }
  if (s < mine) {  // one block is left (U = 2)
    static_assert(U == 2, "the rest is one block");
    Step d;
    one_load(d, s);
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

// Tiles of a launch, at most: sum_e ceil(c_e / BM) <= M / BM + #{e : c_e > 0} row tiles,
// each with all column tiles.
long long tiles8(const LinArgs& a, int BM, int bnc) {
  const long long mt = a.offsets ? (long long)a.M / BM + std::min(a.E, a.M)
                                 : ((long long)a.M + BM - 1) / BM;
  return mt * ((a.N + bnc - 1) / bnc);
}
enum Fp8Path { kRows8, k64, k128, k256 };  // moe_fp8_path
constexpr int kSide[] = {16, 64, 128, 256};
long long tiles8(const LinArgs& a, Fp8Path p) {
  return tiles8(a, kSide[p], p == kRows8 ? 16 : host_gated(a.act) ? kSide[p] / 2 : kSide[p]);
}

struct Fp8Plan {
  Fp8Path path;
  int nks;  // K slices
};

// Path of a product: the least estimated time, in us. The estimates hold what was measured
// (graphs of three calls with their replay's start, no act; M x N x K dense, then 64 experts with evenly drawn rows):
//                        rows    64 (slices)   128 (slices)   256
//   16 x 4096 x 4096      8.5     12.1 (4)      12.9 (8)       25
//   32 x 4096 x 4096     12.0     12.2 (4)      13.3 (8)       25
//   64 x 4096 x 4096     19.1     13.4 (4)      15.2 (8)       27
//   128 x 4096 x 4096    33       15.9 (1)      16.7 (4)       31
//   256 x 4096 x 4096    62       16.0 (1)      20.8 (4)       49
//   512 x 4096 x 4096   119       19.9 (1)      22.9 (1)       49
//   1024 x 4096 x 4096  234       35.5 (1)      23.9 (1)       49
//   2048 x 4096 x 4096  464       61   (1)      38   (1)       50
//   4096 x 4096 x 4096           111   (1)      72   (1)       63
//   8192 x 4096 x 4096           217   (1)     141   (1)      123
//   64 x 4096 x 14336    55       20.3 (4)      22.4 (8)       78
//   1024 x 4096 x 14336          107   (1)      68   (1)      139
//   1024 x 14336 x 4096          101   (1)      69   (1)       60
//   E 64, 256 rows, 1024 x 2048   40   38 (1)   30   (1)       31
//   E 64, 4096 rows, 1024 x 2048 173   47 (1)   33   (1)       34
//   E 64, 8192 rows, 1024 x 2048 318   68 (1)   56   (1)       39
//   E 64, 32768 rows, 1024 x 2048     173 (1)  119   (1)      107
// A stage is 128 k. Few-row kernel: a stream of the weights, and of the rows from L2 once for
// every 16 columns (4.4 TB/s); 3.5 ns a workgroup where those are short, and 0.115 us a stage
// (gated 0.17) where there are few (32 x 192 x 8192 gated 15.2 us, 16 slices of 64-row tiles
// 9.8). 64-row tiles: 0.32 us a stage while a CU has one workgroup, then 0.19 and 0.9 us
// outside the stages a tile and CU (0.23 and 1.4 where segments' weights come from HBM);
// 128-row tiles: 0.48, then 0.45 and 3 (0.53 and 4). Slices add a launch (4 us, with segments 5.5) and their partials' round
// trip. Launches bound by their weights stream them at 0.97 to 1.35 of a copy's time. 256-row
// tiles: one workgroup a CU, 1.25 us a stage on an idle chip, 1.62 on a full one, and 4 us a
// round outside the stages. Over 80 shapes, drawn ones among them, the path taken is 1.2 %
// off the fastest in the mean.
Fp8Plan plan8(const LinArgs& a) {
  const double cols = (host_gated(a.act) ? 2.0 : 1.0) * a.N;  // weight rows of an expert
  // experts with rows, as if each row drew its expert
  const double live = a.offsets ? a.E * (1.0 - std::exp(-(double)a.M / a.E)) : 1.0;
  const double stages = a.K / kBlock8, start = a.offsets ? 7.0 : 5.0;
  // row tiles of a segmented launch: each segment's last one is half full on average
  auto row_tiles = [&](int bm) {
    return a.offsets ? std::max(live, (double)a.M / bm + live / 2) : std::ceil((double)a.M / bm);
  };
  const double hbm = ((double)a.M * a.K + live * cols * a.K) / 5.3e6;
  // What a call costs its caller: the GPU's time, but in a run of calls no less than the
  // host's for its launches; a tenth of the GPU's own time decides between equals.
  auto cost = [](double us, bool two) { return std::max(us, two ? 13.0 : 9.0) + 0.1 * us; };
  const double wgs = row_tiles(16) * (a.N / 16), rows = wgs * std::min(16.0, a.M / live) * a.K;
  Fp8Plan best{kRows8, 1};
  if (!fp8_tiles_ok(a)) return best;
  double t = cost(std::max(3.2 + std::max(0.97 * hbm, 0.0035 * wgs) + rows / 4.4e6,
                           4 + stages * (host_gated(a.act) ? 0.17 : 0.115)), false);
  auto take = [&](Fp8Path path, int nks, double us, double stream) {
    const double c = cost(std::max(us, start + stream * hbm), nks > 1);
    if (c < t) t = c, best = Fp8Plan{path, nks};
  };
  auto small = [&](Fp8Path path, double idle, double full, double tile, double stream) {
    const double tiles = row_tiles(kSide[path]) * std::ceil(cols / kSide[path]);
    for (int nks = 1; nks <= kMaxSlices8; nks *= 2) {
      if (nks > 1 && (a.K / kBlock8 < 4 * nks || tiles * nks > 1024)) break;
      const double n = tiles * nks / 256, st = std::ceil(stages / nks);
      double us = start + std::max(st * idle + tile, n * (st * full + tile));
      if (nks > 1) us += (a.offsets ? 5.5 : 4.0) + 8.0 * a.M * cols * nks / 5e6;
      take(path, nks, us, stream);
    }
  };
  if (a.offsets) small(k64, 0.32, 0.23, 1.4, 1.35), small(k128, 0.48, 0.53, 4.0, 1.03);
  else small(k64, 0.32, 0.19, 0.9, 1.35), small(k128, 0.48, 0.45, 3.0, 1.03);
  const double tiles = row_tiles(256) * std::ceil(cols / 256);
  const double whole = std::floor(tiles / 256), rest = tiles - 256 * whole;
  take(k256, 1, start + 3 + whole * (stages * 1.62 + 4) +
                    (rest > 0 ? stages * std::max(1.25, 1.62 * rest / 256) + 4 : 0.0), 1.05);
  return best;
}

// The plan of a launch that gathers from gT rows: past the tiles' 32-bit offsets, the few-row
// kernel, which needs no workspace either.
Fp8Plan gathered8(const LinArgs& a, const Fp8Plan& p, int gT) {
  const size_t lim = size_t(1) << 32;
  return (size_t)gT * a.K < lim && (size_t)gT * 4 < lim ? p : Fp8Plan{kRows8, 1};
}

template <bool GT>
hipError_t run_rows8(const Fp8Args& f, unsigned grid, hipStream_t s) {
  hipLaunchKernelGGL((fp8_rows_kernel<GT>), dim3(grid), dim3(256), 0, s, f);
  return hipGetLastError();
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

bool linear_fp8_fits(int E, int M, int N, int K, int act, bool grouped, int gather_rows) {
  LinArgs a = shape_args8(E, M, N, K, act, grouped);
  Fp8Plan p = plan8(a);
  if (gather_rows > 0) p = gathered8(a, p, gather_rows);
  // a grid dimension holds less than 2^32 threads: 512 a workgroup at most
  return tiles8(a, p.path) + 8 < (1LL << 32) / 512;
}

size_t linear_fp8_ws_bytes(int E, int M, int N, int K, int act, bool grouped) {
  const LinArgs a = shape_args8(E, M, N, K, act, grouped);
  const Fp8Plan p = plan8(a);
  if (p.nks <= 1) return 0;
  return (size_t)tiles8(a, p.path) * p.nks * kSide[p.path] * kSide[p.path] * sizeof(float);
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
  Fp8Plan p = plan8(shape_args8(E, M, N, K, act, offsets != nullptr));
  if (gather != nullptr) p = gathered8(f.a, p, gT);
  f.a.tiles = (int)tiles8(f.a, p.path);
  f.a.part = static_cast<float*>(ws);
  const unsigned grid = (unsigned)((f.a.tiles + 7LL) / 8 * 8);  // whole rounds of the 8 XCDs
  if (p.path != kRows8) return launch_fp8_tiles(f, kSide[p.path], p.nks, grid, s);
  return host_gated(act) ? run_rows8<true>(f, grid, s) : run_rows8<false>(f, grid, s);
}

}  // namespace moe
