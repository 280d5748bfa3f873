// The 8-bit products (linear_fp8.hip) on square tiles of 64, 128 or 256 rows and as many
// weight rows (BN output columns, or BN / 2 of a gated product).
//
// A wave has 64 weight rows and 32, 64 or 128 rows as accumulators of 16 x 16; the large
// tile's workgroup has 8 waves, two to a SIMD. A stage is a block of 128 k: one
// v_mfma_f32_16x16x128_f8f6f4 a sub-tile, whose sums four FMAs scale into the accumulator
// (which therefore lies in vector registers: the reason for two waves of 128 x 64 where the
// bf16 tiles have one of 128 x 128). The FMAs of an MFMA follow two MFMAs later, and the
// waves of a SIMD take turns, so the matrix core is fed while the other's FMAs run.
//
// Operand rows are copied global -> LDS (global_load_lds, 8 rows of 128 bytes a copy) into a
// ring of stages, chunk c of row r at slot c ^ ((r >> 1) & 7) as in the bf16 tiles; the rows'
// scales of the stage with them. The weights are the MFMA's A operand and the rows its B: a
// lane ends with 4 consecutive columns of one row. In a gated product half of a wave's weight
// sub-tiles holds gate rows, the other the up rows of the same columns. The weights'
// fragments stay in registers over a stage, the rows' come in two sets.
//
// Two barriers a stage. The early one stands behind a wave's first row of MFMAs, when it has
// its weight fragments of the stage in registers: the weights of the stage that takes this
// one's buffers are copied from there on, so that they have more than a whole stage to come
// from HBM (copied behind the late barrier instead: 65536 rows of 256 gated experts 797 ->
// 728 us, 8192 rows of 8 experts x 4096 x 14336 561 -> 509, 8192^3 443 -> 442). The late one
// stands where each wave has its last rows of the stage: behind it the last sub-tile row's
// MFMAs run, the next stage's first fragments are read, and that stage's rows are copied.
//
// Measured (graph replay, no act): 8192^3 442-456 us (2.4 PFLOP/s; 325 us on zeros: the power
// limit, at which MFMAs of this shape on registers alone, without the FMAs, hold 3.2), 4096^3
// 62 us of which a round's prologue, epilogue and launch take about 10 (with a bias and a
// residual 69 to 75 us: 8 to 13 more in the epilogue). Counters: MFMAs busy 40 to 43 % of the
// cycles, 6.1 to 7.8 vector instructions for each of them (four are the scaling FMAs), no LDS
// bank conflicts, and a clock of 1.7 to 2.2 GHz of 2.4. The first form of these tiles, MFMA
// and FMA in turn in one wave, took 791 and 94.
#include <algorithm>
#include <type_traits>
#include <utility>

#include "linear_fp8.hpp"

namespace moe {
namespace {

using namespace lin;

// WM x WN waves with 64 weight rows each. The ring: two stages where two workgroups of a CU
// take turns or LDS holds no more, three for the small tiles, whose launches have few waves
// to hide a copy behind (64 x 4096 x 4096 15.9 us; two stages 19.4, four 18.1; 128 x 128 tiles
// of three stages, one workgroup a CU: 2048 x 4096 x 4096 40 -> 53).
template <int BM_, int BN_, int WM_, int NS_>
struct Tile8 {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = BN / 64, NW = WM * WN;
  static constexpr int STAGES = NS_;                 // of the ring in LDS
  static constexpr int TM = BM / WM / 16, TN = 4;    // sub-tiles of a wave
  static constexpr int ROWB = kBlock8;               // bytes of a stage's row
  static constexpr int XB = BM * ROWB, WB = BN * ROWB;  // stage buffers of rows and weights
  static constexpr int SB = NW * 256;                // and of the rows' scales, more than once
  static constexpr int LDS = STAGES * (XB + WB + SB);
  static constexpr int XI = BM / 8 / NW, WI = BN / 8 / NW;  // row and weight copies of a wave
  static constexpr int PANEL = 1024 / BN;            // column tiles of an n-block of the tile order
  static_assert(TM % 2 == 0 && WI <= TN && XI <= TN && NW * 64 >= BM && BM % 64 == 0 && LDS <= 160 * 1024, "tile");
};

// First row of sub-tile i among those of the tile's first wave (wave wm: wm * 32 further on):
// pairs of sub-tiles go round the WM waves, so that a segment's last, partial row tile
// spreads over all of them.
template <int WM>
__device__ __forceinline__ constexpr int sub_row(int i) {
  return i / 2 * WM * 32 + i % 2 * 16;
}

template <typename F, int... I>
__device__ __forceinline__ void static_for_impl(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_impl(f, std::make_integer_sequence<int, N>{});
}

// Accumulator (i, j) of this thread in slice ks of a tile's partials.
template <typename Sh>
__device__ __forceinline__ float* part8(const LinArgs& a, const LinTile& t, int ks, int nks, int i, int j) {
  return a.part + ((size_t)t.q * nks + ks) * Sh::BM * Sh::BN +
         ((size_t)(i * Sh::TN + j) * (Sh::NW * 64) + threadIdx.x) * 4;
}

// blockIdx.y of gridDim.y: a K slice.
template <typename Sh, int ACT>
__global__ __launch_bounds__(Sh::NW * 64, 2) void fp8_tile_kernel(Fp8Args f) {
  constexpr int BM = Sh::BM, BN = Sh::BN, TM = Sh::TM, TN = Sh::TN, WN = Sh::WN, NW = Sh::NW;
  constexpr int ROWB = Sh::ROWB, XB = Sh::XB, WB = Sh::WB, SB = Sh::SB, XI = Sh::XI, WI = Sh::WI;
  constexpr int WM = Sh::WM, RING = Sh::STAGES, COPIES = XI + WI + 1;
  constexpr int OPEN = (RING - 2) * COPIES + WI;  // copies that may be under way at a late barrier
  constexpr bool GT = ACT == kActGeglu || ACT == kActSwiglu;
  constexpr int H = GT ? 2 : 1;
  constexpr int BC = GT ? BN / 2 : BN;            // output columns of a tile
  __shared__ __attribute__((aligned(16))) uint8_t smem[Sh::LDS];
  const LinArgs& a = f.a;
  LinTile t = lin_tile<BM, Sh::PANEL>(a, BC);
  if (t.M == 0) return;
  // the same in every lane, which the compiler cannot see: the copies' bases are scalars
  t.e = __builtin_amdgcn_readfirstlane(t.e);
  t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
  t.M = __builtin_amdgcn_readfirstlane(t.M);
  t.n0 = __builtin_amdgcn_readfirstlane(t.n0);
  const int N = a.N, K = a.K, M = t.M;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int l16 = lane & 15, kq = lane >> 4;
  const int KT0 = K / kBlock8;
  const int kbase = (int)((long long)blockIdx.y * KT0 / gridDim.y);
  const int KT = (int)((long long)(blockIdx.y + 1) * KT0 / gridDim.y) - kbase;
  const int last = max(KT - 1, 0);  // the planner gives no slice without stages

  // Copy q of a wave fills 8 rows of a stage buffer, of the rows (q < XI) or the weights;
  // lane i has row i / 8 of them, chunk (i & 7) ^ ((row >> 1) & 7). Byte offsets from the
  // operand's base fit 32 bits (checked by the host).
  const uint8_t* xb = static_cast<const uint8_t*>(a.x);
  if (a.gather == nullptr) xb += (size_t)t.row0 * K;
  xb += (size_t)kbase * kBlock8;
  const uint8_t* wb = static_cast<const uint8_t*>(a.w) + (size_t)t.e * H * N * K + (size_t)kbase * kBlock8;
  uint32_t ov[XI + WI];
#pragma unroll
  for (int q = 0; q < XI + WI; ++q) {
    const int r = (q < XI ? wave * XI + q : wave * WI + q - XI) * 8 + (lane >> 3);
    const int c = (lane & 7) ^ ((r >> 1) & 7);
    size_t row;
    if (q < XI) {
      const int p = min(r, M - 1);                // rows past the end: its last
      row = a.gather == nullptr ? (size_t)p : x_row(a, t.row0 + p);
    } else if constexpr (GT) {                    // half of a wave's sub-tiles gate, then up
      const int j = r / 16 % TN;
      row = (size_t)(j / 2) * N + min(t.n0 + r / 64 * 32 + j % 2 * 16 + r % 16, N - 1);
    } else {
      row = (size_t)min(t.n0 + r, N - 1);         // columns past the end: its last
    }
    ov[q] = (uint32_t)(row * K + c * 16);
  }
  // scale of row (wave % (BM / 64)) * 64 + lane
  const uint32_t os = (uint32_t)(x_row(a, t.row0 + min((wave % (BM / 64)) * 64 + lane, M - 1)) * 4);
  const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) uint8_t*)smem);
  constexpr int W0 = RING * XB, S0 = RING * (XB + WB);
  // copy q of stage kt into buffer buf (XI + WI: the scales)
  auto copy = [&](int kt, int buf, int q) {
    if (q == XI + WI) {
      const uint8_t* base = reinterpret_cast<const uint8_t*>(f.xs) + (size_t)(kbase + kt) * f.xrows * 4;
      const uint32_t m0 = lds0 + S0 + buf * SB + wave * 256;
      asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
                   :
                   : "v"(os), "s"(base), "s"(m0)
                   : "memory");
      return;
    }
    const uint8_t* base = (q < XI ? xb : wb) + (size_t)kt * ROWB;
    const uint32_t m0 = lds0 + (q < XI ? buf * XB + (wave * XI + q) * 8 * ROWB
                                       : W0 + buf * WB + (wave * WI + q - XI) * 8 * ROWB);
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                 :
                 : "v"(ov[q]), "s"(base), "s"(m0)
                 : "memory");
  };
  // the weights' scales of this wave's columns, which lie in one block (gate and up): lane l
  // holds those of the stages l, l + 64, ...
  const float* wsp[H];
  float wsv[H];
#pragma unroll
  for (int h = 0; h < H; ++h) wsp[h] = w_scales(f, t.e, h, GT, t.n0 + wn * (GT ? 32 : 64)) + kbase;

  f32x4_t acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const int sw = (lane >> 1) & 7;                 // (row >> 1) & 7 of every fragment row
  const int slot0 = (kq ^ sw) << 4, slot1 = ((4 + kq) ^ sw) << 4;
  const int fx = (wm * 32 + l16) * ROWB, fw = W0 + (wn * 64 + l16) * ROWB;
  const int fs = S0 + (wm * 32 + l16) * 4;
  // pairs of this wave's sub-tile rows that hold data: all except in a partial row tile
  const int nsub = __builtin_amdgcn_readfirstlane(min(TM / 2, (M + (WM - 1 - wm) * 32 + 31) / (WM * 32)));

  // Every wave's weight fragments of the stage are in registers (its first TN MFMAs have
  // them): their buffer is free for those of the stage after next.
  auto early_barrier = [] { asm volatile("s_barrier" ::: "memory"); };

  auto main_loop = [&](auto ns_tag) {
    constexpr int NS = decltype(ns_tag)::value;
    constexpr int NM = NS * TN;
    u32x4_t wf[TN][2], xf[2][2];
    float sx[2], s[2][H];                         // row scales read, and times the weights'
    f32x4_t P[4];
    auto read_w = [&](int buf, int j) {
      wf[j][0] = ld16(smem + buf * WB + fw + j * 16 * ROWB + slot0);
      wf[j][1] = ld16(smem + buf * WB + fw + j * 16 * ROWB + slot1);
    };
    auto read_x = [&](int buf, int i) {
      xf[i & 1][0] = ld16(smem + buf * XB + fx + sub_row<WM>(i) * ROWB + slot0);
      xf[i & 1][1] = ld16(smem + buf * XB + fx + sub_row<WM>(i) * ROWB + slot1);
      sx[i & 1] = *reinterpret_cast<const float*>(smem + buf * SB + fs + sub_row<WM>(i) * 4);
    };
    // prologue: the stages that fill the ring
    static_for<RING>([&](auto st) {
      constexpr int k = decltype(st)::value;
      static_for<COPIES>([&](auto q) { copy(min(k, last), k, decltype(q)::value); });
    });
    wait_vmcnt<(RING - 1) * COPIES>();
    lds_barrier();
    if constexpr (NS > 0) {
      static_for<TN>([&](auto j) { read_w(0, decltype(j)::value); });
      read_x(0, 0);
#pragma unroll
      for (int q = 0; q < 4; ++q) P[q] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int h = 0; h < H; ++h) s[0][h] = s[1][h] = 0.0f;
    }
    int buf = 0;                                  // of stage kt
    for (int kt = 0; kt < KT; ++kt) {
      const int k2 = min(kt + RING, last);        // the stage that takes this one's buffers
      const int next = buf + 1 == RING ? 0 : buf + 1;
      if ((kt & 63) == 0) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
          wsv[h] = wsp[h][min(kt + lane, last)];
          asm volatile("" : "+v"(wsv[h]));        // waited for here, not in every stage
        }
      }
      float sws[H];
#pragma unroll
      for (int h = 0; h < H; ++h)
        sws[h] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wsv[h]), kt & 63));
      if constexpr (NS == 0) {
        early_barrier();
        static_for<WI>([&](auto q) { copy(k2, buf, XI + decltype(q)::value); });
        wait_vmcnt<OPEN>();
        lds_barrier();
        static_for<XI>([&](auto q) { copy(k2, buf, decltype(q)::value); });
        copy(k2, buf, XI + WI);
      } else {
        static_for<NM>([&](auto mc) {
          constexpr int m = decltype(mc)::value, i = m / TN, j = m % TN;
          if constexpr (i == NS - 1 && j == 0) {
            // late: the last rows of this stage are in registers, stage kt + 1 landed: for everyone
            wait_vmcnt<OPEN>();
            lds_barrier();
          }
          P[m % 4] = mma_block(wf[j][0], wf[j][1], xf[i & 1][0], xf[i & 1][1]);
          __builtin_amdgcn_sched_barrier(0);
          if constexpr (m == TN - 1) early_barrier();
          if constexpr (NS == 2 && m == TN - 1)                   // weights, before the late barrier
            static_for<WI>([&](auto q) { copy(k2, buf, XI + decltype(q)::value); });
          if constexpr (NS > 2 && m >= TN - 1 && m < TN - 1 + WI) copy(k2, buf, XI + m - (TN - 1));
          if constexpr (i == NS - 1) {
            if constexpr (j < XI) copy(k2, buf, j);               // rows
            if constexpr (j == 0) copy(k2, buf, XI + WI);         // and scales
            read_w(next, j);
          }
          if constexpr (j == 1) {
            if constexpr (i + 1 < NS) read_x(buf, i + 1);
            else read_x(next, 0);
          }
          // the sums of two MFMAs ago
          constexpr int o = (m + NM - 2) % NM, oi = o / TN, oj = o % TN;
          if constexpr (j == 2) {
#pragma unroll
            for (int h = 0; h < H; ++h) s[i & 1][h] = sx[i & 1] * sws[h];
          }
          fma4(acc[oi][oj], s[oi & 1][GT && oj >= TN / 2 ? H - 1 : 0], P[(m + 2) % 4]);
          __builtin_amdgcn_sched_barrier(0);
        });
      }
      buf = next;
    }
    wait_vmcnt<0>();
    if constexpr (NS > 0) {
      constexpr int i = NS - 1;
      fma4(acc[i][2], s[i & 1][H - 1], P[2]);
      fma4(acc[i][3], s[i & 1][H - 1], P[3]);
    }
  };
  if constexpr (TM == 2) {
    if (nsub > 0) main_loop(std::integral_constant<int, 2>{});
    else main_loop(std::integral_constant<int, 0>{});
  } else if constexpr (TM == 8) {
    switch (nsub) {
      case 4: main_loop(std::integral_constant<int, 8>{}); break;
      case 3: main_loop(std::integral_constant<int, 6>{}); break;
      case 2: main_loop(std::integral_constant<int, 4>{}); break;
      case 1: main_loop(std::integral_constant<int, 2>{}); break;
      default: main_loop(std::integral_constant<int, 0>{}); break;
    }
  } else {
    switch (nsub) {
      case 2: main_loop(std::integral_constant<int, 4>{}); break;
      case 1: main_loop(std::integral_constant<int, 2>{}); break;
      default: main_loop(std::integral_constant<int, 0>{}); break;
    }
  }

  if (gridDim.y > 1) {  // a K slice: fp8_reduce_kernel adds them up
#pragma unroll
    for (int i = 0; i < TM; ++i)
      if (wm * 32 + sub_row<WM>(i) < M)
#pragma unroll
        for (int j = 0; j < TN; ++j)
          *reinterpret_cast<f32x4_t*>(part8<Sh>(a, t, blockIdx.y, gridDim.y, i, j)) = acc[i][j];
    return;
  }
  // Lane: row l16 of each row sub-tile, columns 4 kq .. + 3 of each weight sub-tile. The bias
  // is read once, the residual of RB row sub-tiles together: a load that waits behind the
  // store before it (it may be y itself) costs its whole way to memory (8192 x 4096 x 1024
  // with both 97 -> 76 us; touching the residual some stages earlier: no less).
  constexpr int TC = GT ? TN / 2 : TN, RB = TM < 4 ? TM : 4;
  const int c0 = t.n0 + wn * (GT ? 32 : 64) + kq * 4;
  uint2 bg[TC], bu[TC];
#pragma unroll
  for (int j = 0; j < TC; ++j) {
    bg[j] = bu[j] = make_uint2(0, 0);
    if (a.bias == nullptr) continue;
    const uint16_t* b = static_cast<const uint16_t*>(a.bias) + (size_t)t.e * H * N + min(c0 + j * 16, N - 4);
    bg[j] = *reinterpret_cast<const uint2*>(b);
    if constexpr (GT) bu[j] = *reinterpret_cast<const uint2*>(b + N);
  }
#pragma unroll
  for (int i0 = 0; i0 < TM; i0 += RB) {
    uint2 rv[RB][TC];
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      const int r = min(wm * 32 + sub_row<WM>(i0 + i) + l16, M - 1);
      const uint16_t* p = static_cast<const uint16_t*>(a.res) + (size_t)(t.row0 + r) * N;
#pragma unroll
      for (int j = 0; j < TC; ++j) {
        rv[i][j] = make_uint2(0, 0);
        if (a.res != nullptr) rv[i][j] = *reinterpret_cast<const uint2*>(p + min(c0 + j * 16, N - 4));
      }
    }
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      const int r = wm * 32 + sub_row<WM>(i0 + i) + l16;
      if (r >= M) continue;
#pragma unroll
      for (int j = 0; j < TC; ++j) {
        if (c0 + j * 16 >= N) continue;
        const f32x4_t &g = acc[i0 + i][j], &u = acc[i0 + i][GT ? j + TN / 2 : j];
        const Out4 o = finish4<true>(ACT, g, u, widen4(bg[j]), widen4(bu[j]), a.res != nullptr, widen4(rv[i][j]));
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + (size_t)(t.row0 + r) * N + c0 + j * 16) = pack4(o);
      }
    }
  }
}

// Sums the nks K slices of each tile in slice order, then the epilogue. One workgroup per
// row sub-tile i of a tile (blockIdx.y), so that a launch with few tiles still has many.
template <typename Sh, int ACT>
__global__ __launch_bounds__(Sh::NW * 64) void fp8_reduce_kernel(Fp8Args f, int nks) {
  constexpr bool GT = ACT == kActGeglu || ACT == kActSwiglu;
  constexpr int TN = Sh::TN;
  const LinArgs& a = f.a;
  const LinTile t = lin_tile<Sh::BM, Sh::PANEL>(a, GT ? Sh::BN / 2 : Sh::BN);
  if (t.M == 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / Sh::WN, wn = wave % Sh::WN, i = blockIdx.y;
  const int r0 = wm * 32 + sub_row<Sh::WM>(i), r = r0 + (lane & 15);
  if (r0 >= t.M) return;
  f32x4_t acc[TN];
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    f32x4_t v[kMaxSlices8];
#pragma unroll
    for (int s = 0; s < kMaxSlices8; ++s)  // all loads first, from clamped slices
      v[s] = *reinterpret_cast<const f32x4_t*>(part8<Sh>(a, t, min(s, nks - 1), nks, i, j));
    acc[j] = v[0];
#pragma unroll
    for (int s = 1; s < kMaxSlices8; ++s)
      if (s < nks) acc[j] += v[s];
  }
  if (r >= t.M) return;
#pragma unroll
  for (int j = 0; j < (GT ? TN / 2 : TN); ++j) {
    const int c = t.n0 + wn * (GT ? 32 : 64) + j * 16 + (lane >> 4) * 4;
    if (c < a.N) store4<uint16_t, ACT>(a, t.e, (size_t)(t.row0 + r), c, acc[j], acc[GT ? j + TN / 2 : j]);
  }
}

}  // namespace

namespace lin {

namespace {
template <typename Sh, int ACT>
hipError_t launch_act(const Fp8Args& f, int nks, unsigned grid, hipStream_t s) {
  hipLaunchKernelGGL((fp8_tile_kernel<Sh, ACT>), dim3(grid, nks), dim3(Sh::NW * 64), 0, s, f);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || nks <= 1) return err;
  hipLaunchKernelGGL((fp8_reduce_kernel<Sh, ACT>), dim3(grid, Sh::TM), dim3(Sh::NW * 64), 0, s, f, nks);
  return hipGetLastError();
}
template <typename Sh>
hipError_t launch_shape(const Fp8Args& f, int nks, unsigned grid, hipStream_t s) {
  switch (f.a.act) {
    case kActNone: return launch_act<Sh, kActNone>(f, nks, grid, s);
    case kActGelu: return launch_act<Sh, kActGelu>(f, nks, grid, s);
    case kActSilu: return launch_act<Sh, kActSilu>(f, nks, grid, s);
    case kActGeglu: return launch_act<Sh, kActGeglu>(f, nks, grid, s);
    default: return launch_act<Sh, kActSwiglu>(f, nks, grid, s);
  }
}
}  // namespace

hipError_t launch_fp8_tiles(const Fp8Args& f, int rows, int nks, unsigned grid, hipStream_t s) {
  switch (rows) {
    case 64: return launch_shape<Tile8<64, 64, 2, 3>>(f, nks, grid, s);
    case 128: return launch_shape<Tile8<128, 128, 2, 2>>(f, nks, grid, s);
    default: return launch_shape<Tile8<256, 256, 2, 2>>(f, nks, grid, s);
  }
}

// The kernel's 32-bit byte offsets: 256 buffer rows, an expert's weights and the scales of
// all rows, from their bases (those of gathered rows are the caller's to check).
bool fp8_tiles_ok(const LinArgs& a) {
  const size_t two = a.act == kActGeglu || a.act == kActSwiglu ? 2 : 1, lim = size_t(1) << 32;
  return std::max((size_t)256, two * a.N) * a.K < lim && (size_t)a.M * 4 < lim;
}

}  // namespace lin
}  // namespace moe
