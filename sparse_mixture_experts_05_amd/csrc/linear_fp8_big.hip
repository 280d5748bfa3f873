// The 8-bit products (linear_fp8.hip) on tiles of 256 rows x 256 weight rows: launches with
// enough rows to be bound by the matrix cores.
//
// A workgroup of 8 waves, two to a SIMD; wave w has the rows (w / 4) * 128 and the weight
// rows (w % 4) * 64 as 8 x 4 accumulators of 16 x 16. A stage is a block of 128 k: one
// v_mfma_f32_16x16x128_f8f6f4 a sub-tile, whose sums four FMAs scale into the accumulator
// (which therefore lies in vector registers: the reason for two waves of 128 x 64 where the
// bf16 tiles have one of 128 x 128). The FMAs of an MFMA follow two MFMAs later, and the two
// waves of a SIMD take turns, so the matrix core is fed while the other wave's FMAs run.
//
// The weights' fragments stay in registers over a stage, the rows' come in two sets. One
// barrier a stage stands where each wave has its last rows of the stage in registers: behind
// it the last sub-tile row's MFMAs run, the next stage's first fragments are read, and
// the copies of the stage after it go into the buffer that was just read.
#include <algorithm>
#include <type_traits>
#include <utility>

#include "linear_fp8.hpp"

namespace moe {
namespace {

using namespace lin;

constexpr int BM = 256, BN = 256, TM = 8, TN = 4, WN = 4, NW = 8;
constexpr int ROWB = kBlock8;                     // bytes of a stage's row
constexpr int XB = BM * ROWB, WB = BN * ROWB;     // stage buffers of rows and weights
constexpr int SB = BM * 4;                        // and of the rows' scales
constexpr int kLds = 2 * (XB + WB + 2 * SB);      // waves 4 to 7 copy scales nobody reads
constexpr int kPanel = 4;                         // column tiles of an n-block of the tile order

template <typename F, int... I>
__device__ __forceinline__ void static_for_impl(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_impl(f, std::make_integer_sequence<int, N>{});
}

template <int ACT>
__global__ __launch_bounds__(512, 2) void fp8_big_kernel(Fp8Args f) {
  constexpr bool GT = ACT == kActGeglu || ACT == kActSwiglu;
  constexpr int H = GT ? 2 : 1;
  constexpr int BC = GT ? BN / 2 : BN;            // output columns of a tile
  __shared__ __attribute__((aligned(16))) uint8_t smem[kLds];
  const LinArgs& a = f.a;
  LinTile t = lin_tile<BM, kPanel>(a, BC);
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
  const int KT = K / kBlock8, last = KT - 1;

  // Copy q of a wave fills 8 rows of a stage buffer: rows (q < 4) or weights; lane i has row
  // (wave * 4 + q) * 8 + i / 8, chunk (i & 7) ^ ((row >> 1) & 7). Byte offsets from the
  // operand's base fit 32 bits (checked by the host).
  const uint8_t* xb = static_cast<const uint8_t*>(a.x);
  if (a.gather == nullptr) xb += (size_t)t.row0 * K;
  const uint8_t* wb = static_cast<const uint8_t*>(a.w) + (size_t)t.e * H * N * K;
  uint32_t ov[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int r = (wave * 4 + q % 4) * 8 + (lane >> 3);
    const int c = (lane & 7) ^ ((r >> 1) & 7);
    size_t row;
    if (q < 4) {
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
  uint32_t os;                                    // scale of row (wave % 4) * 64 + lane
  {
    const int p = min((wave % 4) * 64 + lane, M - 1);
    os = (uint32_t)(x_row(a, t.row0 + p) * 4);
  }
  const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) uint8_t*)smem);
  constexpr int W0 = 2 * XB, S0 = 2 * (XB + WB);
  // copy q of stage kt into buffer kt & 1 (8: the scales)
  auto copy = [&](int kt, int buf, int q) {
    if (q == 8) {
      const uint8_t* base = reinterpret_cast<const uint8_t*>(f.xs) + (size_t)kt * f.xrows * 4;
      const uint32_t m0 = lds0 + S0 + buf * 2 * SB + wave * 256;
      asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
                   :
                   : "v"(os), "s"(base), "s"(m0)
                   : "memory");
      return;
    }
    const uint8_t* base = (q < 4 ? xb : wb) + (size_t)kt * ROWB;
    const uint32_t m0 = lds0 + (q < 4 ? buf * XB : W0 + buf * WB) + (wave * 4 + q % 4) * 8 * ROWB;
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
  for (int h = 0; h < H; ++h) wsp[h] = w_scales(f, t.e, h, GT, t.n0 + wn * (GT ? 32 : 64));

  f32x4_t acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const int sw = (lane >> 1) & 7;                 // (row >> 1) & 7 of every fragment row
  const int slot0 = (kq ^ sw) << 4, slot1 = ((4 + kq) ^ sw) << 4;
  const int fx = (wm * 128 + l16) * ROWB, fw = W0 + (wn * 64 + l16) * ROWB;
  const int fs = S0 + (wm * 128 + l16) * 4;
  // sub-tile rows of this wave that hold data, in pairs: all of them except in a segment's
  // last, partial row tile
  const int nsub = __builtin_amdgcn_readfirstlane(min(TM / 2, max(0, (M - wm * 128 + 31) / 32)));

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
      xf[i & 1][0] = ld16(smem + buf * XB + fx + i * 16 * ROWB + slot0);
      xf[i & 1][1] = ld16(smem + buf * XB + fx + i * 16 * ROWB + slot1);
      sx[i & 1] = *reinterpret_cast<const float*>(smem + buf * 2 * SB + fs + i * 64);
    };
    // prologue: stage 0 and the rows of stage 1
    static_for<9>([&](auto q) { copy(0, 0, decltype(q)::value); });
    static_for<4>([&](auto q) { copy(min(1, last), 1, decltype(q)::value); });
    wait_vmcnt<4>();
    lds_barrier();
    if constexpr (NS > 0) {
      static_for<TN>([&](auto j) { read_w(0, decltype(j)::value); });
      read_x(0, 0);
#pragma unroll
      for (int q = 0; q < 4; ++q) P[q] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int h = 0; h < H; ++h) s[0][h] = s[1][h] = 0.0f;
    }
    for (int kt = 0; kt < KT; ++kt) {
      const int buf = kt & 1, k1 = min(kt + 1, last), k2 = min(kt + 2, last);
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
        static_for<5>([&](auto q) { copy(k1, buf ^ 1, 4 + decltype(q)::value); });
        wait_vmcnt<0>();
        lds_barrier();
        static_for<4>([&](auto q) { copy(k2, buf, decltype(q)::value); });
      } else {
        static_for<NM>([&](auto mc) {
          constexpr int m = decltype(mc)::value, i = m / TN, j = m % TN;
          if constexpr (i == NS - 1 && j == 0) {
            // the last rows of this stage are in registers, stage kt + 1 landed: for everyone
            wait_vmcnt<0>();
            lds_barrier();
          }
          P[m % 4] = mma_block(wf[j][0], wf[j][1], xf[i & 1][0], xf[i & 1][1]);
          __builtin_amdgcn_sched_barrier(0);
          if constexpr (m < 4) copy(k1, buf ^ 1, 4 + m);          // weights and scales
          if constexpr (m == 0) copy(k1, buf ^ 1, 8);
          if constexpr (i == NS - 1) {
            copy(k2, buf, j);                                     // rows
            read_w(buf ^ 1, j);
          }
          if constexpr (j == 1) {
            if constexpr (i + 1 < NS) read_x(buf, i + 1);
            else read_x(buf ^ 1, 0);
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
    }
    wait_vmcnt<0>();
    if constexpr (NS > 0) {
      constexpr int i = NS - 1;
      fma4(acc[i][2], s[i & 1][H - 1], P[2]);
      fma4(acc[i][3], s[i & 1][H - 1], P[3]);
    }
  };
  switch (nsub) {
    case 4: main_loop(std::integral_constant<int, 8>{}); break;
    case 3: main_loop(std::integral_constant<int, 6>{}); break;
    case 2: main_loop(std::integral_constant<int, 4>{}); break;
    case 1: main_loop(std::integral_constant<int, 2>{}); break;
    default: main_loop(std::integral_constant<int, 0>{}); break;
  }

  // lane: row l16 of each row sub-tile, columns 4 kq .. + 3 of each weight sub-tile
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int r = wm * 128 + i * 16 + l16;
    if (r >= M) continue;
#pragma unroll
    for (int j = 0; j < (GT ? TN / 2 : TN); ++j) {
      const int c = t.n0 + wn * (GT ? 32 : 64) + j * 16 + kq * 4;
      if (c < N) store4<uint16_t, ACT>(a, t.e, (size_t)(t.row0 + r), c, acc[i][j], acc[i][GT ? j + TN / 2 : j]);
    }
  }
}

}  // namespace

namespace lin {

hipError_t launch_fp8_big(const Fp8Args& f, unsigned grid, hipStream_t s) {
  switch (f.a.act) {
    case kActNone: hipLaunchKernelGGL((fp8_big_kernel<kActNone>), dim3(grid), dim3(512), 0, s, f); break;
    case kActGelu: hipLaunchKernelGGL((fp8_big_kernel<kActGelu>), dim3(grid), dim3(512), 0, s, f); break;
    case kActSilu: hipLaunchKernelGGL((fp8_big_kernel<kActSilu>), dim3(grid), dim3(512), 0, s, f); break;
    case kActGeglu: hipLaunchKernelGGL((fp8_big_kernel<kActGeglu>), dim3(grid), dim3(512), 0, s, f); break;
    default: hipLaunchKernelGGL((fp8_big_kernel<kActSwiglu>), dim3(grid), dim3(512), 0, s, f); break;
  }
  return hipGetLastError();
}

// The kernel's 32-bit byte offsets: 256 buffer rows, an expert's weights, and gathered rows
// and the scales of all rows, from their bases.
bool fp8_big_ok(const LinArgs& a) {
  const size_t two = a.act == kActGeglu || a.act == kActSwiglu ? 2 : 1, lim = size_t(1) << 32;
  const size_t rows = a.gather ? (size_t)a.gT : (size_t)a.M;
  return std::max((size_t)BM, two * a.N) * a.K < lim && rows * 4 < lim && (!a.gather || rows * a.K < lim);
}

}  // namespace lin
}  // namespace moe
