// The products with an epilogue (linear.hip) on large tiles: launches with
// enough rows to be bound by the matrix cores.
//
// A workgroup of 4 waves (one per SIMD) computes 256 rows x 256 weight rows;
// wave w the 128 x 128 block (rows (w / 2) * 128, weight rows (w % 2) * 128) as
// 8 x 8 accumulators of v_mfma_f32_16x16x32_bf16 (all 256 accumulation
// registers). Of the two shapes of this rate it is the one that draws less power: on
// random data, registers only, it holds 1790-1850 TFLOP/s where v_mfma_f32_32x32x16
// holds 1500-1600 (both 2235 on zeros), and large products run at that limit: a
// 64-deep stage of 256 tiles takes 1.37 us on random data and 0.97 on zeros (1.53 and
// 0.91 with 32x32x16). The weights are the MFMA's A operand and the rows its B, so a lane
// ends with runs of 4 consecutive output columns of one row: bias and residual
// come and the result goes 8 bytes at a time, with no exchange between lanes.
// A gated product gives each wave the gate rows of 64 columns in its first four
// weight sub-tiles and their up rows in the other four: both factors of an output
// meet in one lane, and the tile has 128 output columns.
//
// With one wave per SIMD nothing else feeds the matrix core, so the stage is
// hand-ordered: the 16 fragment reads of the next 32-deep k slice and the LDS
// copies of the stage after the next (global_load_lds, the rows in two stage
// buffers, the weights in three) sit between the slice's 64 MFMAs, held there by
// sched_barrier.
//
// Tile order and the split of a long K in the last round are plan.hpp's. A
// grouped launch reads its tiles from a table that a planning launch writes from
// the device's offsets; a dense launch works its tile out in place.
#include <algorithm>
#include <type_traits>
#include <utility>

#include "linear.hpp"
#include "plan.hpp"

namespace moe {
namespace {

using namespace lin;

constexpr int kThreads = 256;
constexpr int BM = 256;                          // rows of a tile
// Column tiles per n-block of the tile order: the same panel width for both tiles.
template <int BN>
constexpr int kBlock = plan::kBlockCols * 256 / BN;
constexpr int kTableInt4 = plan::kEntryInts / 4;
constexpr size_t kPartTiles = (size_t)plan::kXcds * plan::kSlots;  // split units at most

template <typename F, int... I>
__device__ __forceinline__ void static_for_impl(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_impl(f, std::make_integer_sequence<int, N>{});
}

// The planner's view of a launch: weight rows as columns (a gated product has
// 2 N), the dense form as the one group that has no offsets.
MOE_HD inline plan::Shape shape_of(const LinArgs& a, bool gated_act) {
  const int cols = gated_act ? 2 * a.N : a.N;
  plan::Shape s{};
  if (a.offsets != nullptr) {
    s.E = a.E, s.rows = a.M, s.routed_N = cols, s.routed_K = a.K;
    s.shared_N = cols, s.shared_K = a.K;
  } else {
    s.shared_M = a.M, s.shared_N = cols, s.shared_K = a.K;
    s.routed_N = cols, s.routed_K = a.K;
  }
  s.split = a.part != nullptr ? 1 : 0;
  s.slots = a.slots;
  return s;
}

// Writes the tile table of a grouped launch: entries [0, slots) for the product
// (workgroup g: slot g / 8 on XCD g % 8), then kReduceSlots for its split-K
// reduce. Every workgroup scans the segments and resolves 256 slots.
template <int BN>
__global__ __launch_bounds__(kThreads) void lin_plan_kernel(LinArgs a) {
  __shared__ plan::Tables L;
  const plan::Shape sh = shape_of(a, gated(a.act));
  const int tid = threadIdx.x;
  int off, cnt, all, big, sml;
  plan::group_entry<BM, BN>(sh, a.offsets, tid, off, cnt, all, big, sml);
  L.goff[tid] = off;
  L.gcnt[tid] = cnt;
  L.pa[tid] = all;
  L.ps[tid] = 0;  // no pairs of short segments
  __syncthreads();
  for (int d = 1; d < 256; d <<= 1) {
    const int v = tid >= d ? L.pa[tid - d] : 0;
    __syncthreads();
    L.pa[tid] += v;
    __syncthreads();
  }
  const plan::Sched S = plan::finish_schedule(sh, L);
  const int i = blockIdx.x * kThreads + tid;
  if (i >= a.slots + plan::kReduceSlots) return;
  const int mode = i < a.slots ? 0 : 1;
  const int g = mode ? i - a.slots : i;
  plan::Tile ta{}, tb{};
  const int kind = plan::resolve_slot<BM, BN, kBlock<BN>>(sh, S, L, g % plan::kXcds,
                                                                g / plan::kXcds, mode, ta, tb);
  int e[plan::kEntryInts];
  plan::encode_entry(kind, ta, tb, e);
  int4* dst = const_cast<int4*>(a.table) + (size_t)kTableInt4 * i;
#pragma unroll
  for (int q = 0; q < kTableInt4; ++q)
    dst[q] = make_int4(e[4 * q], e[4 * q + 1], e[4 * q + 2], e[4 * q + 3]);
}

// The same in every lane (the planner's values come through LDS or arithmetic the
// compiler cannot prove uniform; the copies take their bases from scalars).
__device__ __forceinline__ plan::Tile uniform(const plan::Tile& t) {
  auto u = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
  return plan::Tile{u(t.group), u(t.e), u(t.row0), u(t.M), u(t.n0), u(t.spl), u(t.ks), u(t.unit0)};
}

// Tile of slot i (of the product, or with reduce of its reduce launch). L: LDS
// scratch for the dense form. False: no work.
template <int BN>
__device__ __forceinline__ bool tile_of(const LinArgs& a, bool gt, int i, bool reduce,
                                        plan::Tables& L, plan::Tile& t) {
  if (a.offsets != nullptr) {
    const int4* e = a.table + (size_t)kTableInt4 * (reduce ? a.slots + i : i);
    const int4 d0 = e[0];
    if (d0.x != 0) return false;
    const int4 d1 = e[1], d2 = e[2];
    t = uniform(plan::Tile{0, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w, d2.x});
    return true;
  }
  const plan::Shape sh = shape_of(a, gt);
  if (threadIdx.x == 0) {
    int off, cnt, all, big, sml;
    plan::group_entry<BM, BN>(sh, nullptr, 0, off, cnt, all, big, sml);
    L.goff[0] = off, L.gcnt[0] = cnt, L.pa[0] = all, L.pf[0] = all, L.ps[0] = 0;
  }
  __syncthreads();
  const plan::Sched S = plan::finish_schedule(sh, L);
  plan::Tile tb;
  const int kind = plan::resolve_slot<BM, BN, kBlock<BN>>(
      sh, S, L, i % plan::kXcds, i / plan::kXcds, reduce ? 1 : 0, t, tb);
  __syncthreads();  // L is the first stage buffer
  t = uniform(t);
  return kind == 0;
}

// Weight row of row r of a tile of 32 TN weight rows: the expert's row n0 + r, or
// for a gated product (n0, N in output columns) wave half r / (16 TN), sub-tile
// (r / 16) % TN: half of them gate rows, then the up rows of the same columns.
template <bool GT, int TN>
__device__ __forceinline__ size_t tile_weight_row(int r, int n0, int N) {
  if constexpr (!GT) return (size_t)min(n0 + r, N - 1);
  constexpr int HS = TN / 2;
  const int j = (r >> 4) % TN;
  return (size_t)(j / HS) * N + min(n0 + r / (16 * TN) * (16 * HS) + j % HS * 16 + (r & 15), N - 1);
}

template <int ACT, bool RES, int TN>
__global__ __launch_bounds__(256, 1) void lin_big_kernel(LinArgs a) {
  constexpr bool GT = ACT == kActGeglu || ACT == kActSwiglu;
  constexpr int NW = 4, BK = 64;
  constexpr int ROWB = BK * 2;                 // 128 bytes = 8 chunks of 16
  constexpr int TM = 8;                        // 16 x 16 sub-tiles of a wave: 8 x TN
  constexpr int BN = 32 * TN;                  // weight rows of a tile
  constexpr int RPI = 8;                       // rows per copy instruction
  constexpr int A_INST = BM / RPI / NW, B_INST = BN / RPI / NW;  // copies per wave per stage
  constexpr int A_STAGE = BM * ROWB, B_STAGE = BN * ROWB;
  constexpr int LDS_BYTES = 2 * A_STAGE + 3 * B_STAGE;
  constexpr int BC = GT ? BN / 2 : BN;         // output columns of a tile
  static_assert(LDS_BYTES <= 160 * 1024 && BM * BC * 2 <= LDS_BYTES, "LDS of one workgroup");
  __shared__ __attribute__((aligned(16))) uint8_t smem[LDS_BYTES];

  plan::Tile t;
  if (!tile_of<BN>(a, GT, blockIdx.x, false, *reinterpret_cast<plan::Tables*>(smem), t)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int N = a.N, K = a.K, M = t.M;
  const int n0 = GT ? t.n0 / 2 : t.n0;         // first output column
  const int nvalid = min(BC, N - n0);
  const int wm = wave >> 1, wn = wave & 1;
  const int wv = __builtin_amdgcn_readfirstlane(wave);

  // Copy q of a wave fills 8 rows of a stage buffer, lane i row (wave * 8 + q) *
  // 8 + i / 8, slot i & 7, which holds chunk (i & 7) ^ ((r >> 1) & 7) of the row
  // (the 16 lanes a 128-bit LDS read serves together then hit all 64 banks
  // once). ov: byte offset of the lane's chunk of K stage 0 from the operand's
  // base (the host checked that it fits 32 bits); rows and columns past the end
  // are clamped.
  const uint16_t* xb = static_cast<const uint16_t*>(a.x);
  if (a.gather == nullptr) xb += (size_t)t.row0 * K;
  const uint16_t* wb = static_cast<const uint16_t*>(a.w) + (size_t)t.e * (GT ? 2 : 1) * N * K;
  const int lrow = lane >> 3;
  uint32_t ov[A_INST + B_INST];
#pragma unroll
  for (int q = 0; q < A_INST; ++q) {
    const int r = (wave * A_INST + q) * RPI + lrow;
    const int c = (lane & 7) ^ ((r >> 1) & 7);
    const int p = min(r, M - 1);
    const size_t row = a.gather == nullptr ? (size_t)p : x_row(a, t.row0 + p);
    ov[q] = (uint32_t)((row * K + c * 8) * 2);
  }
#pragma unroll
  for (int q = 0; q < B_INST; ++q) {
    const int r = (wave * B_INST + q) * RPI + lrow;
    const int c = (lane & 7) ^ ((r >> 1) & 7);
    ov[A_INST + q] = (uint32_t)((tile_weight_row<GT, TN>(r, n0, N) * K + c * 8) * 2);
  }
  const int KT0 = K / BK;
  const int kbase = t.ks * KT0 / t.spl;
  const int KT = (t.ks + 1) * KT0 / t.spl - kbase;
  const int last = KT - 1;
  const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) uint8_t*)smem);
  const uint8_t* A8 = reinterpret_cast<const uint8_t*>(xb);
  const uint8_t* B8 = reinterpret_cast<const uint8_t*>(wb);
  auto a_buf = [&](int kt) { return smem + (kt & 1) * A_STAGE; };
  auto b_buf = [&](int slot) { return smem + 2 * A_STAGE + slot * B_STAGE; };
  // copy q of stage kt: rows (q < 8) into row buffer slot, else weights into weight
  // buffer slot
  auto copy = [&](int kt, int slot, int q) {
    const size_t kb = (size_t)(kbase + kt) * (BK * 2);
    const uint32_t m0 =
        q < A_INST ? lds0 + (uint32_t)(slot * A_STAGE + (wv * A_INST + q) * RPI * ROWB)
                   : lds0 + (uint32_t)(2 * A_STAGE + slot * B_STAGE +
                                       (wv * B_INST + q - A_INST) * RPI * ROWB);
    const uint8_t* base = (q < A_INST ? A8 : B8) + kb;
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                 :
                 : "v"(ov[q]), "s"(base), "s"(m0)
                 : "memory");
  };

  f32x4_t acc[TM][TN];  // [row sub-tile][weight sub-tile]
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  // Every fragment row of this lane is lane % 16 of a 16-row sub-tile: one LDS offset
  // per operand, the sub-tiles 16 rows apart (a constant of the read).
  const int fa0 = (wm * 128 + (lane & 15)) * ROWB;
  const int fb0 = (wn * (BN / 2) + (lane & 15)) * ROWB;
  const int sw = (lane >> 1) & 7;
  const int kq = lane >> 4;
  // pairs of row sub-tiles of this wave that hold data: all of them except in a
  // segment's last, partial row tile (a wave-uniform count)
  const int nsub = __builtin_amdgcn_readfirstlane(min(TM / 2, max(0, (M - wm * 128 + 31) / 32)));

  u32x4_t ca[TM], cb[TN], na[TM], nb[TN];
  constexpr int NM = TM * TN, NR = TM + TN;  // MFMAs, fragment reads of a k slice
  // fragment read r of k slice ks: b0, a0, the other b, the other a (the order of
  // first use)
  auto read_r = [&](const uint8_t* sa, const uint8_t* sb, int ks, int r, u32x4_t (&fa_)[TM],
                    u32x4_t (&fb_)[TN]) {
    const int off = ((ks * 4 + kq) ^ sw) << 4;
    if (r == 0) fb_[0] = ld16(sb + fb0 + off);
    else if (r == 1) fa_[0] = ld16(sa + fa0 + off);
    else if (r <= TN) fb_[r - 1] = ld16(sb + fb0 + (r - 1) * 16 * ROWB + off);
    else fa_[r - TN] = ld16(sa + fa0 + (r - TN) * 16 * ROWB + off);
  };
  // NS: row sub-tiles with data, a compile-time count, so that a partial tile's
  // loop has no branch between its MFMAs (its empty sub-tiles are skipped)
  auto main_loop = [&](auto ns_tag) {
    constexpr int NS = decltype(ns_tag)::value;
    // one k slice: NM MFMAs on (fa_, fb_); over the first half of them the
    // reads of slice rks of the buffers (rsa, rsb) into (ra_, rb_); copies q0 .. q1-1
    // (of stage ckt into slot) spread evenly
    auto slice = [&](const u32x4_t (&fa_)[TM], const u32x4_t (&fb_)[TN], const uint8_t* rsa,
                     const uint8_t* rsb, int rks, u32x4_t (&ra_)[TM], u32x4_t (&rb_)[TN],
                     auto q0c, auto q1c, int ckt, int slot) {
      constexpr int q0 = decltype(q0c)::value, nq = decltype(q1c)::value - q0;
      static_for<NM>([&](auto mc) {
        constexpr int m = decltype(mc)::value, i = m / TN, j = m % TN;
        if constexpr (i < NS) acc[i][j] = mma16<uint16_t>(fb_[j], fa_[i], acc[i][j]);
        constexpr int r = (m * NR * 2 + NM - 1) / NM;  // the first read not before m
        constexpr bool reads = r < NR && r * NM / (NR * 2) == m;
        constexpr bool copies = (m * nq) / NM != ((m + 1) * nq) / NM;
        if constexpr (reads || copies || m % 4 == 3) __builtin_amdgcn_sched_barrier(0);
        if constexpr (reads) {
          read_r(rsa, rsb, rks, r, ra_, rb_);
          __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (copies) {
          constexpr int q = q0 + (m * nq) / NM;
          copy(ckt, slot, q);
          __builtin_amdgcn_sched_barrier(0);
        }
      });
    };
    using Q0 = std::integral_constant<int, 0>;  // copies: rows, then weights
    using Q1 = std::integral_constant<int, A_INST>;
    using Q2 = std::integral_constant<int, A_INST + B_INST>;
    // prologue: stages 0 and 1 and the weights of stage 2 in flight, in the order
    // the waits count them; stage 0 landed everywhere
    static_for<A_INST + B_INST>([&](auto q) { copy(0, 0, decltype(q)::value); });
    static_for<A_INST + B_INST>([&](auto q) { copy(min(1, last), 1, decltype(q)::value); });
    static_for<B_INST>([&](auto q) { copy(min(2, last), 2, A_INST + decltype(q)::value); });
    wait_vmcnt<A_INST + 2 * B_INST>();
    lds_barrier();
    static_for<NR>([&](auto r) { read_r(a_buf(0), b_buf(0), 0, decltype(r)::value, ca, cb); });
    // One code path for every stage: past the end the copies fetch the last stage
    // again into buffers nobody reads any more and the reads fetch a stale buffer
    // (both in bounds); the copies are drained before the epilogue reuses the LDS.
    int bs = 0;  // weight slot of stage kt (kt mod 3)
    for (int kt = 0; kt < KT; ++kt) {
      const int bs1 = bs == 2 ? 0 : bs + 1;
      const int bsp = bs == 0 ? 2 : bs - 1;  // slot of stage kt-1 = stage kt+2
      const int k2 = min(kt + 2, last);
      slice(ca, cb, a_buf(kt), b_buf(bs), 1, na, nb, Q1{}, Q2{}, k2, bsp);
      // stage kt+1 landed for this wave (only the weights of stage kt+2 issued
      // above may still be in flight), then for everyone; stage kt fully read, so
      // row buffer kt & 1 is free
      wait_vmcnt<B_INST>();
      lds_barrier();
      slice(na, nb, a_buf(kt + 1), b_buf(bs1), 0, ca, cb, Q0{}, Q1{}, k2, kt & 1);
      bs = bs1;
    }
    wait_vmcnt<0>();
    // every accumulator leaves each variant in its accumulation registers, so the
    // variants meet the epilogue with one register assignment
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) asm volatile("" : "+a"(acc[i][j]));
  };
  switch (nsub) {
    case 4: main_loop(std::integral_constant<int, 8>{}); break;
    case 3: main_loop(std::integral_constant<int, 6>{}); break;
    case 2: main_loop(std::integral_constant<int, 4>{}); break;
    case 1: main_loop(std::integral_constant<int, 2>{}); break;
    default: main_loop(std::integral_constant<int, 0>{}); break;
  }

  // 16x16 D layout: lane holds row lane % 16 of x (column of D) and the weight rows
  // 4 (lane / 16) .. + 3 of each sub-tile.
  if (t.unit0 >= 0) {
    // one K slice of a split tile: 16 bytes per lane in accumulator order; the
    // reduce launch sums the slices and runs the epilogue
    float* P = a.part + (size_t)(t.unit0 + t.ks) * BM * BN + wave * (BM * BN / 4) + lane * 4;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        asm volatile("" : "+a"(acc[i][j]));
        *reinterpret_cast<f32x4_t*>(P + (i * TN + j) * 256) = acc[i][j];
      }
    return;
  }
  // Finished columns go to a [256 x BC] bf16 tile in LDS (the stages are free),
  // then whole rows to memory, 16 bytes a lane. The 16-byte chunks of a row are
  // XOR-swizzled by its low bits, so the rows of a write spread over the banks.
  constexpr int CROWB = BC * 2;
  constexpr int SWZ = (CROWB / 16 < 16 ? CROWB / 16 : 16) - 1;
  const uint16_t* bias = static_cast<const uint16_t*>(a.bias);
  const uint16_t* res = static_cast<const uint16_t*>(a.res);
  const int lr = wm * 128 + (lane & 15);            // first row of this lane in the tile
  const int lc = wn * (BC / 2) + kq * 4;            // first column
  constexpr int STEPS = GT ? TN / 2 : TN;           // weight sub-tiles that give outputs
  // the bias of every sub-tile up front (a branch in every step would have the
  // compiler spill accumulators)
  uint2 bgs[STEPS], bus[GT ? STEPS : 1];
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    bgs[s] = make_uint2(0u, 0u);
    if constexpr (GT) bus[s] = make_uint2(0u, 0u);
  }
  if (bias != nullptr) {
    bias += (size_t)t.e * (GT ? 2 : 1) * N + n0;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int cc = min(lc + s * 16, nvalid - 4);
      bgs[s] = *reinterpret_cast<const uint2*>(bias + cc);
      if constexpr (GT) bus[s] = *reinterpret_cast<const uint2*>(bias + N + cc);
    }
  }
  if constexpr (RES) res += (size_t)t.row0 * N + n0;
  lds_barrier();  // every wave has read the last stage
  static_for<STEPS>([&](auto sc) {
    constexpr int j = decltype(sc)::value;
    const int col = lc + j * 16;
    const Out4 bg = widen4(bgs[j]), bu = widen4(bus[GT ? j : 0]);
    uint2 rv[TM];
    if constexpr (RES) {
#pragma unroll
      for (int i = 0; i < TM; ++i)
        rv[i] = *reinterpret_cast<const uint2*>(res + (size_t)min(lr + i * 16, M - 1) * N +
                                                min(col, nvalid - 4));
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      // pinned to the accumulation registers up to here: without this the compiler
      // reads all of them out before the first branch of the epilogue, and spills
      asm volatile("" : "+a"(acc[i][j]));
      if constexpr (GT) asm volatile("" : "+a"(acc[i][j + TN / 2]));
      Out4 r{};
      if constexpr (RES) r = widen4(rv[i]);
      const uint2 o = pack4(finish4<true>(ACT, acc[i][j], acc[i][GT ? j + TN / 2 : j], bg, bu, RES, r));
      const int row = lr + i * 16;
      *reinterpret_cast<uint2*>(smem + row * CROWB + (((col >> 3) ^ (row & SWZ)) << 4) + (kq & 1) * 8) = o;
    }
    __builtin_amdgcn_sched_barrier(0);
  });
  lds_barrier();
  constexpr int LPR = CROWB / 16, RPW = 64 / LPR;   // lanes per row, rows per store
  uint16_t* y = static_cast<uint16_t*>(a.y) + (size_t)t.row0 * N + n0;
  const int cl = lane % LPR;
  const bool cok = cl * 8 < nvalid;  // N % 64 == 0: 8-column chunks are all or nothing
#pragma unroll 4
  for (int it = 0; it < BM / NW / RPW; ++it) {
    const int row = wave * (BM / NW) + it * RPW + lane / LPR;
    const u32x4_t v = ld16(smem + row * CROWB + ((cl ^ (row & SWZ)) << 4));
    if (cok && row < M) st16(y + (size_t)row * N + cl * 8, v);
  }
}

// Sums the K slices of each split tile in slice order and runs the epilogue.
// kReduceParts workgroups share a tile (one wave's row sub-tiles are spread over
// them), so the partials stream through many CUs.
constexpr int kReduceParts = 8;

template <int ACT, int TN>
__global__ __launch_bounds__(kThreads) void lin_reduce_kernel(LinArgs a) {
  constexpr bool GT = ACT == kActGeglu || ACT == kActSwiglu;
  constexpr int BN = 32 * TN;
  __shared__ plan::Tables L;
  plan::Tile t;
  if (!tile_of<BN>(a, GT, blockIdx.x / kReduceParts, true, L, t)) return;
  const int N = a.N;
  const int n0 = GT ? t.n0 / 2 : t.n0;
  const int nvalid = N - n0;
  const float* P = a.part + (size_t)t.unit0 * BM * BN;
  const int spl = t.spl;
  constexpr int JS = GT ? TN / 2 : TN;  // weight sub-tiles that give outputs
  constexpr int RUNS = 4 * 8 * JS * 64;  // runs of 4 columns in a tile
  for (int e = (blockIdx.x % kReduceParts) * kThreads + threadIdx.x; e < RUNS;
       e += kReduceParts * kThreads) {
    // e = ((wave * 8 + i) * JS + j) * 64 + lane, the partials' order
    const int lane = e & 63, j = (e >> 6) % JS, wi = (e >> 6) / JS;
    const int wave = wi >> 3, i = wi & 7;
    const int row = (wave >> 1) * 128 + i * 16 + (lane & 15);
    const int col = (wave & 1) * (JS * 16) + j * 16 + (lane >> 4) * 4;
    if (row >= t.M || col >= nvalid) continue;
    const float* src = P + (size_t)wave * (BM * BN / 4) + lane * 4;
    f32x4_t g{}, u{};
    f32x4_t vg[plan::kMaxSplit], vu[plan::kMaxSplit];
#pragma unroll
    for (int ks = 0; ks < plan::kMaxSplit; ++ks) {  // all loads first, from clamped slices
      const float* sl = src + (size_t)min(ks, spl - 1) * BM * BN;
      vg[ks] = *reinterpret_cast<const f32x4_t*>(sl + (i * TN + j) * 256);
      if constexpr (GT) vu[ks] = *reinterpret_cast<const f32x4_t*>(sl + (i * TN + j + TN / 2) * 256);
    }
#pragma unroll
    for (int ks = 0; ks < plan::kMaxSplit; ++ks)
      if (ks < spl) {
        g += vg[ks];
        if constexpr (GT) u += vu[ks];
      }
    store4<uint16_t>(a, t.e, (size_t)(t.row0 + row), n0 + col, g, u);
  }
}

// Split flag, workgroups and workspace layout (partial tiles | table) of a launch.
struct BigLayout {
  bool split;
  int slots;
  size_t part, table, bytes;
};

template <int BN>
BigLayout big_layout(const LinArgs& a) {
  LinArgs b = a;
  b.part = nullptr;
  b.slots = 0;
  plan::Shape sh = shape_of(b, a.act == kActGeglu || a.act == kActSwiglu);
  BigLayout L{};
  sh.split = L.split = plan::split_ok(sh);
  L.slots = plan::launch_slots<BM, BN>(sh);
  L.table = L.split ? kPartTiles * BM * BN * sizeof(float) : 0;
  L.bytes = L.table + (a.offsets ? (size_t)(L.slots + plan::kReduceSlots) * kTableInt4 * sizeof(int4) : 0);
  return L;
}

template <int ACT, int TN>
hipError_t run_big(const LinArgs& a, hipStream_t s) {
  if (a.res != nullptr)
    hipLaunchKernelGGL((lin_big_kernel<ACT, true, TN>), dim3(a.slots), dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((lin_big_kernel<ACT, false, TN>), dim3(a.slots), dim3(kThreads), 0, s, a);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || a.part == nullptr) return err;
  hipLaunchKernelGGL((lin_reduce_kernel<ACT, TN>), dim3(plan::kReduceSlots * kReduceParts),
                     dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

template <int TN>
hipError_t launch_big_tn(LinArgs a, void* ws, hipStream_t s) {
  const BigLayout L = big_layout<32 * TN>(a);
  uint8_t* base = static_cast<uint8_t*>(ws);
  a.part = L.split ? reinterpret_cast<float*>(base) : nullptr;
  a.slots = L.slots;
  if (a.offsets) {
    a.table = reinterpret_cast<const int4*>(base + L.table);
    const int n = L.slots + plan::kReduceSlots;
    hipLaunchKernelGGL((lin_plan_kernel<32 * TN>), dim3((n + kThreads - 1) / kThreads), dim3(kThreads),
                       0, s, a);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  switch (a.act) {
    case kActNone: return run_big<kActNone, TN>(a, s);
    case kActGelu: return run_big<kActGelu, TN>(a, s);
    case kActSilu: return run_big<kActSilu, TN>(a, s);
    case kActGeglu: return run_big<kActGeglu, TN>(a, s);
    default: return run_big<kActSwiglu, TN>(a, s);
  }
}

}  // namespace

namespace lin {

// The kernel's 32-bit byte offsets: 256 buffer rows and an expert's weights from the
// tile's base, and gathered rows from x.
constexpr size_t kOffsets = size_t(1) << 32;
bool big_ok(const LinArgs& a) {
  const bool gt = a.act == kActGeglu || a.act == kActSwiglu;
  return std::max((size_t)BM, (size_t)(gt ? 2 : 1) * a.N) * a.K * 2 < kOffsets;
}
bool big_gather_ok(const LinArgs& a) { return (size_t)a.gT * a.K * 2 < kOffsets; }

size_t big_ws_bytes(const LinArgs& a, bool half) {
  return half ? big_layout<128>(a).bytes : big_layout<256>(a).bytes;
}

int big_slices(const LinArgs& a, bool half) {
  LinArgs b = a;
  b.part = nullptr;
  b.slots = 0;
  plan::Shape sh = shape_of(b, a.act == kActGeglu || a.act == kActSwiglu);
  sh.split = plan::split_ok(sh);
  if (!sh.split) return 1;
  if (a.offsets != nullptr) return 0;
  plan::Tables L;
  L.pf[0] = L.pa[0] = plan::cdiv(sh.shared_M, BM) * plan::cdiv(sh.shared_N, half ? 128 : 256);
  L.ps[0] = 0;
  return plan::finish_schedule(sh, L).spl;
}

hipError_t launch_big(LinArgs a, bool half, void* ws, hipStream_t s) {
  return half ? launch_big_tn<4>(a, ws, s) : launch_big_tn<8>(a, ws, s);
}

}  // namespace lin
}  // namespace moe
