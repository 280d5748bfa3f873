// What the kernels of 8-bit products share.
#pragma once

#include "linear.hpp"

namespace moe {
namespace lin {

constexpr int kBlock8 = 128;  // elements of a scale block, a stage of K and a fragment row

struct Fp8Args {
  LinArgs a;
  const float* xs;  // [K / 128, rows of x]
  const float* ws;  // [E, (2,) ceil(N / 128), K / 128]
  int xrows;
};

typedef int v8i_t __attribute__((ext_vector_type(8)));

// 16 x 16 products of one block: lane l holds 32 bytes of row l % 16 of each operand.
// D as mma16.
__device__ __forceinline__ f32x4_t mma_block(u32x4_t a0, u32x4_t a1, u32x4_t b0, u32x4_t b1) {
  const v8i_t a = __builtin_bit_cast(v8i_t, __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7));
  const v8i_t b = __builtin_bit_cast(v8i_t, __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7));
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0,
                                                          0, 0, 0, 0);
}

// Scales of the weights of 128 output columns around column c of expert e: its first block.
__device__ __forceinline__ const float* w_scales(const Fp8Args& f, int e, int half, bool gt, int c) {
  const int nkb = f.a.K / kBlock8, nnb = (f.a.N + kBlock8 - 1) / kBlock8;
  return f.ws + (((size_t)e * (gt ? 2 : 1) + half) * nnb + min(c / kBlock8, nnb - 1)) * nkb;
}

__device__ __forceinline__ void fma4(f32x4_t& acc, float s, const f32x4_t& p) {
#pragma unroll
  for (int c = 0; c < 4; ++c) acc[c] = fmaf(s, p[c], acc[c]);
}

constexpr int kMaxSlices8 = 16;

// Square tiles of 64, 128 or 256 rows (linear_fp8_tiles.hip), dense or grouped, K in nks
// slices (their partial tiles in a.part).
bool fp8_tiles_ok(const LinArgs& a);  // the offsets fit the kernel's addressing
hipError_t launch_fp8_tiles(const Fp8Args& f, int rows, int nks, unsigned grid, hipStream_t s);

}  // namespace lin
}  // namespace moe
