// Quantisation to 8-bit floating point (e4m3, the OCP form) with one scale for each
// block of 128 elements of a row (the rows of a product) or of 128 x 128 elements (its
// weights).
//
//   amax = the block's largest finite |x|
//   s    = the least power of two with amax / s <= 448, at least 2^-126; 1 if amax = 0
//   q    = x / s rounded to e4m3, nearest, ties to even
//
// A power of two divides x exactly, so q is one rounding of x, the same in any arithmetic,
// and a scale is one byte of exponent. It costs accuracy where a few elements hold most of a
// block: amax / 448 rounds twice and uses the range up to 448, which keeps the block's
// largest element (all but) exactly. Error of the quantised values relative to the data's
// norm, power of two against amax / 448, 2^22 bf16 values: Gaussian 2.66e-2 and 2.57e-2,
// with 1 % of the elements up to 200 times as large 2.67e-2 and 0.98e-2. The products
// (linear_fp8.hip) take scales of any mantissa, so a caller can bring those. An infinity or
// NaN becomes e4m3's NaN and leaves the rest of its block alone.
//
// Bound by memory: one read, half (bf16) or a quarter (fp32) of that written, in one pass: a
// block stays in registers between its maximum and its rounding. In a graph (a copy: 5.1 to
// 5.3 TB/s): 16384 x 4096 bf16 33 us (6.0 TB/s), fp32 62 us (5.4); 8 weights of 14336 x 4096
// bf16 248 us (5.7), fp32 407 us (5.8). One row of 4096 is a launch (2.7 us, 9 a call).
#include "common.hpp"
#include "kernels.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kBlock = 128;

// 8 elements in fp32.
struct V8 {
  float v[8];
};
__device__ __forceinline__ V8 load8(const uint16_t* p) {
  const u32x4_t q = ld16(p);
  V8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.v[2 * i] = bf16_to_f32(q[i] & 0xffffu);
    r.v[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
  }
  return r;
}
__device__ __forceinline__ V8 load8(const float* p) {
  const u32x4_t a = ld16(p), b = ld16(p + 4);
  V8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.v[i] = __uint_as_float(a[i]), r.v[4 + i] = __uint_as_float(b[i]);
  return r;
}

__device__ __forceinline__ float amax8(const V8& x) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = fabsf(x.v[i]);
    m = fmaxf(m, a < INFINITY ? a : 0.0f);  // false for a NaN too
  }
  return m;
}

// Largest value over the 16 lanes of a block.
__device__ __forceinline__ float max16(float m) {
  m = fmaxf(m, __uint_as_float(partner<0>(__float_as_uint(m))));
  m = fmaxf(m, __uint_as_float(partner<1>(__float_as_uint(m))));
  m = fmaxf(m, __uint_as_float(partner<2>(__float_as_uint(m))));
  return fmaxf(m, __uint_as_float(partner<3>(__float_as_uint(m))));
}

// Biased exponent of the scale of a block: that of amax / 448 rounded up to a power of
// two (448 = 1.75 * 2^8: a mantissa above 1.75 carries into the exponent).
__device__ __forceinline__ uint32_t scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  if (u == 0) return 127;
  return (uint32_t)max((int)((u + 0x1fffffu) >> 23) - 8, 1);
}

// 8 values over 2^(e - 127) as e4m3.
__device__ __forceinline__ uint2 pack8(const V8& x, uint32_t e) {
  const float inv = __uint_as_float((254u - e) << 23);
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)  // finite ones are 448 at most
    v[i] = fabsf(x.v[i]) < INFINITY ? x.v[i] * inv : __uint_as_float(0x7fc00000u);
  uint2 r;
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
  r.x = (uint32_t)lo;
  r.y = (uint32_t)hi;
  return r;
}

// Rows: a workgroup takes 16 rows x 4 blocks, 16 lanes a block: a wave reads 4 blocks of
// one row together, and the scales of 16 rows of a block, which lie next to each other,
// leave in one store.
constexpr int kRows = 16, kKb = 4;

template <typename T>
__global__ __launch_bounds__(kThreads) void quantize_rows_kernel(const T* __restrict__ x, int rows,
                                                                int K, uint8_t* __restrict__ q,
                                                                float* __restrict__ scale) {
  __shared__ float sc[kKb][kRows];
  const int nkb = K / kBlock, groups = (nkb + kKb - 1) / kKb;
  const int row0 = (int)(blockIdx.x / groups) * kRows, kb0 = (int)(blockIdx.x % groups) * kKb;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int kb = kb0 + (lane >> 4);
  const size_t col = (size_t)min(kb, nkb - 1) * kBlock + (lane & 15) * 8;
  V8 v[kRows / 4];
#pragma unroll
  for (int i = 0; i < kRows / 4; ++i)
    v[i] = load8(x + (size_t)min(row0 + i * 4 + wave, rows - 1) * K + col);
#pragma unroll
  for (int i = 0; i < kRows / 4; ++i) {
    const int r = i * 4 + wave;
    const uint32_t e = scale_exponent(max16(amax8(v[i])));
    if ((lane & 15) == 0) sc[lane >> 4][r] = __uint_as_float(e << 23);
    if (row0 + r < rows && kb < nkb)
      *reinterpret_cast<uint2*>(q + (size_t)(row0 + r) * K + col) = pack8(v[i], e);
  }
  __syncthreads();
  const int t = threadIdx.x;
  if (t < kKb * kRows && kb0 + t / kRows < nkb && row0 + t % kRows < rows)
    scale[(size_t)(kb0 + t / kRows) * rows + row0 + t % kRows] = sc[t / kRows][t % kRows];
}

// Weights: a workgroup takes one 128 x 128 block, which stays in registers between its
// maximum and its store. The last block of an N that is no multiple of 128 has fewer rows.
template <typename T>
__global__ __launch_bounds__(kThreads) void quantize_weight_kernel(const T* __restrict__ w, int N,
                                                                  int K, uint8_t* __restrict__ q,
                                                                  float* __restrict__ scale) {
  __shared__ float top[4];
  const int nkb = K / kBlock, nnb = (N + kBlock - 1) / kBlock;
  const int kb = (int)(blockIdx.x % nkb), nb = (int)(blockIdx.x / nkb % nnb);
  const size_t mat = blockIdx.x / nkb / nnb;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const size_t at = mat * N * K + (size_t)kb * kBlock + (lane & 15) * 8;
  const int row = nb * kBlock + (threadIdx.x >> 4);  // and every 16th after it
  V8 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = load8(w + at + (size_t)min(row + 16 * i, N - 1) * K);
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, amax8(v[i]));
  m = max16(m);
  m = fmaxf(m, __uint_as_float(partner<4>(__float_as_uint(m))));
  m = fmaxf(m, __uint_as_float(partner<5>(__float_as_uint(m))));
  if (lane == 0) top[wave] = m;
  __syncthreads();
  const uint32_t e = scale_exponent(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (row + 16 * i < N)
      *reinterpret_cast<uint2*>(q + at + (size_t)(row + 16 * i) * K) = pack8(v[i], e);
  if (threadIdx.x == 0) scale[blockIdx.x] = __uint_as_float(e << 23);
}

long long row_groups(int rows, int K) {
  return ((long long)rows + kRows - 1) / kRows * ((K / kBlock + kKb - 1) / kKb);
}
long long weight_blocks(int count, int N, int K) {
  return (long long)((N + kBlock - 1) / kBlock) * (K / kBlock) * count;
}
constexpr long long kMaxGrid = (1LL << 32) / kThreads;  // a grid holds less than 2^32 threads

}  // namespace

bool quantize_fits(int rows, int K) { return row_groups(rows, K) < kMaxGrid; }
bool quantize_weight_fits(int count, int N, int K) {
  const long long per = (long long)((N + kBlock - 1) / kBlock) * (K / kBlock);
  return per < kMaxGrid && weight_blocks(count, N, K) < kMaxGrid;
}

hipError_t launch_quantize(const void* x, int rows, int K, bool bf16, void* q, float* scale,
                           hipStream_t s) {
  const dim3 grid((unsigned)row_groups(rows, K)), block(kThreads);
  uint8_t* out = static_cast<uint8_t*>(q);
  if (bf16)
    hipLaunchKernelGGL((quantize_rows_kernel<uint16_t>), grid, block, 0, s,
                       static_cast<const uint16_t*>(x), rows, K, out, scale);
  else
    hipLaunchKernelGGL((quantize_rows_kernel<float>), grid, block, 0, s,
                       static_cast<const float*>(x), rows, K, out, scale);
  return hipGetLastError();
}

hipError_t launch_quantize_weight(const void* w, int count, int N, int K, bool bf16, void* q,
                                  float* scale, hipStream_t s) {
  const dim3 grid((unsigned)weight_blocks(count, N, K)), block(kThreads);
  uint8_t* out = static_cast<uint8_t*>(q);
  if (bf16)
    hipLaunchKernelGGL((quantize_weight_kernel<uint16_t>), grid, block, 0, s,
                       static_cast<const uint16_t*>(w), N, K, out, scale);
  else
    hipLaunchKernelGGL((quantize_weight_kernel<float>), grid, block, 0, s,
                       static_cast<const float*>(w), N, K, out, scale);
  return hipGetLastError();
}

}  // namespace moe
