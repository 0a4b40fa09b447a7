// Quantisation to e4m3 with one scale for each block of 128: along a row
// (activations) or 128 x 128 (weights).
//
//   amax = max |v| of the block;  c = max(fl32(amax / 448), 2^-126), 1 where
//   amax = 0;  q = e4m3(fl32(v / c)), to nearest even.
// |v / c| <= 448 (1 + 2^-23), which rounds to at most 448, the largest e4m3
// value, so nothing saturates; the lower bound keeps c a normal number where
// all of the block is below 448 2^-126.  A block with a NaN or an infinity
// gets such a scale, so everything it stands for reads back as NaN.  The
// division is the correctly rounded one: a product with 448 / amax would move
// values that lie next to a border between two codes.
//
// Bound by memory: each value is read once, 16 bytes a lane, and held in
// registers between the maximum and the division.  16384 x 4096 in bf16: 44 us,
// 4.6 TB/s (a large copy: 5.0).
#include "norm_ops.h"
#include "tq_device.h"

namespace tq {

// 8 neighbouring values as f32 (p 16-byte aligned)
template <typename T>
__device__ __forceinline__ void load8(const T* p, float v[8]) {
  typedef typename Vec8<T>::type V8;
  const V8 r = *reinterpret_cast<const V8*>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (float)r[i];
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float v[8]) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i];
    v[4 + i] = b[i];
  }
}

// |v| as bits: ordered like the values, with infinities and then NaN on top
__device__ __forceinline__ uint32_t abs_bits(float v) {
  return __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu;
}

__device__ __forceinline__ float block_scale(uint32_t amax) {
  if (amax == 0) return 1.0f;
  const float c = __builtin_bit_cast(float, amax) / 448.0f;
  return c < 1.17549435e-38f ? 1.17549435e-38f : c;
}

// The correctly rounded quotients v / c of 8 values, as codes.  By Markstein's
// method, with r = 1 / c correctly rounded, p = v r and the exact remainder
// e = v - p c (one fma), p + e r rounds v / c correctly: two fma and a product
// a value instead of a division each, which bound the kernel (16384 x 4096 in
// bf16: 53 -> 44 us).  e is exact while no bit of it is below 2^-149: it is a
// multiple of the steps of p and c, and quotients below 2^-11 are zero codes
// however they are rounded, so p's step is 2^-34 at least, and 2^-34 2^-23 c is
// 2^-149 from c = 2^-92 up.  (All 2^23 scales from 2^-92 on, and from 1 on, with
// the three values on either side of each border between two codes: no quotient
// differs from the division; from 2^-94 on some do.)  Below, and for scales that
// are no numbers, the divisions are made.
__device__ __forceinline__ u32x2 quant8(const float v[8], float c) {
  float q[8];
  if (c >= 0x1p-92f && c <= 3.0e38f) {
    const float r = 1.0f / c;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float p = v[i] * r;
      // (the negated remainder, so that its zero leaves a quotient of -0 alone)
      q[i] = __builtin_fmaf(-__builtin_fmaf(p, c, -v[i]), r, p);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = v[i] / c;
  }
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
  return u32x2{(uint32_t)lo, (uint32_t)hi};
}

__device__ __forceinline__ uint32_t max16(uint32_t v) {
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o, 64));
  return v;
}

// 16 lanes take a block of a row, 8 values each
template <typename T>
__global__ __launch_bounds__(256) void quant_rows_kernel(const T* __restrict__ x, uint32_t nblk, uint32_t nkb, int d,
                                                         long ldx, uint8_t* __restrict__ q,
                                                         float* __restrict__ scale) {
  const uint32_t blk = blockIdx.x * 16u + (threadIdx.x >> 4);
  const uint32_t row = blk / nkb;
  const int col = (int)(blk - row * nkb) * 128 + (threadIdx.x & 15) * 8;
  const bool live = blk < nblk;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (live && col < d) load8(x + row * ldx + col, v);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
  const float c = block_scale(max16(m));
  if (!live) return;
  if (col < d) *reinterpret_cast<u32x2*>(q + (size_t)row * d + col) = quant8(v, c);
  if ((threadIdx.x & 15) == 0) scale[blk] = c;
}

// a workgroup takes a 128 x 128 block of one matrix: 16 lanes a row, 16 rows
// at a time
template <typename T>
__global__ __launch_bounds__(256) void quant_blocks_kernel(const T* __restrict__ w, int d_out, int d_in,
                                                           uint8_t* __restrict__ q, float* __restrict__ scale) {
  __shared__ uint32_t s_max[4];
  const int nkb = (d_in + 127) >> 7, nob = (d_out + 127) >> 7;
  const long b = blockIdx.x;
  const int kb = (int)(b % nkb), ob = (int)(b / nkb % nob);
  const size_t base = (size_t)(b / ((long)nkb * nob)) * d_out * d_in;
  const int col = kb * 128 + (threadIdx.x & 15) * 8;
  const int r0 = ob * 128 + (threadIdx.x >> 4);
  float v[8][8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    if (r0 + 16 * i < d_out && col < d_in) load8(w + base + (size_t)(r0 + 16 * i) * d_in + col, v[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[i][j]));
  }
  m = max16(m);
  m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
  m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
  if ((threadIdx.x & 63) == 0) s_max[threadIdx.x >> 6] = m;
  __syncthreads();
  const float c = block_scale(max(max(s_max[0], s_max[1]), max(s_max[2], s_max[3])));
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (r0 + 16 * i < d_out && col < d_in)
      *reinterpret_cast<u32x2*>(q + base + (size_t)(r0 + 16 * i) * d_in + col) = quant8(v[i], c);
  if (threadIdx.x == 0) scale[b] = c;
}

template <typename T>
static void rows_go(const void* x, uint32_t nblk, uint32_t nkb, int d, long ldx, void* q, float* scale, hipStream_t s) {
  hipLaunchKernelGGL(quant_rows_kernel<T>, dim3((nblk + 15) / 16), dim3(256), 0, s, reinterpret_cast<const T*>(x),
                     nblk, nkb, d, ldx, reinterpret_cast<uint8_t*>(q), scale);
}

// (the caller keeps the number of blocks below 2^28)
void launch_quant_rows(const void* x, int dtype, int rows, int d, long ldx, void* q, float* scale,
                       hipStream_t s) {
  const uint32_t nkb = (uint32_t)(d + 127) / 128, nblk = (uint32_t)rows * nkb;
  if (nblk == 0) return;
  if (dtype == 0) rows_go<half_t>(x, nblk, nkb, d, ldx, q, scale, s);
  else if (dtype == 1) rows_go<__bf16>(x, nblk, nkb, d, ldx, q, scale, s);
  else rows_go<float>(x, nblk, nkb, d, ldx, q, scale, s);
}

void launch_quant_blocks(const void* w, int dtype, int groups, int d_out, int d_in, void* q, float* scale,
                         hipStream_t s) {
  const dim3 grid((unsigned)((long)groups * ((d_out + 127) / 128) * ((d_in + 127) / 128))), block(256);
  uint8_t* o = reinterpret_cast<uint8_t*>(q);
  if (dtype == 0)
    hipLaunchKernelGGL(quant_blocks_kernel<half_t>, grid, block, 0, s, (const half_t*)w, d_out, d_in, o, scale);
  else if (dtype == 1)
    hipLaunchKernelGGL(quant_blocks_kernel<__bf16>, grid, block, 0, s, (const __bf16*)w, d_out, d_in, o, scale);
  else
    hipLaunchKernelGGL(quant_blocks_kernel<float>, grid, block, 0, s, (const float*)w, d_out, d_in, o, scale);
}

}  // namespace tq
