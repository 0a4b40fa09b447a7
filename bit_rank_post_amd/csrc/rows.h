// Device helpers of the kernels that work along rows: vectors of 8 values,
// sums and maxima over a wave.
#pragma once
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
template <typename T>
__device__ __forceinline__ void store8(T* p, const float v[8]) {
  typedef typename Vec8<T>::type V8;
  V8 r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = (T)v[i];
  *reinterpret_cast<V8*>(p) = r;
}
template <>
__device__ __forceinline__ void store8<float>(float* p, const float v[8]) {
  *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
  *reinterpret_cast<f32x4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
}
// 8 neighbouring values as they lie in memory, for loads ahead of their use
template <typename T> struct Raw8 {
  typename Vec8<T>::type v;
  __device__ __forceinline__ void load(const T* p) { v = *reinterpret_cast<const typename Vec8<T>::type*>(p); }
  __device__ __forceinline__ float get(int i) const { return (float)v[i]; }
};
template <> struct Raw8<float> {
  f32x4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const f32x4*>(p);
    b = *reinterpret_cast<const f32x4*>(p + 4);
  }
  __device__ __forceinline__ float get(int i) const { return i < 4 ? a[i] : b[i - 4]; }
};
__device__ __forceinline__ float wave_sum(float v) {
  v = group_sum<32>(v);
  return v + __shfl_xor(v, 32, 64);
}

// |v| as bits: ordered like the values, with infinities and then NaN on top
__device__ __forceinline__ uint32_t abs_bits(float v) {
  return __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu;
}

}  // namespace tq
