// Between the two products of a layer of experts: SwiGLU, its gradient, and
// quantisation of rows to 8-bit integers, alone or of SwiGLU's result.
//
//   swiglu    h = silu(g) u,  silu(g) = g s,  s = 1 / (1 + e^-g);  a = (g | u)
//   gradient  du = dh g s,  dg = dh u s (1 + g (1 - s))
//   int8      amax = max |v| of the row;  c = max(fl32(amax / 127), 2^-126), 1
//             where amax = 0;  q = rint(fl32(v / c))
// All in f32; h, da and q are rounded once.  |v / c| <= 127 (1 + 2^-23) rounds
// to 127 at most, so nothing saturates and -128 never appears.  A row with a
// NaN or an infinity gets a scale of NaN and codes of 0: all that it stands
// for, and every product with it, reads NaN.
//
// Bound by memory.  swiglu and its gradient are streams of vectors of 8: 32768 x
// 14336 in bf16 497 us, 5.7 TB/s of what they must move (a large copy: 4.9), the
// gradient of 24960 x 1408 with dh in f32 and h again 86 us, 5.7 TB/s.  A row to be
// quantised is read once and stays in registers as f32 between the maximum and
// the division: below 2048 values in one wave, which needs no barrier, above in
// a workgroup; above 32768 the rest is read again (24960 x 1408, of SwiGLU in f16:
// 41 us, 4.3 TB/s).
#include "layer_ops.h"
#include "rows.h"

namespace tq {

// 1 / (1 + e^-g).  The exponent's product with log2 e is carried to twice 32
// bits (t + lo), since its rounding alone would cost |g| 2^-25 of e^-g; the
// hardware's base-2 exponential and reciprocal add about an ulp each.  Below
// -88, where the sigmoid leaves the normal numbers, it is taken as 0 (off by
// less than 2^-126).  rest: 1 - s, as e^-g s, which keeps its bits where s is
// next to 1 (the difference has an error of 2^-24 of s, which the slope of silu
// multiplies by g: 10 units of 2^-24 of a slope of 1 at g = 10, by the product
// a hundredth); above 88 it is taken as 0.
__device__ __forceinline__ float sigmoid(float g, float* rest = nullptr) {
  const float v = fminf(fmaxf(g, -88.f), 88.f);
  const float L = -1.44269504f, LL = -1.92596303e-8f;      // -log2 e = L + LL
  const float t = v * L;
  const float lo = __builtin_fmaf(v, LL, __builtin_fmaf(v, L, -t));
  float e = __builtin_amdgcn_exp2f(t);
  e = __builtin_fmaf(e, lo * 0.693147181f, e);
  const float s = __builtin_amdgcn_rcpf(1.f + e);
  if (rest != nullptr) *rest = g > 88.f ? 0.f : e * s;
  return g < -88.f ? 0.f : s;
}

// The rows that a call works on: [lo, hi), clamped so that any offsets stay
// inside 0 .. rows.
__device__ __forceinline__ void live_rows(const int* off, int groups, int rows, int* lo, int* hi) {
  *lo = 0;
  *hi = rows;
  if (off == nullptr) return;
  *lo = min(max(off[0], 0), rows);
  *hi = min(max(off[groups], *lo), rows);
}

// ---- elementwise ----------------------------------------------------------------

// Vector v of rows r0 .. r0 + n - 1 taken as one list of n * nv vectors.
template <typename A, typename H>
__global__ __launch_bounds__(256) void swiglu_kernel(SwigluArgs a, int r0, uint32_t items, uint32_t nv) {
  int lo, hi;
  live_rows(a.off, a.groups, a.rows, &lo, &hi);
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  const uint32_t r = i / nv;
  const long row = (long)r0 + r;
  if (i >= items || row < lo || row >= hi) return;
  const int c = (int)(i - r * nv) * 8;
  float g[8], u[8];
  const A* p = reinterpret_cast<const A*>(a.a) + row * a.lda + c;
  load8(p, g);
  load8(p + a.ff, u);
#pragma unroll
  for (int j = 0; j < 8; ++j) g[j] = g[j] * sigmoid(g[j]) * u[j];
  store8(reinterpret_cast<H*>(a.h) + row * a.ldh + c, g);
}

template <typename A, typename H>
__global__ __launch_bounds__(256) void swiglu_grad_kernel(SwigluArgs a, int r0, uint32_t items, uint32_t nv) {
  int lo, hi;
  live_rows(a.off, a.groups, a.rows, &lo, &hi);
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  const uint32_t r = i / nv;
  const long row = (long)r0 + r;
  if (i >= items || row < lo || row >= hi) return;
  const int c = (int)(i - r * nv) * 8;
  float g[8], u[8], dh[8], h[8];
  const A* p = reinterpret_cast<const A*>(a.a) + row * a.lda + c;
  load8(p, g);
  load8(p + a.ff, u);
  load8(reinterpret_cast<const H*>(a.dh) + row * a.lddh + c, dh);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float rest;
    const float s = sigmoid(g[j], &rest), gs = g[j] * s;
    h[j] = gs * u[j];
    const float du = dh[j] * gs;
    // s (1 + g (1 - s)) = s + g s (1 - s); the larger factor meets it first, or a
    // product on the way could leave f32 where the gradient does not
    const bool up = __builtin_fabsf(u[j]) > __builtin_fabsf(dh[j]);
    g[j] = __builtin_fmaf(gs, rest, s) * (up ? u[j] : dh[j]) * (up ? dh[j] : u[j]);
    u[j] = du;
  }
  A* o = reinterpret_cast<A*>(a.da) + row * a.ldda + c;
  store8(o, g);
  store8(o + a.ff, u);
  if (a.h != nullptr) store8(reinterpret_cast<A*>(a.h) + row * a.ldh + c, h);
}

// ---- quantisation of rows ---------------------------------------------------------

template <typename T> struct PlainRows {
  const T* p;
  long ld;
  __device__ __forceinline__ void get(long row, int c, int, float v[8]) const { load8(p + row * ld + c, v); }
};
template <typename T> struct SwigluRows {
  const T* p;
  long ld;
  __device__ __forceinline__ void get(long row, int c, int d, float v[8]) const {
    float u[8];
    load8(p + row * ld + c, v);
    load8(p + row * ld + d + c, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = v[j] * sigmoid(v[j]) * u[j];
  }
};

// The scale of a row from its largest |v|; NaN where that is no number.
__device__ __forceinline__ float row_scale8(uint32_t amax) {
  if (amax == 0) return 1.0f;
  if (amax >= 0x7F800000u) return __builtin_nanf("");
  const float c = __builtin_bit_cast(float, amax) / 127.0f;
  return c < 1.17549435e-38f ? 1.17549435e-38f : c;
}

// Codes of 8 values.  The correctly rounded quotients come from the correctly
// rounded reciprocal, a product and two fma (Markstein), which is a division's
// result while no bit of the remainder is below 2^-149: quotients below 2^-2
// are code 0 however they are rounded, so the product's step is 2^-26 at least,
// and 2^-26 2^-23 c is 2^-149 from c = 2^-100 up; from 2^-92 it is used.  (All
// 2^23 scales from 1 on, with the values on either side of each border between
// two codes: every code is that of the division; a product with 1 / c alone
// gives another code for 5 % of them.)  Adding 1.5 2^23 rounds to the nearest
// whole number, ties to even, and leaves it in the low byte.
__device__ __forceinline__ u32x2 codes8(const float v[8], float c) {
  float q[8];
  if (c >= 0x1p-92f) {
    const float r = 1.0f / c;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float p = v[i] * r;
      q[i] = __builtin_fmaf(-__builtin_fmaf(p, c, -v[i]), r, p);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = v[i] / c;
  }
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = __builtin_bit_cast(uint32_t, q[i] + 12582912.0f);
  u32x2 o;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __builtin_amdgcn_perm(b[4 * h + 1], b[4 * h], 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[4 * h + 3], b[4 * h + 2], 0x04000C0Cu);
    o[h] = lo | hi;
  }
  return c == c ? o : u32x2{0u, 0u};          // (no number: codes of 0)
}

__device__ __forceinline__ uint32_t wave_max_u(uint32_t v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o, 64));
  return v;
}

// A row is taken by a wave (WAVE) or by the workgroup; each thread keeps VPT
// vectors.  Rows of a workgroup that are longer still are read again for the
// codes.
template <class Rows, bool WAVE, int VPT>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void int8_rows_kernel(Rows x, Int8RowsArgs a) {
  __shared__ uint32_t s_max[2][16];
  const int NTH = WAVE ? 64 : blockDim.x;
  const int tid = WAVE ? threadIdx.x & 63 : threadIdx.x;
  int lo, hi;
  live_rows(a.off, a.groups, a.rows, &lo, &hi);
  const long first = WAVE ? (long)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  const long stride = (long)gridDim.x * (WAVE ? 4 : 1);
  const int nv = a.d >> 3;
  int ph = 0;
  for (long row = lo + first; row < hi; row += stride, ph ^= 1) {
    float v[VPT][8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = tid + i * NTH;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
      if (c < nv) x.get(row, c * 8, a.d, v[i]);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[i][j]));
    if constexpr (!WAVE) {
      for (int c = tid + VPT * NTH; c < nv; c += NTH) {
        float f[8];
        x.get(row, c * 8, a.d, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, abs_bits(f[j]));
      }
    }
    m = wave_max_u(m);
    if constexpr (!WAVE) {
      // (two sets: a wave that is a row ahead writes the other one)
      if ((threadIdx.x & 63) == 0) s_max[ph][threadIdx.x >> 6] = m;
      __syncthreads();
      m = 0;
      for (int w = 0; w < NTH >> 6; ++w) m = max(m, s_max[ph][w]);
    }
    const float c = row_scale8(m);
    int8_t* q = a.q + row * a.d;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int k = tid + i * NTH;
      if (k < nv) *reinterpret_cast<u32x2*>(q + k * 8) = codes8(v[i], c);
    }
    if constexpr (!WAVE) {
      for (int k = tid + VPT * NTH; k < nv; k += NTH) {
        float f[8];
        x.get(row, k * 8, a.d, f);
        *reinterpret_cast<u32x2*>(q + k * 8) = codes8(f, c);
      }
    }
    if (tid == 0) a.scale[row] = c;
  }
}

// ---- launch -----------------------------------------------------------------------

// Rows in parts whose vectors a 32-bit index counts.
template <class F>
static void in_parts(int rows, int ff, F launch) {
  const uint32_t nv = (uint32_t)ff / 8;
  const long part = ((1L << 31) - 256) / nv;
  for (long r0 = 0; r0 < rows; r0 += part) {
    const uint32_t n = (uint32_t)(rows - r0 < part ? rows - r0 : part);
    launch((int)r0, n * nv, nv, dim3((n * nv + 255) / 256));
  }
}

template <typename A, typename H>
static void go_swiglu(const SwigluArgs& a, bool grad, hipStream_t s) {
  in_parts(a.rows, a.ff, [&](int r0, uint32_t items, uint32_t nv, dim3 grid) {
    if (grad) hipLaunchKernelGGL((swiglu_grad_kernel<A, H>), grid, dim3(256), 0, s, a, r0, items, nv);
    else hipLaunchKernelGGL((swiglu_kernel<A, H>), grid, dim3(256), 0, s, a, r0, items, nv);
  });
}
template <typename A>
static void go_swiglu_h(const SwigluArgs& a, bool grad, int hdt, hipStream_t s) {
  if (hdt == 0) go_swiglu<A, half_t>(a, grad, s);
  else if (hdt == 1) go_swiglu<A, __bf16>(a, grad, s);
  else go_swiglu<A, float>(a, grad, s);
}
static void go_swiglu_a(const SwigluArgs& a, bool grad, int adt, int hdt, hipStream_t s) {
  if (adt == 0) go_swiglu_h<half_t>(a, grad, hdt, s);
  else if (adt == 1) go_swiglu_h<__bf16>(a, grad, hdt, s);
  else go_swiglu_h<float>(a, grad, hdt, s);
}
void launch_swiglu(const SwigluArgs& a, int adt, int hdt, hipStream_t s) { go_swiglu_a(a, false, adt, hdt, s); }
void launch_swiglu_grad(const SwigluArgs& a, int adt, int hdt, hipStream_t s) { go_swiglu_a(a, true, adt, hdt, s); }

template <class Rows>
static void go_int8(const Int8RowsArgs& a, Rows x, hipStream_t s) {
  const int nv = a.d / 8;
  const long most = 1 << 16;                    // workgroups; more rows are taken in turns
  const unsigned by_wave = (unsigned)(((long)a.rows + 3) / 4 < most ? ((long)a.rows + 3) / 4 : most);
  const unsigned by_group = (unsigned)(a.rows < most ? a.rows : most);
  // us for 64, 4096 and 16384 rows of bf16, a wave and a workgroup (two vectors a
  // thread) a row: 1024 values 2.9, 3.9, 10.9 and 3.1, 4.6, 11.1; 1408: 3.3, 4.6, 14.8
  // and 3.1, 5.6, 14.8; 2048: 3.6, 5.4, 18.9 and 3.2, 6.1, 17.9; 4096: 4.8, 10.5, 35.6 and
  // 3.3, 11.2, 31.6.  Two and four vectors a thread: 8192 values 3.4, 17.8, 70.7 and
  // 3.9, 19.2, 76.1; 14336 values, 64 and 4096 rows: 4.2, 38.0 and 4.1, 32.3.
  if (nv <= 128) {
    hipLaunchKernelGGL((int8_rows_kernel<Rows, true, 2>), dim3(by_wave), dim3(256), 0, s, x, a);
  } else if (nv < 256) {
    hipLaunchKernelGGL((int8_rows_kernel<Rows, true, 4>), dim3(by_wave), dim3(256), 0, s, x, a);
  } else if (nv <= 1024) {
    hipLaunchKernelGGL((int8_rows_kernel<Rows, false, 2>), dim3(by_group), dim3((nv + 127) / 128 * 64), 0, s, x, a);
  } else {
    const int waves = (nv + 255) / 256 < 16 ? (nv + 255) / 256 : 16;
    hipLaunchKernelGGL((int8_rows_kernel<Rows, false, 4>), dim3(by_group), dim3(64 * waves), 0, s, x, a);
  }
}
template <typename T>
static void go_int8_t(const Int8RowsArgs& a, bool swiglu, hipStream_t s) {
  const T* p = reinterpret_cast<const T*>(a.x);
  if (swiglu) go_int8(a, SwigluRows<T>{p, a.ldx}, s);
  else go_int8(a, PlainRows<T>{p, a.ldx}, s);
}
void launch_int8_rows(const Int8RowsArgs& a, int xdt, bool swiglu, hipStream_t s) {
  if (xdt == 0) go_int8_t<half_t>(a, swiglu, s);
  else if (xdt == 1) go_int8_t<__bf16>(a, swiglu, s);
  else go_int8_t<float>(a, swiglu, s);
}

}  // namespace tq
