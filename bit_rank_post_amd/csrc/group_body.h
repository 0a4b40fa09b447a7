// Device helpers shared by the kernels of the grouped products: operand types
// and matrix instructions, the rows of a group, work items.
#pragma once
#include "group_gemm.h"
#include "tq_device.h"

#include <type_traits>

namespace tq {

struct e4m3_t { uint8_t v; };
struct i8_t { int8_t v; };

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

template <typename T> struct Elem { static constexpr int BYTES = 2; };
template <> struct Elem<e4m3_t> { static constexpr int BYTES = 1; };
template <> struct Elem<i8_t> { static constexpr int BYTES = 1; };

// sums of products: f32, and of 8-bit integers exact 32-bit integers
template <typename T> struct Sum { typedef f32x4 type; };
template <> struct Sum<i8_t> { typedef i32x4 type; };

// 16 elements of k for 16 rows of the A or B operand of one stage half: the
// 16 bytes of each lane.  16-bit: the operand of one 16x16x32 MFMA; 8-bit
// integers: of one 16x16x64 MFMA; e4m3: two of them make the operand of one
// 16x16x128 MFMA (which bytes of k a lane holds is free, as long as A and B
// agree).
template <typename T>
__device__ __forceinline__ typename Sum<T>::type mfma_half(u32x4 a, u32x4 b, typename Sum<T>::type c) {
  if constexpr (std::is_same<T, i8_t>::value) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
  } else {
    typedef typename Vec8<T>::type V8;
    return mfma16(__builtin_bit_cast(V8, a), __builtin_bit_cast(V8, b), c);
  }
}

// The 8-bit matrix instructions add 8 neighbouring products at a time, each
// cut at 2^-13 of the power of two below the largest of the 8 (measured: a
// product 2^-14 of its neighbour is lost, 2^-13 is kept, across eights all is
// kept in f32; the 16x16x32 form, at half the rate, cuts the same).  That is
// the one rounding below 32 bits here: about 2^-16 of a result of random
// values, against 2^-9 of its rounding to bf16; the way around it, exact
// conversion to f16 and 16-bit MFMA, runs at half the rate and needs more
// registers than a 256 x 256 tile leaves.  A product in 8 bits is asked for
// its rate, and at 16-bit outputs its error against 64 bits is that of f32 sums.
__device__ __forceinline__ f32x4 mfma_e4m3(u32x4 a0, u32x4 a1, u32x4 b0, u32x4 b1) {
  i32x8 a, b;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = (int)a0[i];
    a[4 + i] = (int)a1[i];
    b[i] = (int)b0[i];
    b[4 + i] = (int)b1[i];
  }
  // formats 0, 0: e4m3; scales 2^0
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0,
                                                          0x7F7F7F7F, 0, 0x7F7F7F7F);
}

// Rows of group g: [lo, hi), clamped so that any offsets stay inside 0 .. rows.
__device__ __forceinline__ void group_span(const GroupArgs& a, int g, int* lo, int* hi) {
  if (a.off == nullptr) {
    *lo = 0;
    *hi = a.rows;
    return;
  }
  const int l = min(max(a.off[g], 0), a.rows);
  *lo = l;
  *hi = min(max(a.off[g + 1], l), a.rows);
}

// Row of x for position r of the grouped rows, or -1 (a row of zeros).
__device__ __forceinline__ int source_row(const GroupArgs& a, int v) {
  if (v < 0) return -1;
  const int q = a.div_shift < 0 ? v : (int)(__umulhi((uint32_t)v, a.div_mul) >> a.div_shift);
  return q < a.x_rows ? q : -1;
}

// Tiles of NT rows over all groups (each wave on its own, from registers).
template <int NT>
__device__ __forceinline__ int count_row_tiles(const GroupArgs& a, int lane) {
  int n = 0;
  for (int g = lane; g < a.groups; g += 64) {
    int lo, hi;
    group_span(a, g, &lo, &hi);
    n += (hi - lo + NT - 1) / NT;
  }
  return __builtin_amdgcn_readfirstlane(wave_sum_i(n));
}

// Group and first row of row tile `tile` (tile < count_row_tiles).
template <int NT>
__device__ __forceinline__ void find_row_tile(const GroupArgs& a, int lane, int tile, int* g, int* row0,
                                              int* nrow) {
  int before = 0;
  for (int g0 = 0; g0 < a.groups; g0 += 64) {
    int lo = 0, hi = 0;
    if (g0 + lane < a.groups) group_span(a, g0 + lane, &lo, &hi);
    const int inc = before + wave_incl_scan_i((hi - lo + NT - 1) / NT, lane);
    const uint64_t past = __ballot(inc > tile);
    if (past != 0) {
      const int l = __ffsll((unsigned long long)past) - 1;
      const int tiles = (hi - lo + NT - 1) / NT;
      const int first = __shfl(inc - tiles, l, 64);
      const int glo = __shfl(lo, l, 64), ghi = __shfl(hi, l, 64);
      *g = __builtin_amdgcn_readfirstlane(g0 + l);
      // (offsets that break the rules may count more tiles than int holds)
      if (tile < first || tile - first >= __shfl(tiles, l, 64)) break;
      const int r0 = glo + (tile - first) * NT;
      *row0 = __builtin_amdgcn_readfirstlane(r0);
      *nrow = __builtin_amdgcn_readfirstlane(min(NT, ghi - r0));
      return;
    }
    before = __shfl(inc, 63, 64);
  }
  *g = 0;
  *row0 = 0;
  *nrow = 0;
}

// Work item of this workgroup: XCD x (workgroups x, x + 8, ...) takes one run
// of consecutive items; inside a run, bands of 8 row tiles go over all m
// tiles, so that the workgroups running together on an XCD share few rows of
// each operand through its L2.
__device__ __forceinline__ bool take_item(int ntile, int mtile, int* n, int* m) {
  const int total = ntile * mtile;
  const int per = (total + 7) >> 3;
  const int li = blockIdx.x >> 3;
  const int item = (blockIdx.x & 7) * per + li;
  if (li >= per || item >= total) return false;
  const int band = item / (8 * mtile), rem = item - band * (8 * mtile);
  const int width = min(8, ntile - band * 8);
  *m = rem / width;
  *n = band * 8 + rem % width;
  return true;
}

// The tile of this workgroup: m tile, group, first row and rows.  Up to 64
// groups, their spans are read once and stay in the lanes.
template <int NT>
__device__ __forceinline__ bool locate_row_tile(const GroupArgs& a, int lane, int mtile, int* m, int* g,
                                                int* row0, int* nrow) {
  int it;
  if (a.groups > 64) {
    if (!take_item(count_row_tiles<NT>(a, lane), mtile, &it, m)) return false;
    find_row_tile<NT>(a, lane, it, g, row0, nrow);
  } else {
    int lo = 0, hi = 0;
    if (lane < a.groups) group_span(a, lane, &lo, &hi);
    const int tiles = (hi - lo + NT - 1) / NT;
    const int inc = wave_incl_scan_i(tiles, lane);
    if (!take_item(__builtin_amdgcn_readlane(inc, 63), mtile, &it, m)) return false;
    const uint64_t past = __ballot(inc > it);
    const int l = past != 0 ? __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)past) - 1) : 0;
    const int first = __builtin_amdgcn_readlane(inc - tiles, l);
    const int glo = __builtin_amdgcn_readlane(lo, l), ghi = __builtin_amdgcn_readlane(hi, l);
    // (offsets that break the rules may count more tiles than int holds)
    if (past == 0 || it < first || it - first >= __builtin_amdgcn_readlane(tiles, l)) return false;
    *g = l;
    *row0 = glo + (it - first) * NT;
    *nrow = min(NT, ghi - *row0);
  }
  *g = __builtin_amdgcn_readfirstlane(*g);
  *row0 = __builtin_amdgcn_readfirstlane(*row0);
  *nrow = __builtin_amdgcn_readfirstlane(*nrow);
  *m = __builtin_amdgcn_readfirstlane(*m);
  return *nrow > 0;
}

// Products of 8-bit integers: scales of the four outputs o .. o+3 of group g
// (outputs past the last: 0), and of a row of x (-1: a row of zeros).
__device__ __forceinline__ f32x4 output_scales(const GroupArgs& a, int g, int o) {
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  const float* p = a.ws + (size_t)g * a.d_out + o;
  if (a.vec_scales) {
    if (o < a.d_out) s = *reinterpret_cast<const f32x4*>(p);
    return s;
  }
#pragma unroll
  for (int v = 0; v < 4; ++v)
    if (o + v < a.d_out) s[v] = p[v];
  return s;
}
__device__ __forceinline__ float row_scale(const GroupArgs& a, int row) { return row >= 0 ? a.xs[row] : 0.f; }

// The sums of four outputs of one row as they are stored.  8-bit integers:
// fl32(fl32(fl32(sum) w_scale) x_scale), three roundings in all; the sum is an
// integer of 1 at least or 0, so its product with a normal scale is one.
__device__ __forceinline__ f32x4 finish(const f32x4& v, const f32x4&, float) { return v; }
__device__ __forceinline__ f32x4 finish(const i32x4& v, const f32x4& ws, float xs) {
  f32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = (float)v[i] * ws[i] * xs;
  return r;
}

// Four neighbouring outputs at `at`, `left` of which exist.
__device__ __forceinline__ void store4(const GroupArgs& a, size_t at, const f32x4& v, int left) {
  if (a.out_dtype == 2) {
    float* p = reinterpret_cast<float*>(a.out) + at;
    if (a.vec_out && left >= 4) *reinterpret_cast<f32x4*>(p) = v;
    else
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) p[i] = v[i];
    return;
  }
  uint16_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float f = v[i];
    h[i] = a.out_dtype == 0 ? __builtin_bit_cast(uint16_t, (half_t)f) : __builtin_bit_cast(uint16_t, (__bf16)f);
  }
  uint16_t* p = reinterpret_cast<uint16_t*>(a.out) + at;
  if (a.vec_out && left >= 4)
    *reinterpret_cast<u32x2*>(p) = u32x2{h[0] | ((uint32_t)h[1] << 16), h[2] | ((uint32_t)h[3] << 16)};
  else
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) p[i] = h[i];
}

}  // namespace tq
