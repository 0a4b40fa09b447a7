// Grouped products of few rows per group: y[r][o] = sum_i W_g[o][i] x[s(r)][i]
// for decode batches, 16-bit operands or e4m3 with block scales.
//
// Bound by the weights' bytes: each weight meets at most 16 rows.  So weights
// go from memory straight to the registers of the one wave that uses them, in
// the fragment layout of the MFMA (16 outputs x 16 bytes of k a lane, 128
// bytes of each row a step), without LDS.  A workgroup takes 16 outputs of one
// group's tile of 16 rows; its waves share k in interleaved runs of D steps
// (each requests the D steps of its next run before it multiplies the last),
// and their sums are added in LDS in wave order.
#include "group_body.h"

namespace tq {

// A run is D steps of 128 bytes of k: 2 D fragment loads of W and of x each.
template <typename T, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void group_rows_kernel(GroupArgs a) {
  constexpr bool F8 = sizeof(T) == 1;
  constexpr int ES = Elem<T>::BYTES, KS = 128 / ES, D = 2;
  __shared__ f32x4 s_sum[WAVES > 1 ? WAVES - 1 : 1][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, lg = lane >> 4;

  int g, row0, nrow, m;
  const int mtile = (a.d_out + 15) >> 4;
  if (!locate_row_tile<16>(a, lane, mtile, &m, &g, &row0, &nrow)) return;
  const int m0 = m * 16;

  const int K = a.d_in, nstep = (K + KS - 1) / KS, nrun = (nstep + D - 1) / D;
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(
      reinterpret_cast<const char*>(a.w) + ((size_t)g * a.d_out + m0) * a.d_in * ES, (uint32_t)OOB);
  const uint32_t vw = m0 + l16 < a.d_out ? (uint32_t)l16 * a.d_in * ES + lg * 16u : OOB;
  int row = l16 < nrow ? l16 : -1;
  if (row >= 0 && a.src != nullptr) row = source_row(a, a.src[row0 + l16]);
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(
      reinterpret_cast<const char*>(a.x) + (a.src != nullptr ? 0 : (size_t)row0 * a.ldx * ES), (uint32_t)OOB);
  const uint32_t vx = row >= 0 ? (uint32_t)row * (uint32_t)(a.ldx * ES) + lg * 16u : OOB;
  // scales of this lane's row and of the outputs' block
  const int nkb = (K + 127) >> 7;
  __amdgpu_buffer_rsrc_t rs;
  uint32_t vs = OOB;
  const int* wsp = nullptr;
  if constexpr (F8) {
    rs = make_rsrc(a.src != nullptr ? a.xs : a.xs + (size_t)row0 * nkb, (uint32_t)OOB);
    if (row >= 0) vs = (uint32_t)row * nkb * 4u;
    wsp = reinterpret_cast<const int*>(a.ws) + ((size_t)g * ((a.d_out + 127) >> 7) + (m0 >> 7)) * nkb;
  }

  struct Run {
    u32x4 w[D][2], x[D][2];
    float s[D];
  };
  auto fetch = [&](int run, Run& r) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int st = run * D + d;
      const bool live = st < nstep;
      const uint32_t so = live ? st * 128u : 0u;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // bytes 64 h + 16 lg of the step's 128: past the row, nothing is read
        const bool ok = live && st * 128 + h * 64 + lg * 16 < K * ES;
        r.w[d][h] = bload128(rw, ok ? vw + h * 64u : OOB, so);
        r.x[d][h] = bload128(rx, ok ? vx + h * 64u : OOB, so);
      }
      if constexpr (F8)
        r.s[d] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, live ? vs : OOB, live ? st * 4u : 0u, 0)) *
                 __builtin_bit_cast(float, sload(wsp, live ? st : 0));
    }
  };
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](const Run& r) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if constexpr (F8) {
        const f32x4 p = mfma_e4m3(r.w[d][0], r.w[d][1], r.x[d][0], r.x[d][1]);
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[v] = __builtin_fmaf(p[v], r.s[d], acc[v]);
      } else {
        acc = mfma_half<T>(r.w[d][0], r.x[d][0], acc);
        acc = mfma_half<T>(r.w[d][1], r.x[d][1], acc);
      }
    }
  };
  Run r0, r1;
  int run = wave;
  if (run < nrun) fetch(run, r0);
  for (; run < nrun; run += 2 * WAVES) {
    if (run + WAVES < nrun) fetch(run + WAVES, r1);
    multiply(r0);
    if (run + WAVES >= nrun) break;
    if (run + 2 * WAVES < nrun) fetch(run + 2 * WAVES, r0);
    multiply(r1);
  }

  if constexpr (WAVES > 1) {
    if (wave > 0) s_sum[wave - 1][lane] = acc;
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int i = 0; i < WAVES - 1; ++i) acc += s_sum[i][lane];
  }
  if (l16 >= nrow) return;
  const int left = a.d_out - (m0 + 4 * lg);
  const size_t at = (size_t)(row0 + l16) * a.ldo + m0 + 4 * lg;
  if (a.out_dtype == 2) {
    float* p = reinterpret_cast<float*>(a.out) + at;
    if (a.vec_out && left >= 4) *reinterpret_cast<f32x4*>(p) = acc;
    else
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) p[i] = acc[i];
  } else {
    uint16_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float v = acc[i];
      h[i] = a.out_dtype == 0 ? __builtin_bit_cast(uint16_t, (half_t)v) : __builtin_bit_cast(uint16_t, (__bf16)v);
    }
    uint16_t* p = reinterpret_cast<uint16_t*>(a.out) + at;
    if (a.vec_out && left >= 4)
      *reinterpret_cast<u32x2*>(p) = u32x2{h[0] | ((uint32_t)h[1] << 16), h[2] | ((uint32_t)h[3] << 16)};
    else
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) p[i] = h[i];
  }
}

long group_rows_grid(const GroupArgs& a) {
  const long mtile = (a.d_out + 15) / 16;
  const long ntile = a.groups == 1 ? ((long)a.rows + 15) / 16
                                   : (long)a.rows / 16 + (a.groups < a.rows ? a.groups : a.rows);
  return (mtile * ntile + 7) / 8 * 8;
}

template <typename T>
static void go_rows(const GroupArgs& a, long grid, hipStream_t s) {
  // At least about 3000 waves when k is long enough to give each two runs
  // (256 bytes of k): 4 waves a workgroup from 768 workgroups up (60 experts of
  // 2048 -> 1408, 32 tokens top-4: 56 us; 8 waves: 72 us), 8 or 16 below.
  const int runs = (a.d_in * Elem<T>::BYTES + 255) / 256;
  if (grid < 384 && runs >= 32)
    hipLaunchKernelGGL((group_rows_kernel<T, 16>), dim3((unsigned)grid), dim3(1024), 0, s, a);
  else if (grid < 768 && runs >= 16)
    hipLaunchKernelGGL((group_rows_kernel<T, 8>), dim3((unsigned)grid), dim3(512), 0, s, a);
  else
    hipLaunchKernelGGL((group_rows_kernel<T, 4>), dim3((unsigned)grid), dim3(256), 0, s, a);
}

void launch_group_rows(const GroupArgs& a, GroupType type, hipStream_t s) {
  const long grid = group_rows_grid(a);
  if (grid <= 0) return;
  if (type == GROUP_E4M3) go_rows<e4m3_t>(a, grid, s);
  else if (type == GROUP_F16) go_rows<half_t>(a, grid, s);
  else go_rows<__bf16>(a, grid, s);
}

}  // namespace tq
