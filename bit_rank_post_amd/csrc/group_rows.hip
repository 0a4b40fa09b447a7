// Grouped products y[r][o] = sum_i W_g[o][i] x[s(r)][i] without LDS staging, for
// decode batches and for products of few tiles; 16-bit operands or e4m3 with
// block scales.
//
// Bound by the weights' bytes: each weight meets few rows.  So weights go from
// memory straight to the registers of the one wave that uses them, in the
// fragment layout of the MFMA (16 outputs x 16 bytes of k a lane, 128 bytes of
// each row a step).  A workgroup takes 16 x 16 or 32 x 32 outputs x rows of one
// group; its waves share k in interleaved runs of D steps (each requests its
// next run before it multiplies the last), and their sums are added in LDS in
// wave order.  60 experts of 2048 -> 1408, 32 tokens top-4, f16: 57 us, 5.4 TB/s
// of the weights of the 53 experts that have rows (a plain read of a larger
// buffer: 5.5); one row through 4096 -> 14336 in e4m3: 15 us, 4 TB/s, where the
// start and the last loads count.
#include "group_body.h"

namespace tq {

// A workgroup takes 16 FM outputs x 16 FN rows; a run is D steps of 128 bytes
// of k: 2 D FM fragment loads of W and 2 D FN of x.
template <typename T, int WAVES, int FM, int FN, int D>
__global__ __launch_bounds__(64 * WAVES) void group_rows_kernel(GroupArgs a) {
  constexpr bool F8 = sizeof(T) == 1;
  constexpr int ES = Elem<T>::BYTES, KS = 128 / ES;
  __shared__ f32x4 s_sum[WAVES > 1 ? WAVES - 1 : 1][FM * FN][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, lg = lane >> 4;

  int g, row0, nrow, m;
  const int mtile = (a.d_out + 16 * FM - 1) / (16 * FM);
  if (!locate_row_tile<16 * FN>(a, lane, mtile, &m, &g, &row0, &nrow)) return;
  const int m0 = m * 16 * FM;

  const int K = a.d_in, nstep = (K + KS - 1) / KS, nrun = (nstep + D - 1) / D;
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(
      reinterpret_cast<const char*>(a.w) + ((size_t)g * a.d_out + m0) * a.d_in * ES, (uint32_t)OOB);
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(
      reinterpret_cast<const char*>(a.x) + (a.src != nullptr ? 0 : (size_t)row0 * a.ldx * ES), (uint32_t)OOB);
  uint32_t vw[FM], vx[FN], vs[FN];
  const int nkb = (K + 127) >> 7;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int o = 16 * i + l16;
    vw[i] = m0 + o < a.d_out ? (uint32_t)o * a.d_in * ES + lg * 16u : OOB;
  }
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int r = 16 * j + l16;
    int row = r < nrow ? r : -1;
    if (row >= 0 && a.src != nullptr) row = source_row(a, a.src[row0 + r]);
    vx[j] = row >= 0 ? (uint32_t)row * (uint32_t)(a.ldx * ES) + lg * 16u : OOB;
    vs[j] = row >= 0 ? (uint32_t)row * nkb * 4u : OOB;
  }
  // scales of this lane's rows and of the outputs' block
  __amdgpu_buffer_rsrc_t rs;
  const int* wsp = nullptr;
  if constexpr (F8) {
    static_assert(128 % (16 * FM) == 0, "outputs inside a scale block");
    rs = make_rsrc(a.src != nullptr ? a.xs : a.xs + (size_t)row0 * nkb, (uint32_t)OOB);
    wsp = reinterpret_cast<const int*>(a.ws) + ((size_t)g * ((a.d_out + 127) >> 7) + (m0 >> 7)) * nkb;
  }

  struct Run {
    u32x4 w[D][FM][2], x[D][FN][2];
    float s[D][FN];
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
#pragma unroll
        for (int i = 0; i < FM; ++i) r.w[d][i][h] = bload128(rw, ok ? vw[i] + h * 64u : OOB, so);
#pragma unroll
        for (int j = 0; j < FN; ++j) r.x[d][j][h] = bload128(rx, ok ? vx[j] + h * 64u : OOB, so);
      }
      if constexpr (F8) {
        const float w = live ? __builtin_bit_cast(float, sload(wsp, st)) : 0.f;
#pragma unroll
        for (int j = 0; j < FN; ++j)
          r.s[d][j] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                                                    rs, live ? vs[j] : OOB, live ? st * 4u : 0u, 0)) * w;
      }
    }
  };
  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](const Run& r) {
#pragma unroll
    for (int d = 0; d < D; ++d)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          if constexpr (F8) {
            const f32x4 p = mfma_e4m3(r.w[d][i][0], r.w[d][i][1], r.x[d][j][0], r.x[d][j][1]);
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[i][j][v] = __builtin_fmaf(p[v], r.s[d][j], acc[i][j][v]);
          } else {
            acc[i][j] = mfma_half<T>(r.w[d][i][0], r.x[d][j][0], acc[i][j]);
            acc[i][j] = mfma_half<T>(r.w[d][i][1], r.x[d][j][1], acc[i][j]);
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

  // the waves' sums, added in wave order; wave 0 stores
  if (wave > 0) {
#pragma unroll
    for (int f = 0; f < FM * FN; ++f) s_sum[wave - 1][f][lane] = acc[f / FN][f % FN];
  }
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int f = 0; f < FM * FN; ++f) {
    f32x4 v = acc[f / FN][f % FN];
#pragma unroll
    for (int i = 0; i < WAVES - 1; ++i) v += s_sum[i][f][lane];
    const int r = 16 * (f % FN) + l16, o = m0 + 16 * (f / FN) + 4 * lg;
    if (r < nrow) store4(a, (size_t)(row0 + r) * a.ldo + o, v, a.d_out - o);
  }
}

void group_rows_shape(GroupRows r, int* mt, int* nt) {
  *mt = *nt = r == ROWS_16x16 ? 16 : 32;
}

long group_rows_grid(const GroupArgs& a, GroupRows shape) {
  int mt, nt;
  group_rows_shape(shape, &mt, &nt);
  const long mtile = (a.d_out + mt - 1) / mt;
  const long ntile = a.groups == 1 ? ((long)a.rows + nt - 1) / nt
                                   : (long)a.rows / nt + (a.groups < a.rows ? a.groups : a.rows);
  return (mtile * ntile + 7) / 8 * 8;
}

template <typename T, int WAVES, int F, int D>
static void go(const GroupArgs& a, long grid, hipStream_t s) {
  hipLaunchKernelGGL((group_rows_kernel<T, WAVES, F, F, D>), dim3((unsigned)grid), dim3(64 * WAVES), 0, s, a);
}

template <typename T>
static void go_rows(const GroupArgs& a, GroupRows shape, long grid, hipStream_t s) {
  // At least about 3000 waves when k is long enough to give each two runs
  // (256 bytes of k): 4 waves a workgroup from 768 workgroups up (60 experts of
  // 2048 -> 1408, 32 tokens top-4: 56 us; 8 waves: 72 us), 8 or 16 below.
  const int runs = (a.d_in * Elem<T>::BYTES + 255) / 256;
  if (shape == ROWS_32x32) {
    if (runs >= 16) go<T, 8, 2, 2>(a, grid, s);
    else go<T, 4, 2, 2>(a, grid, s);
  } else if (grid < 384 && runs >= 32) {
    go<T, 16, 1, 2>(a, grid, s);
  } else if (grid < 768 && runs >= 16) {
    go<T, 8, 1, 2>(a, grid, s);
  } else {
    go<T, 4, 1, 2>(a, grid, s);
  }
}

void launch_group_rows(const GroupArgs& a, GroupType type, GroupRows shape, hipStream_t s) {
  const long grid = group_rows_grid(a, shape);
  if (grid <= 0) return;
  if (type == GROUP_E4M3) go_rows<e4m3_t>(a, shape, grid, s);
  else if (type == GROUP_F16) go_rows<half_t>(a, shape, grid, s);
  else go_rows<__bf16>(a, shape, grid, s);
}

}  // namespace tq
