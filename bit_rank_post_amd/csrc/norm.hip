// Norms before and after a block, fused with its gate and residual scale.
//
//   forward   r1 = (mean(b^2) + eps)^-1/2,  p = w_post b r1   (p = b without w_post)
//             y  = x + alpha gate p                            (y = x without b)
//             r2 = (mean(y^2) + eps)^-1/2,  n = w_next y r2    with y as it is stored
//   backward  h  = w_next dn,  u = y r2:
//             dx = dy + r2 (h - u mean(h u)),   dw_next = sum_t dn u
//             c  = b r1,  e = alpha gate dx:
//             db = r1 (w_post e - c mean(w_post e c)),  dw_post = sum_t e c
//             dgate = alpha dx p, summed over the row for a gate per row
// All sums, statistics and weight gradients are held in f32; x + alpha gate p
// is rounded once, to the residual stream's type, and n and r2 follow from
// that rounded y, so that the backward pass (which reads y) and a norm of y
// alone agree with it.  dw are summed over rows by each workgroup in
// registers, then over workgroups in a fixed order: the same inputs give the
// same bits.
//
// Bound by memory: every input is read once and every output written once; a
// row stays in the registers of its threads (VPT vectors of 8 values each)
// between the reductions.  16384 x 4096 in bf16: forward 97 us, gradients 162
// us (158 and 7 for the join alone), 5.5 and 5.0 TB/s of what they must move (a
// large copy: 5.0).  One row of 4096: 4 us.  Rows above 8192 values take two
// vectors a thread in the gradients, which spill some registers: 4096 x 16384 in
// bf16 282 us.
#include "norm_ops.h"
#include "rows.h"

namespace tq {

__device__ __forceinline__ void load8w(const void* p, int dt, int at, float v[8]) {
  if (dt == 0) load8(reinterpret_cast<const half_t*>(p) + at, v);
  else if (dt == 1) load8(reinterpret_cast<const __bf16*>(p) + at, v);
  else load8(reinterpret_cast<const float*>(p) + at, v);
}

// Sum over the threads of a row: the workgroup, or with ROWS a wave (each wave
// then has a row of its own).  s: 16 floats; a caller that reduces twice
// passes two arrays.
template <bool ROWS>
__device__ __forceinline__ float row_sum(float v, float* s) {
  v = wave_sum(v);
  if constexpr (!ROWS) {
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    const int n = blockDim.x >> 6;
    v = 0.f;
    for (int i = 0; i < n; ++i) v += s[i];
  }
  return v;
}

template <typename S, typename A, bool ROWS, int VPT>
__global__ __launch_bounds__(ROWS ? 256 : 1024) void norm_forward_kernel(NormArgs a) {
  __shared__ float s_a[16], s_b[16];
  const int NTH = ROWS ? 64 : blockDim.x;       // threads of a row
  const long t = ROWS ? (long)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  const int tid = ROWS ? threadIdx.x & 63 : threadIdx.x;
  if (t >= a.T) return;
  const int nv = a.d >> 3;
  float y[VPT][8], b[VPT][8];
  const S* x = reinterpret_cast<const S*>(a.x) + t * a.ld_x;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = tid + i * NTH;
#pragma unroll
    for (int j = 0; j < 8; ++j) y[i][j] = b[i][j] = 0.f;
    if (c < nv) {
      load8(x + c * 8, y[i]);
      if (a.b != nullptr) load8(reinterpret_cast<const A*>(a.b) + t * a.ld_b + c * 8, b[i]);
    }
  }
  if (a.b != nullptr) {
    float r1 = 1.f;
    if (a.w_post != nullptr) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(b[i][j], b[i][j], ss);
      r1 = rsqrtf(row_sum<ROWS>(ss, s_a) / (float)a.d + a.eps);
      if (a.rstd_post != nullptr && tid == 0) a.rstd_post[t] = r1;
    }
    const float k = a.gate == 1 ? a.alpha * reinterpret_cast<const float*>(a.gate_p)[t * a.ld_gate] : a.alpha;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = tid + i * NTH;
      if (c >= nv) continue;
      float w[8], g[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = g[j] = 1.f;
      if (a.w_post != nullptr) load8w(a.w_post, a.wdt, c * 8, w);
      if (a.gate == 2) load8(reinterpret_cast<const A*>(a.gate_p) + t * a.ld_gate + c * 8, g);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        y[i][j] = (float)(S)__builtin_fmaf(k * g[j], b[i][j] * r1 * w[j], y[i][j]);
      store8(reinterpret_cast<S*>(a.y) + t * a.ld_y + c * 8, y[i]);
    }
  }
  if (a.n == nullptr) return;
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(y[i][j], y[i][j], ss);
  const float r2 = rsqrtf(row_sum<ROWS>(ss, s_b) / (float)a.d + a.eps);
  if (a.rstd_next != nullptr && tid == 0) a.rstd_next[t] = r2;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = tid + i * NTH;
    if (c >= nv) continue;
    float w[8];
    load8w(a.w_next, a.wdt, c * 8, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] *= y[i][j] * r2;
    store8(reinterpret_cast<A*>(a.n) + t * a.ld_n + c * 8, w);
  }
}

// Workgroup w takes rows w, w + nparts, ... (with ROWS: its waves rows 4w .. 4w+3,
// then 4 nparts further on)
template <typename S, typename A, bool ROWS, int VPT>
__global__ __launch_bounds__(ROWS ? 256 : 1024) void norm_backward_kernel(NormArgs a) {
  __shared__ float s_a[2][16], s_b[2][16];
  const int NTH = ROWS ? 64 : blockDim.x;
  const int part = blockIdx.x;
  const int tid = ROWS ? threadIdx.x & 63 : threadIdx.x;
  const long first = ROWS ? (long)part * 4 + (threadIdx.x >> 6) : part;
  const long stride = ROWS ? (long)a.nparts * 4 : a.nparts;
  const int nv = a.d >> 3;
  const float inv_d = 1.f / (float)a.d;
  const bool has_b = a.b != nullptr, has_post = a.w_post != nullptr, has_next = a.dn != nullptr;
  float gp[VPT][8], gn[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) gp[i][j] = gn[i][j] = 0.f;
  // With one vector a thread, a row's inputs are requested while the row before
  // it is worked on (two vectors do not fit 128 registers so).
  constexpr bool AHEAD = VPT == 1;
  Raw8<S> q_dy[VPT], q_y[VPT];
  Raw8<A> q_dn[VPT], q_b[VPT];
  auto request = [&](long t) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = tid + i * NTH;
      if (c >= nv) continue;
      if (a.dy != nullptr) q_dy[i].load(reinterpret_cast<const S*>(a.dy) + t * a.ld_dy + c * 8);
      if (has_next) {
        q_y[i].load(reinterpret_cast<const S*>(a.y) + t * a.ld_y + c * 8);
        q_dn[i].load(reinterpret_cast<const A*>(a.dn) + t * a.ld_dn + c * 8);
      }
      if (has_b) q_b[i].load(reinterpret_cast<const A*>(a.b) + t * a.ld_b + c * 8);
    }
  };
  int ph = 0;
  if (AHEAD && first < a.T) request(first);
  for (long t = first; t < a.T; t += stride, ph ^= 1) {
    if (!AHEAD) request(t);
    float u[VPT][8], dx[VPT][8];
    Raw8<S> y_[VPT];
    Raw8<A> dn_[VPT], b_[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = tid + i * NTH;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u[i][j] = 0.f;
        dx[i][j] = c < nv && a.dy != nullptr ? q_dy[i].get(j) : 0.f;
      }
      y_[i] = q_y[i];
      dn_[i] = q_dn[i];
      b_[i] = q_b[i];
    }
    if (AHEAD && t + stride < a.T) request(t + stride);
    if (has_next) {
      const float r2 = a.rstd_next[t];
      float h[VPT][8];
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = tid + i * NTH;
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = 0.f;
        if (c >= nv) continue;
        float w[8];
        load8w(a.w_next, a.wdt, c * 8, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          u[i][j] = y_[i].get(j) * r2;
          h[i][j] = dn_[i].get(j);
          gn[i][j] = __builtin_fmaf(h[i][j], u[i][j], gn[i][j]);
          h[i][j] *= w[j];
          dot = __builtin_fmaf(h[i][j], u[i][j], dot);
        }
      }
      const float mean = row_sum<ROWS>(dot, s_a[ph]) * inv_d;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) dx[i][j] += r2 * (h[i][j] - u[i][j] * mean);
    }
    if (a.dx != nullptr) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = tid + i * NTH;
        if (c < nv) store8(reinterpret_cast<S*>(a.dx) + t * a.ld_dx + c * 8, dx[i]);
      }
    }
    if (!has_b) continue;
    // u: c = b r1;  dx: w_post e
    const float r1 = has_post ? a.rstd_post[t] : 1.f;
    const float gt = a.gate == 1 ? reinterpret_cast<const float*>(a.gate_p)[t * a.ld_gate] : 1.f;
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = tid + i * NTH;
      if (c >= nv) continue;
      float w[8], g[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = g[j] = 1.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) u[i][j] = b_[i].get(j);
      if (has_post) load8w(a.w_post, a.wdt, c * 8, w);
      if (a.gate == 2) {
        load8(reinterpret_cast<const A*>(a.gate_p) + t * a.ld_gate + c * 8, g);
        if (a.dgate != nullptr) {
          float dg[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) dg[j] = a.alpha * dx[i][j] * (u[i][j] * r1 * w[j]);
          store8(reinterpret_cast<A*>(a.dgate) + t * a.ld_dgate + c * 8, dg);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u[i][j] *= r1;
        const float e = a.alpha * g[j] * dx[i][j];      // without a gate per row
        gp[i][j] = __builtin_fmaf(gt * e, u[i][j], gp[i][j]);
        dx[i][j] = w[j] * e;
        dot = __builtin_fmaf(dx[i][j], u[i][j], dot);
      }
    }
    float sum = 0.f;
    if (has_post || a.gate == 1) sum = row_sum<ROWS>(dot, s_b[ph]);
    if (a.gate == 1 && a.dgate != nullptr && tid == 0)
      reinterpret_cast<float*>(a.dgate)[t * a.ld_dgate] = sum;
    if (a.db == nullptr) continue;
    const float mean = has_post ? sum * inv_d : 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = tid + i * NTH;
      if (c >= nv) continue;
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = r1 * gt * (dx[i][j] - u[i][j] * mean);
      store8(reinterpret_cast<A*>(a.db) + t * a.ld_db + c * 8, o);
    }
  }
  if constexpr (ROWS) {
    // the four waves' sums first, in wave order
    __shared__ float s_w[3][2][8][64];
    const int wave = threadIdx.x >> 6;
    if (wave > 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s_w[wave - 1][0][j][tid] = gp[0][j];
        s_w[wave - 1][1][j][tid] = gn[0][j];
      }
    }
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int w = 0; w < 3; ++w)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        gp[0][j] += s_w[w][0][j][tid];
        gn[0][j] += s_w[w][1][j][tid];
      }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = tid + i * NTH;
    if (c >= nv) continue;
    // (one part is the whole sum; dw is 4-byte aligned only)
    if (a.nparts == 1) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (a.dw_post != nullptr) a.dw_post[c * 8 + j] = gp[i][j];
        if (a.dw_next != nullptr) a.dw_next[c * 8 + j] = gn[i][j];
      }
      continue;
    }
    if (a.dw_post != nullptr) store8(a.part + (size_t)part * a.d + c * 8, gp[i]);
    if (a.dw_next != nullptr) store8(a.part + (size_t)(a.nparts + part) * a.d + c * 8, gn[i]);
  }
}

// dw[c] = sum over the parts, in a fixed order: 32 columns a workgroup, the
// parts in 32 interleaved runs of four sums each, joined in LDS
__global__ __launch_bounds__(1024) void norm_join_kernel(NormArgs a) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float* dw = blockIdx.y == 0 ? a.dw_post : a.dw_next;
  if (dw == nullptr) return;
  const float* p = a.part + (blockIdx.y == 0 ? 0 : (size_t)a.nparts * a.d);
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  if (c < a.d) {
    for (int i = run; i < a.nparts; i += 128) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i + 32 * k < a.nparts) v[k] += p[(size_t)(i + 32 * k) * a.d + c];
    }
  }
  s[run][lane] = (v[0] + v[1]) + (v[2] + v[3]);
  __syncthreads();
  if (run == 0 && c < a.d) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += s[i][lane];
    dw[c] = t;
  }
}

// Threads of a row of nv vectors with vpt a thread, in whole waves (5632
// values: 704 threads, all at work, or 352 with two vectors).
static int row_threads(int nv, int vpt) { return ((nv + vpt - 1) / vpt + 63) / 64 * 64; }

// Rows up to 512 values are a wave's, longer ones a workgroup's with two
// vectors a thread (16384 x 4096 in bf16: 98 us; one vector 98, four 111; at
// 5632: 106, 114, 117).
template <typename S, typename A>
static void forward_go(const NormArgs& a, hipStream_t s) {
  const int nv = a.d >> 3;
  if (nv <= 64)
    hipLaunchKernelGGL((norm_forward_kernel<S, A, true, 1>), dim3((a.T + 3) / 4), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((norm_forward_kernel<S, A, false, 2>), dim3(a.T), dim3(row_threads(nv, 2)), 0, s, a);
}

// Rows are dealt to as many workgroups as run at once, 1024 threads on each of
// 256 CUs: more only add partial sums (16384 x 4096 in bf16: 256
// workgroups of 512 threads 202 us, 512 166 us, 1024 179 us).
int norm_parts(int T, int d) {
  const int nv = d >> 3;
  const int most = nv <= 64 ? 1024 : 256 * (1024 / row_threads(nv, nv <= 1024 ? 1 : 2));
  const int want = nv <= 64 ? (T + 3) / 4 : T;
  return want < most ? (want > 0 ? want : 1) : most;
}

template <typename S, typename A>
static void backward_go(const NormArgs& a, hipStream_t s) {
  const int nv = a.d >> 3;
  if (nv <= 64)
    hipLaunchKernelGGL((norm_backward_kernel<S, A, true, 1>), dim3(a.nparts), dim3(256), 0, s, a);
  else if (nv <= 1024)
    hipLaunchKernelGGL((norm_backward_kernel<S, A, false, 1>), dim3(a.nparts), dim3(row_threads(nv, 1)), 0, s, a);
  else
    hipLaunchKernelGGL((norm_backward_kernel<S, A, false, 2>), dim3(a.nparts), dim3(row_threads(nv, 2)), 0, s, a);
  if (a.nparts > 1 && (a.dw_post != nullptr || a.dw_next != nullptr))
    hipLaunchKernelGGL(norm_join_kernel, dim3((a.d + 31) / 32, 2), dim3(1024), 0, s, a);
}

template <bool FWD, typename S>
static void pick(const NormArgs& a, int adt, hipStream_t s) {
  if (adt == 0) FWD ? forward_go<S, half_t>(a, s) : backward_go<S, half_t>(a, s);
  else if (adt == 1) FWD ? forward_go<S, __bf16>(a, s) : backward_go<S, __bf16>(a, s);
  else FWD ? forward_go<S, float>(a, s) : backward_go<S, float>(a, s);
}

void launch_norm_forward(const NormArgs& a, int sdt, int adt, hipStream_t s) {
  if (a.T <= 0) return;
  if (sdt == 0) pick<true, half_t>(a, adt, s);
  else if (sdt == 1) pick<true, __bf16>(a, adt, s);
  else pick<true, float>(a, adt, s);
}

void launch_norm_backward(const NormArgs& a, int sdt, int adt, hipStream_t s) {
  if (sdt == 0) pick<false, half_t>(a, adt, s);
  else if (sdt == 1) pick<false, __bf16>(a, adt, s);
  else pick<false, float>(a, adt, s);
}

}  // namespace tq
