// The sum over a token's slots after the last product of a layer of experts,
// and its gradient.
//
//   y[t]  = add[t] + sum_j w[t][j] z[inv[t k + j]]         (w = 1 without weights)
//   dz[inv[t k + j]] = w[t][j] dy[t],  dw[t][j] = dy[t] . z[inv[t k + j]]
// A slot whose inv lies outside 0 .. rows - 1 was dropped: it adds nothing and
// its dw is 0.  Sums run in f32, the slots in order, and are rounded once; the
// sum of a dot product has one fixed order too, so the same inputs give the
// same bits.  Without weights, y of the rows' gradients is the gradient of
// gathering them from x.
//
// Bound by memory.  Sum: a thread takes 8 values of a token and requests them
// from four slots at a time: 16384 tokens of two slots of 4096 values and an
// addend, bf16: 98 us, 5.5 TB/s of what it must move (a large copy: 4.9); 32 tokens of
// four of 2048: 3 us.  Gradient: of few tokens a wave takes a slot, so that they
// still make many waves, and the waves of one token find its dy in the cache; from
// 4096 tokens a wave takes a token, keeps dy in registers and requests the next
// slot's z ahead (4160 tokens of six of 2048 bf16: 50 us, 4.4 TB/s).  Both, us, a wave a
// slot and a wave a token: 1024 tokens of six slots of 2048 11.3, 13.1, of eight of 4096
// 35.0, 36.3; 2048: 25.9, 25.6 and 66.1, 62.5; 4000: 51.6, 46.3 and 119, 129; 4160: 55.0, 50.3
// and 127, 132; of four of 2048 4000 tokens 38.0, 33.1, 8192 70.2, 66.0; 16384 of two of
// 4096 139, 139.  (Rows of 2048 would take a wave a token from 2048 tokens on; the border
// is where it is not the slower way by more than 4 % for any of these.)
#include "layer_ops.h"
#include "rows.h"

namespace tq {

__device__ __forceinline__ int slot_row(const SlotSumArgs& a, int v) { return v >= 0 && v < a.rows ? v : -1; }

template <typename Z, typename Y>
__global__ __launch_bounds__(256) void slot_sum_kernel(SlotSumArgs a, int t0, uint32_t items, uint32_t nv) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= items) return;
  const uint32_t r = i / nv;
  const long t = (long)t0 + r;
  const int c = (int)(i - r * nv) * 8;
  const int* inv = a.inv + t * a.topk;
  const float* w = a.w == nullptr ? nullptr : a.w + t * a.topk;
  const Z* z = reinterpret_cast<const Z*>(a.z) + c;
  float y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = 0.f;
  for (int j0 = 0; j0 < a.topk; j0 += 4) {
    Raw8<Z> v[4];
    float g[4];
    int row[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) row[q] = j0 + q < a.topk ? slot_row(a, inv[j0 + q]) : -1;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (row[q] >= 0) {
        v[q].load(z + (long)row[q] * a.ldz);
        g[q] = w == nullptr ? 1.f : w[j0 + q];
      }
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (row[q] >= 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = __builtin_fmaf(g[q], v[q].get(e), y[e]);
      }
  }
  if (a.add != nullptr) {
    float b[8];
    load8(reinterpret_cast<const Y*>(a.add) + t * a.ld_add + c, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] += b[e];
  }
  store8(reinterpret_cast<Y*>(a.y) + t * a.ldy + c, y);
}

template <typename Z, typename Y>
__global__ __launch_bounds__(256) void slot_sum_grad_kernel(SlotSumArgs a) {
  const int lane = threadIdx.x & 63;
  const long slots = (long)a.T * a.topk, stride = (long)gridDim.x * 4;
  for (long s = (long)blockIdx.x * 4 + (threadIdx.x >> 6); s < slots; s += stride) {
    const long t = s / a.topk;
    const int row = slot_row(a, a.inv[s]);
    float dot = 0.f;
    if (row >= 0) {
      const float g = a.w == nullptr ? 1.f : a.w[s];
      const Y* dy = reinterpret_cast<const Y*>(a.dy) + t * a.ld_dy;
      const Z* z = reinterpret_cast<const Z*>(a.z) + (long)row * a.ldz;
      Z* dz = reinterpret_cast<Z*>(a.dz) + (long)row * a.ld_dz;
      for (int c0 = 0; c0 < a.d; c0 += 4 * 512) {
        Raw8<Y> u[4];
        Raw8<Z> v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c = c0 + q * 512 + lane * 8;
          if (c < a.d) {
            u[q].load(dy + c);
            if (a.dw != nullptr) v[q].load(z + c);
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c = c0 + q * 512 + lane * 8;
          if (c >= a.d) continue;
          if (a.dw != nullptr) {
#pragma unroll
            for (int e = 0; e < 8; ++e) dot = __builtin_fmaf(u[q].get(e), v[q].get(e), dot);
          }
          if (a.dz != nullptr) {
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = g * u[q].get(e);
            store8(dz + c, o);
          }
        }
      }
    }
    if (a.dw != nullptr) {
      dot = wave_sum(dot);
      if (lane == 0) a.dw[s] = dot;
    }
  }
}

// A wave takes a token of up to 512 VPT values.
template <typename Z, typename Y, int VPT>
__global__ __launch_bounds__(256) void slot_sum_grad_tokens_kernel(SlotSumArgs a, int t0) {
  const int lane = threadIdx.x & 63;
  const long t = (long)t0 + blockIdx.x * 4u + (threadIdx.x >> 6);
  if (t >= a.T) return;
  Raw8<Y> u[VPT];
  const Y* dy = reinterpret_cast<const Y*>(a.dy) + t * a.ld_dy;
#pragma unroll
  for (int q = 0; q < VPT; ++q)
    if (q * 512 + lane * 8 < a.d) u[q].load(dy + q * 512 + lane * 8);
  Raw8<Z> v[2][VPT];
  int row[2];
  auto request = [&](int j, int b) {
    row[b] = j < a.topk ? slot_row(a, a.inv[t * a.topk + j]) : -1;
    if (row[b] < 0 || a.dw == nullptr) return;
    const Z* z = reinterpret_cast<const Z*>(a.z) + (long)row[b] * a.ldz;
#pragma unroll
    for (int q = 0; q < VPT; ++q)
      if (q * 512 + lane * 8 < a.d) v[b][q].load(z + q * 512 + lane * 8);
  };
  auto slot = [&](int j, int b) {
    const long s = t * a.topk + j;
    float dot = 0.f;
    if (row[b] >= 0) {
      const float g = a.w == nullptr ? 1.f : a.w[s];
      Z* dz = reinterpret_cast<Z*>(a.dz) + (long)row[b] * a.ld_dz;
#pragma unroll
      for (int q = 0; q < VPT; ++q) {
        const int c = q * 512 + lane * 8;
        if (c >= a.d) continue;
        if (a.dw != nullptr) {
#pragma unroll
          for (int e = 0; e < 8; ++e) dot = __builtin_fmaf(u[q].get(e), v[b][q].get(e), dot);
        }
        if (a.dz != nullptr) {
          float o[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = g * u[q].get(e);
          store8(dz + c, o);
        }
      }
    }
    if (a.dw != nullptr) {
      dot = wave_sum(dot);
      if (lane == 0) a.dw[s] = dot;
    }
  };
  request(0, 0);
  for (int j = 0; j < a.topk; j += 2) {
    request(j + 1, 1);
    slot(j, 0);
    if (j + 1 >= a.topk) break;
    request(j + 2, 0);
    slot(j + 1, 1);
  }
}

template <typename Z, typename Y>
static void go_sum(const SlotSumArgs& a, bool grad, hipStream_t s) {
  if (grad && a.T >= 4096 && a.d <= 4096) {
    // (2^24 workgroups of 256 threads are a launch)
    for (long t0 = 0; t0 < a.T; t0 += 1 << 24) {
      const long n = a.T - t0 < (1 << 24) ? a.T - t0 : 1 << 24;
      const dim3 grid((unsigned)((n + 3) / 4));
      if (a.d <= 2048) hipLaunchKernelGGL((slot_sum_grad_tokens_kernel<Z, Y, 4>), grid, dim3(256), 0, s, a, (int)t0);
      else hipLaunchKernelGGL((slot_sum_grad_tokens_kernel<Z, Y, 8>), grid, dim3(256), 0, s, a, (int)t0);
    }
    return;
  }
  if (grad) {
    const long slots = (long)a.T * a.topk, groups = (slots + 3) / 4;
    hipLaunchKernelGGL((slot_sum_grad_kernel<Z, Y>), dim3((unsigned)(groups < (1 << 20) ? groups : 1 << 20)), dim3(256), 0,
                       s, a);
    return;
  }
  // tokens in parts whose vectors a 32-bit index counts
  const uint32_t nv = (uint32_t)a.d / 8;
  const long part = ((1L << 31) - 256) / nv;
  for (long t0 = 0; t0 < a.T; t0 += part) {
    const uint32_t n = (uint32_t)(a.T - t0 < part ? a.T - t0 : part);
    hipLaunchKernelGGL((slot_sum_kernel<Z, Y>), dim3((n * nv + 255) / 256), dim3(256), 0, s, a, (int)t0, n * nv, nv);
  }
}
template <typename Z>
static void go_sum_y(const SlotSumArgs& a, bool grad, int ydt, hipStream_t s) {
  if (ydt == 0) go_sum<Z, half_t>(a, grad, s);
  else if (ydt == 1) go_sum<Z, __bf16>(a, grad, s);
  else go_sum<Z, float>(a, grad, s);
}
static void go_sum_z(const SlotSumArgs& a, bool grad, int zdt, int ydt, hipStream_t s) {
  if (zdt == 0) go_sum_y<half_t>(a, grad, ydt, s);
  else if (zdt == 1) go_sum_y<__bf16>(a, grad, ydt, s);
  else go_sum_y<float>(a, grad, ydt, s);
}
void launch_slot_sum(const SlotSumArgs& a, int zdt, int ydt, hipStream_t s) { go_sum_z(a, false, zdt, ydt, s); }
void launch_slot_sum_grad(const SlotSumArgs& a, int zdt, int ydt, hipStream_t s) { go_sum_z(a, true, zdt, ydt, s); }

}  // namespace tq
