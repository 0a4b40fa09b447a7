// A whole layer of experts that are not packed, for a few tokens, in two kernels.
//
//   up:    h[s] = RND_act(silu(W_gate,e x_t) W_up,e x_t)     s = t k + j, e = ids[s]
//   down:  z[s] = w[s] W_down,e h[s],  y[t] = add[t] + sum_j z[t k + j]
//
// Bound by the weights' bytes: each weight of an expert that is chosen meets
// the few tokens that chose it.  Weights go from memory straight to the
// registers of the one wave that uses them, in the fragment layout of the MFMA
// (16 outputs x 16 bytes of k a lane).  A workgroup takes 16 outputs of one
// expert (the up kernel 16 of the gate and the same 16 of the up matrix, whose
// product it then forms) for all of the expert's slots, 16 FN at a time; its
// waves share k in interleaved runs of D steps of 128 bytes, each requesting
// its next run before it multiplies the last, and their sums are added in LDS in
// wave order.  The slots of an expert are found by each workgroup in ids, so
// nothing runs ahead of the first product.
//
// y needs all experts of a token.  A workgroup of the down kernel stores its
// z and counts itself done for its 16 outputs; the last one adds the slots of
// each token in order.  So the sum has one order whichever workgroup is last,
// and there is no third launch and no atomic on y.  The up kernel sets the
// counters to zero.
//
// 8-bit weights (integers with an f32 scale for each output) are unpacked to
// the activations' type, exactly, next to the MFMA; the scale meets the sum.
// Few tokens are bound by the weights' bytes, so the activations keep 16 bits.
#include "group_body.h"
#include "layer_ops.h"

namespace tq {

// 16 integers of 8 bits (one lane's 16 bytes of k) as two MFMA operands.
// f16: the byte plus 128 in the low bits of 1024.0, less 1152.  bf16 holds 8
// bits, so every integer converts exactly; the upper halves of the f32 values.
template <typename T> struct Unpack8;
template <> struct Unpack8<half_t> {
  static __device__ __forceinline__ void get(u32x4 v, u32x4& a, u32x4& b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t t = v[i] ^ 0x80808080u;
      const half2v off = {(half_t)-1152.f, (half_t)-1152.f};
      const uint32_t lo = __builtin_bit_cast(
          uint32_t, __builtin_bit_cast(half2v, __builtin_amdgcn_perm(0x64646464u, t, 0x04010400u)) + off);
      const uint32_t hi = __builtin_bit_cast(
          uint32_t, __builtin_bit_cast(half2v, __builtin_amdgcn_perm(0x64646464u, t, 0x04030402u)) + off);
      u32x4& o = i < 2 ? a : b;
      o[2 * (i & 1)] = lo;
      o[2 * (i & 1) + 1] = hi;
    }
  }
};
template <> struct Unpack8<__bf16> {
  static __device__ __forceinline__ void get(u32x4 v, u32x4& a, u32x4& b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t f[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = __builtin_bit_cast(uint32_t, (float)(int8_t)(v[i] >> (8 * j)));
      u32x4& o = i < 2 ? a : b;
      o[2 * (i & 1)] = __builtin_amdgcn_perm(f[1], f[0], 0x07060302u);
      o[2 * (i & 1) + 1] = __builtin_amdgcn_perm(f[3], f[2], 0x07060302u);
    }
  }
};

// The expert of work unit `unit` and its slots, ascending, in s_slot.  With no
// more slots than experts, unit u is slot u, and the first slot of an expert
// works for all of them; else unit u is expert u.  Every wave looks through
// ids; the first one writes the list.  Returns the number of slots, 0 when
// there is nothing to do.
__device__ __forceinline__ int find_slots(const ExpertsArgs& a, int unit, int lane, int wave, int* s_slot, int* expert) {
  const int S = a.T * a.topk;
  const bool by_slot = S <= a.experts;
  const int e = by_slot ? a.ids[unit] : unit;
  *expert = e;
  if (e < 0 || e >= a.experts) return 0;
  int n = 0, first = -1;
  for (int s0 = 0; s0 < S; s0 += 64) {
    const int s = s0 + lane;
    const bool mine = s < S && a.ids[s] == e;
    const uint64_t m = __ballot(mine);
    if (m == 0) continue;
    if (first < 0) first = s0 + __ffsll((unsigned long long)m) - 1;
    if (wave == 0 && mine) s_slot[n + __popcll(m & ((1ull << lane) - 1))] = s;
    n += __popcll(m);
  }
  if (by_slot && first != unit) return 0;
  return n;
}

// Sums of FM x FN fragments over the waves, in wave order; the result goes to
// wave j for column fragment j.
template <int WAVES, int FM, int FN>
__device__ __forceinline__ void join_waves(f32x4 (&acc)[FM][FN], f32x4 (*s_sum)[FM * FN][64], int wave, int lane,
                                           f32x4 (&sum)[FM]) {
  static_assert(WAVES >= FN, "a wave for each column fragment");
#pragma unroll
  for (int f = 0; f < FM * FN; ++f) s_sum[wave][f][lane] = acc[f / FN][f % FN];
  __syncthreads();
  if (wave < FN) {
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      sum[i] = s_sum[0][i * FN + wave][lane];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) sum[i] += s_sum[w][i * FN + wave][lane];
    }
  }
}

// FM fragments of 16 rows of a matrix [..][K] (their bases in wb, rows that
// exist in wn) times 16 FN columns, whose rows of 16-bit values start xo bytes
// into xb (OOB: zeros).  The waves share k; acc holds this wave's part.
template <typename T, bool I8, int WAVES, int FM, int FN, int D>
__device__ __forceinline__ void part_of_product(const char* const (&wb)[FM], int wn, int K, const char* xb,
                                                const uint32_t (&xo)[FN], int wave, int lane, f32x4 (&acc)[FM][FN]) {
  constexpr int ES = I8 ? 1 : 2, XB = I8 ? 2 : 1;   // bytes of a weight; 16-byte loads of x for one of W
  const int l16 = lane & 15, lg = lane >> 4;
  const int bytes = K * ES, nstep = (bytes + 127) >> 7, nrun = (nstep + D - 1) / D;
  __amdgpu_buffer_rsrc_t rw[FM];
#pragma unroll
  for (int i = 0; i < FM; ++i) rw[i] = make_rsrc(wb[i], (uint32_t)OOB);
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(xb, (uint32_t)OOB);
  const uint32_t vw = l16 < wn ? (uint32_t)l16 * (uint32_t)bytes + lg * 16u : OOB;
  struct Run {
    u32x4 w[D][FM][2], x[D][FN][2][XB];
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
        const bool ok = live && st * 128 + h * 64 + lg * 16 < bytes;
#pragma unroll
        for (int i = 0; i < FM; ++i) r.w[d][i][h] = bload128(rw[i], ok ? vw + h * 64u : OOB, so);
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int q = 0; q < XB; ++q)
            r.x[d][j][h][q] = bload128(rx, ok && xo[j] != OOB ? xo[j] + (h * 64u + lg * 16u) * XB + q * 16u : OOB, so * XB);
      }
    }
  };
  auto multiply = [&](const Run& r) {
#pragma unroll
    for (int d = 0; d < D; ++d)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < FM; ++i) {
          if constexpr (I8) {
            u32x4 w0, w1;
            Unpack8<T>::get(r.w[d][i][h], w0, w1);
#pragma unroll
            for (int j = 0; j < FN; ++j) {
              acc[i][j] = mfma_half<T>(w0, r.x[d][j][h][0], acc[i][j]);
              acc[i][j] = mfma_half<T>(w1, r.x[d][j][h][1], acc[i][j]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = mfma_half<T>(r.w[d][i][h], r.x[d][j][h][0], acc[i][j]);
          }
        }
  };
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
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
}

// scales of outputs o .. o + 3 (those below n)
__device__ __forceinline__ f32x4 scales4(const float* p, int o, int n) {
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int v = 0; v < 4; ++v)
    if (o + v < n) s[v] = p[o + v];
  return s;
}

template <typename T, bool I8, int WAVES, int FN, int D>
__global__ __launch_bounds__(64 * WAVES) void experts_up_kernel(ExpertsArgs a, int mtile) {
  __shared__ int s_slot[EXPERTS_SLOTS];
  __shared__ f32x4 s_sum[WAVES][2 * FN][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, lg = lane >> 4;
  if (blockIdx.x == gridDim.x - 1) {
    // one workgroup more: clears the counters, counts the experts with a slot
    for (int i = threadIdx.x; i < experts_tiles(a.d); i += 64 * WAVES) a.done[i] = 0;
    int* s_hit = s_slot;                        // [1024 / 32]
    if (threadIdx.x < 32) s_hit[threadIdx.x] = 0;
    __syncthreads();
    for (int s = threadIdx.x; s < a.T * a.topk; s += 64 * WAVES) {
      const int e = a.ids[s];
      if (e >= 0 && e < a.experts) atomicOr(&s_hit[e >> 5], 1 << (e & 31));
    }
    __syncthreads();
    if (wave == 0) {
      const int n = wave_sum_i(lane < 32 ? __popc((unsigned)s_hit[lane & 31]) : 0);
      if (lane == 0) *a.hit = n;
    }
    return;
  }
  const int unit = blockIdx.x / mtile, m0 = (blockIdx.x - unit * mtile) * 16;
  int e;
  const int n = __builtin_amdgcn_readfirstlane(find_slots(a, unit, lane, wave, s_slot, &e));
  if (n == 0) return;
  e = __builtin_amdgcn_readfirstlane(e);
  __syncthreads();

  constexpr int ES = I8 ? 1 : 2;
  const char* w = reinterpret_cast<const char*>(a.w_up) + ((size_t)e * 2 * a.ff + m0) * a.d * ES;
  const char* const wb[2] = {w, w + (size_t)a.ff * a.d * ES};
  for (int c0 = 0; c0 < n; c0 += 16 * FN) {
    uint32_t xo[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int c = c0 + 16 * j + l16;
      xo[j] = c < n ? (uint32_t)(s_slot[c] / a.topk) * (uint32_t)(a.ldx * 2) : OOB;
    }
    f32x4 acc[2][FN], sum[2];
    part_of_product<T, I8, WAVES, 2, FN, D>(wb, a.ff - m0, a.d, reinterpret_cast<const char*>(a.x), xo, wave, lane, acc);
    if (c0 > 0) __syncthreads();
    join_waves<WAVES, 2, FN>(acc, s_sum, wave, lane, sum);
    const int c = c0 + 16 * wave + l16, o = m0 + 4 * lg;
    if (wave >= FN || c >= n || o >= a.ff) continue;
    if constexpr (I8) {
      const f32x4 sg = scales4(a.s_up + (size_t)e * 2 * a.ff, o, a.ff), su = scales4(a.s_up + ((size_t)e * 2 + 1) * a.ff, o, a.ff);
      sum[0] *= sg;
      sum[1] *= su;
    }
    typedef T T4 __attribute__((ext_vector_type(4)));
    T4 h;
#pragma unroll
    for (int v = 0; v < 4; ++v) h[v] = (T)(silu_f(sum[0][v]) * sum[1][v]);
    *reinterpret_cast<T4*>(reinterpret_cast<T*>(a.h) + (size_t)s_slot[c] * a.ff + o) = h;   // ff % 8 == 0
  }
}

// y of 16 outputs from o0: the slots of each token in order
template <int WAVES>
__device__ __forceinline__ void add_slots(const ExpertsArgs& a, int o0, bool any) {
  for (int i = threadIdx.x; i < a.T * 16; i += 64 * WAVES) {
    const int t = i >> 4, o = o0 + (i & 15);
    if (o >= a.d) continue;
    float y = 0.f;
    if (any)
      for (int j = 0; j < a.topk; ++j) {
        const int s = t * a.topk + j, e = a.ids[s];
        if (e >= 0 && e < a.experts) y += a.z[(size_t)s * a.d + o];
      }
    const size_t at = (size_t)t * a.ldy + o, from = (size_t)t * a.ld_add + o;
    if (a.ydt == 2) {
      if (a.add != nullptr) y += reinterpret_cast<const float*>(a.add)[from];
      reinterpret_cast<float*>(a.y)[at] = y;
    } else if (a.ydt == 1) {
      if (a.add != nullptr) y += (float)reinterpret_cast<const __bf16*>(a.add)[from];
      reinterpret_cast<__bf16*>(a.y)[at] = (__bf16)y;
    } else {
      if (a.add != nullptr) y += (float)reinterpret_cast<const half_t*>(a.add)[from];
      reinterpret_cast<half_t*>(a.y)[at] = (half_t)y;
    }
  }
}

template <typename T, bool I8, int WAVES, int FN, int D>
__global__ __launch_bounds__(64 * WAVES) void experts_down_kernel(ExpertsArgs a, int mtile) {
  __shared__ int s_slot[EXPERTS_SLOTS];
  __shared__ f32x4 s_sum[WAVES][FN][64];
  __shared__ int s_last;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, lg = lane >> 4;
  const int unit = blockIdx.x / mtile, m = blockIdx.x - unit * mtile, m0 = m * 16;
  const int hit = *a.hit;
  int e;
  const int n = __builtin_amdgcn_readfirstlane(find_slots(a, unit, lane, wave, s_slot, &e));
  if (n == 0) {
    if (hit == 0 && unit == 0) add_slots<WAVES>(a, m0, false);      // no slot at all
    return;
  }
  e = __builtin_amdgcn_readfirstlane(e);
  __syncthreads();

  constexpr int ES = I8 ? 1 : 2;
  const char* const wb[1] = {reinterpret_cast<const char*>(a.w_down) + ((size_t)e * a.d + m0) * a.ff * ES};
  for (int c0 = 0; c0 < n; c0 += 16 * FN) {
    uint32_t xo[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int c = c0 + 16 * j + l16;
      xo[j] = c < n ? (uint32_t)s_slot[c] * (uint32_t)(a.ff * 2) : OOB;
    }
    f32x4 acc[1][FN], sum[1];
    part_of_product<T, I8, WAVES, 1, FN, D>(wb, a.d - m0, a.ff, reinterpret_cast<const char*>(a.h), xo, wave, lane, acc);
    if (c0 > 0) __syncthreads();
    join_waves<WAVES, 1, FN>(acc, s_sum, wave, lane, sum);
    const int c = c0 + 16 * wave + l16, o = m0 + 4 * lg;
    if (wave >= FN || c >= n || o >= a.d) continue;
    const int s = s_slot[c];
    const float g = a.w[s];
    if constexpr (I8) sum[0] *= scales4(a.s_down + (size_t)e * a.d, o, a.d);
    *reinterpret_cast<f32x4*>(a.z + (size_t)s * a.d + o) = sum[0] * g;        // d % 8 == 0
  }
  // this workgroup's z before its count, the count before the others' z
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0)
    s_last = __hip_atomic_fetch_add(a.done + m, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == hit - 1;
  __syncthreads();
  if (s_last == 0) return;
  __threadfence();
  add_slots<WAVES>(a, m0, true);
}

template <typename T, bool I8, int WAVES, int FN, int D>
static void go_up(const ExpertsArgs& a, hipStream_t s) {
  const int mtile = (a.ff + 15) / 16, S = a.T * a.topk, units = S <= a.experts ? S : a.experts;
  hipLaunchKernelGGL((experts_up_kernel<T, I8, WAVES, FN, D>), dim3((unsigned)(mtile * units + 1)), dim3(64 * WAVES), 0, s, a, mtile);
}
template <typename T, bool I8, int WAVES, int FN, int D>
static void go_down(const ExpertsArgs& a, hipStream_t s) {
  const int mtile = experts_tiles(a.d), S = a.T * a.topk, units = S <= a.experts ? S : a.experts;
  hipLaunchKernelGGL((experts_down_kernel<T, I8, WAVES, FN, D>), dim3((unsigned)(mtile * units)), dim3(64 * WAVES), 0, s, a, mtile);
}

// Waves of a workgroup: 8 where there are few workgroups and each wave still
// has two runs of k, else 4.  Columns: 16 unless more slots of one expert are
// likely; an expert with more of them goes over its weights again.
template <typename T, bool I8, int FN, int D>
static void go_waves(const ExpertsArgs& a, hipStream_t s) {
  const int S = a.T * a.topk, units = S <= a.experts ? S : a.experts;
  const int up = (a.ff + 15) / 16 * units, down = experts_tiles(a.d) * units;
  const int run = 128 * D / (I8 ? 1 : 2);       // values of k in a run
  if constexpr (FN < 4) {
    if (up < 768 && a.d >= 16 * run) go_up<T, I8, 8, FN, D>(a, s);
    else go_up<T, I8, 4, FN, D>(a, s);
    if (down < 768 && a.ff >= 16 * run) go_down<T, I8, 8, FN, D>(a, s);
    else go_down<T, I8, 4, FN, D>(a, s);
  } else {
    go_up<T, I8, 4, FN, D>(a, s);
    go_down<T, I8, 4, FN, D>(a, s);
  }
}

template <typename T, bool I8>
static void go_cols(const ExpertsArgs& a, hipStream_t s) {
  const int S = a.T * a.topk;
  if (a.T <= 16 || S <= 6 * a.experts) go_waves<T, I8, 1, 2>(a, s);
  else if (a.T <= 32 || S <= 20 * a.experts) go_waves<T, I8, 2, I8 ? 1 : 2>(a, s);
  else go_waves<T, I8, 4, 1>(a, s);
}

void launch_experts(const ExpertsArgs& a, int act, bool int8, hipStream_t s) {
  if (act == 0) {
    if (int8) go_cols<half_t, true>(a, s);
    else go_cols<half_t, false>(a, s);
  } else {
    if (int8) go_cols<__bf16, true>(a, s);
    else go_cols<__bf16, false>(a, s);
  }
}

}  // namespace tq
