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
// product it then forms), or 32 or 64, for all of the expert's slots, 16 FN at a
// time; its waves share k in interleaved steps of 128 bytes, each requesting its
// next step before it multiplies the last, and their sums are added in LDS in
// wave order.  The slots of an expert are found by each workgroup in ids, so
// nothing runs ahead of the first product.
//
// y needs all experts of a token.  A workgroup of the down kernel stores its
// z and counts itself done for its 16 outputs; the last one adds the slots of
// each token in order.  So the sum has one order whichever workgroup is last,
// and there is no third launch and no atomic on y.  The up kernel sets the
// counters to zero.  A single token's down workgroups go over all its slots
// instead.
//
// A call for 32 tokens through four of 60 experts of 2048 -> 1408, f16: 176 us, 5.2
// TB/s of the 53 experts' weights (a plain read of a larger buffer: 5.5); for one token
// through two of eight of 4096 -> 14336 in 8 bits: 74 us, 4.7 TB/s.
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

// Every wave's FM x FN fragments in LDS, and one of them added over the waves in
// wave order.
template <int FM, int FN>
__device__ __forceinline__ void put_parts(const f32x4 (&acc)[FM][FN], f32x4 (*s_sum)[FM * FN][64], int wave, int lane) {
#pragma unroll
  for (int f = 0; f < FM * FN; ++f) s_sum[wave][f][lane] = acc[f / FN][f % FN];
  __syncthreads();
}
template <int WAVES, int F>
__device__ __forceinline__ f32x4 sum_parts(const f32x4 (*s_sum)[F][64], int f, int lane) {
  f32x4 v = s_sum[0][f][lane];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) v += s_sum[w][f][lane];
  return v;
}

// A step of k: 128 bytes of each of 16 FM weight rows, and what they meet of 16 FN
// columns of 16-bit values.
template <typename T, bool I8, int FM, int FN> struct Step {
  static constexpr int XB = I8 ? 2 : 1;         // 16-byte loads of a column for one of a weight row
  u32x4 w[FM][2], x[FN][2][XB];

  // step st of rows of `bytes` bytes: vw, xo are byte offsets of this lane's row
  // and column (OOB: zeros)
  __device__ __forceinline__ void fetch(int st, int bytes, int lg, const __amdgpu_buffer_rsrc_t (&rw)[FM],
                                        const uint32_t (&vw)[FM], __amdgpu_buffer_rsrc_t rx, const uint32_t (&xo)[FN]) {
    const uint32_t so = st * 128u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // bytes 64 h + 16 lg of the step's 128: past the row, nothing is read
      const bool ok = st * 128 + h * 64 + lg * 16 < bytes;
#pragma unroll
      for (int i = 0; i < FM; ++i) w[i][h] = bload128(rw[i], ok ? vw[i] + h * 64u : OOB, so);
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int q = 0; q < XB; ++q)
          x[j][h][q] = bload128(rx, ok && xo[j] != OOB ? xo[j] + (h * 64u + lg * 16u) * XB + q * 16u : OOB, so * XB);
    }
  }
  __device__ __forceinline__ void multiply(f32x4 (&acc)[FM][FN]) const {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        if constexpr (I8) {
          u32x4 w0, w1;
          Unpack8<T>::get(w[i][h], w0, w1);
#pragma unroll
          for (int j = 0; j < FN; ++j) {
            acc[i][j] = mfma_half<T>(w0, x[j][h][0], acc[i][j]);
            acc[i][j] = mfma_half<T>(w1, x[j][h][1], acc[i][j]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < FN; ++j) acc[i][j] = mfma_half<T>(w[i][h], x[j][h][0], acc[i][j]);
        }
      }
  }
};

// FM fragments of 16 weight rows of K values times 16 FN columns of 16-bit values,
// for `tiles` such products one after the other.  The waves share k in
// interleaved steps; a wave requests its next step, of the next product too,
// before it multiplies the last.  (The last request of a run is not made, so the
// compiler's waits for a step cover its successor too: more requests in flight are
// no gain here, they were 3 to 8 % slower with 16-bit weights.)  tile(t, rw, vw,
// xo) sets what Step::fetch takes; done(t, acc) gets this wave's part; all waves
// call it for all tiles.
template <typename T, bool I8, int WAVES, int FM, int FN, class Tile, class Done>
__device__ __forceinline__ void stream_tiles(int tiles, int K, const char* xb, int wave, int lane, Tile tile, Done done) {
  const int lg = lane >> 4;
  const int bytes = K * (I8 ? 1 : 2), nstep = (bytes + 127) >> 7, per = (nstep + WAVES - 1) / WAVES;
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(xb, (uint32_t)OOB);
  __amdgpu_buffer_rsrc_t rw[FM];
  uint32_t vw[FM], xo[FN];
  int ft = -1, fi = per;                        // tile and step that were requested last
  auto request = [&](Step<T, I8, FM, FN>& r) {
    if (fi == per) {
      fi = 0;
      if (++ft < tiles) tile(ft, rw, vw, xo);
    }
    if (ft >= tiles) return;
    // (a step past the last one reads nothing)
    r.fetch(wave + WAVES * fi, bytes, lg, rw, vw, rx, xo);
    ++fi;
  };
  f32x4 acc[FM][FN];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  };
  clear();
  Step<T, I8, FM, FN> r0, r1;
  int t = 0, i = 0;
  request(r0);
  for (;;) {
    request(r1);
    r0.multiply(acc);
    if (++i == per) {
      done(t, acc);
      if (++t == tiles) break;
      clear();
      i = 0;
    }
    request(r0);
    r1.multiply(acc);
    if (++i == per) {
      done(t, acc);
      if (++t == tiles) break;
      clear();
      i = 0;
    }
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

// 16 P outputs of the gate and the same of the up matrix.  ONE: a single token,
// whose slots are the work units as they are.
template <typename T, bool I8, int WAVES, int P, int FN, bool ONE>
__global__ __launch_bounds__(64 * WAVES) void experts_up_kernel(ExpertsArgs a, int mtile) {
  __shared__ int s_slot[ONE ? 1 : EXPERTS_SLOTS];
  __shared__ f32x4 s_sum[ONE ? 1 : 2][WAVES][2 * P * FN][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, lg = lane >> 4;
  if (!ONE && blockIdx.x == gridDim.x - 1) {
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
  const int unit = blockIdx.x / mtile, m0 = (blockIdx.x - unit * mtile) * 16 * P;
  int e, n = 1;
  if constexpr (ONE) {
    e = a.ids[unit];
    if (e < 0 || e >= a.experts) return;
  } else {
    n = __builtin_amdgcn_readfirstlane(find_slots(a, unit, lane, wave, s_slot, &e));
    if (n == 0) return;
    e = __builtin_amdgcn_readfirstlane(e);
    __syncthreads();
  }
  constexpr int ES = I8 ? 1 : 2;
  const int chunks = ONE ? 1 : (n + 16 * FN - 1) / (16 * FN);
  const char* const w0 = reinterpret_cast<const char*>(a.w_up) + (size_t)e * 2 * a.ff * a.d * ES;
  stream_tiles<T, I8, WAVES, 2 * P, FN>(
      chunks, a.d, reinterpret_cast<const char*>(a.x), wave, lane,
      [&](int t, __amdgpu_buffer_rsrc_t (&rw)[2 * P], uint32_t (&vw)[2 * P], uint32_t (&xo)[FN]) {
        const int c0 = t * 16 * FN;
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const char* w = w0 + (size_t)(m0 + 16 * p) * a.d * ES;
          rw[p] = make_rsrc(w, (uint32_t)OOB);
          rw[P + p] = make_rsrc(w + (size_t)a.ff * a.d * ES, (uint32_t)OOB);
          vw[p] = vw[P + p] = l16 < a.ff - m0 - 16 * p ? (uint32_t)l16 * (uint32_t)(a.d * ES) + lg * 16u : OOB;
        }
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const int c = c0 + 16 * j + l16;
          xo[j] = c < n ? (ONE ? 0u : (uint32_t)(s_slot[c] / a.topk) * (uint32_t)(a.ldx * 2)) : OOB;
        }
      },
      [&](int t, const f32x4 (&acc)[2 * P][FN]) {
        // (two places for the parts: a wave that is a tile ahead writes the other)
        f32x4(*const sum)[2 * P * FN][64] = s_sum[ONE ? 0 : t & 1];
        put_parts<2 * P, FN>(acc, sum, wave, lane);
        const int c0 = t * 16 * FN;
        for (int f = wave; f < P * FN; f += WAVES) {
          const int c = c0 + 16 * (f % FN) + l16, o = m0 + 16 * (f / FN) + 4 * lg;
          f32x4 g = sum_parts<WAVES, 2 * P * FN>(sum, f, lane), u = sum_parts<WAVES, 2 * P * FN>(sum, P * FN + f, lane);
          if (c >= n || o >= a.ff) continue;
          if constexpr (I8) {
            g *= scales4(a.s_up + (size_t)e * 2 * a.ff, o, a.ff);
            u *= scales4(a.s_up + ((size_t)e * 2 + 1) * a.ff, o, a.ff);
          }
          typedef T T4 __attribute__((ext_vector_type(4)));
          T4 h;
#pragma unroll
          for (int v = 0; v < 4; ++v) h[v] = (T)(silu_f(g[v]) * u[v]);
          const int s = ONE ? unit : s_slot[c];
          *reinterpret_cast<T4*>(reinterpret_cast<T*>(a.h) + (size_t)s * a.ff + o) = h;       // ff % 8 == 0
        }
      });
}

// y[t][o] = add[t][o] + v
__device__ __forceinline__ void put_y(const ExpertsArgs& a, int t, int o, float v) {
  const size_t at = (size_t)t * a.ldy + o, from = (size_t)t * a.ld_add + o;
  if (a.ydt == 2) {
    if (a.add != nullptr) v += reinterpret_cast<const float*>(a.add)[from];
    reinterpret_cast<float*>(a.y)[at] = v;
  } else if (a.ydt == 1) {
    if (a.add != nullptr) v += (float)reinterpret_cast<const __bf16*>(a.add)[from];
    reinterpret_cast<__bf16*>(a.y)[at] = (__bf16)v;
  } else {
    if (a.add != nullptr) v += (float)reinterpret_cast<const half_t*>(a.add)[from];
    reinterpret_cast<half_t*>(a.y)[at] = (half_t)v;
  }
}

// y of M outputs from o0: the slots of each token in order
template <int WAVES, int M>
__device__ __forceinline__ void add_slots(const ExpertsArgs& a, int o0, bool any) {
  for (int i = threadIdx.x; i < a.T * M; i += 64 * WAVES) {
    const int t = i / M, o = o0 + i % M;
    if (o >= a.d) continue;
    float y = 0.f;
    if (any)
      for (int j = 0; j < a.topk; ++j) {
        const int s = t * a.topk + j, e = a.ids[s];
        if (e >= 0 && e < a.experts) y += __hip_atomic_load(a.z + (size_t)s * a.d + o, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    put_y(a, t, o, y);
  }
}

// 16 FM outputs
template <typename T, bool I8, int WAVES, int FM, int FN>
__global__ __launch_bounds__(64 * WAVES) void experts_down_kernel(ExpertsArgs a, int mtile) {
  __shared__ int s_slot[EXPERTS_SLOTS];
  __shared__ f32x4 s_sum[2][WAVES][FM * FN][64];
  __shared__ int s_last;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, lg = lane >> 4;
  const int unit = blockIdx.x / mtile, m = blockIdx.x - unit * mtile, m0 = m * 16 * FM;
  const int hit = *a.hit;
  int e;
  const int n = __builtin_amdgcn_readfirstlane(find_slots(a, unit, lane, wave, s_slot, &e));
  if (n == 0) {
    if (hit == 0 && unit == 0) add_slots<WAVES, 16 * FM>(a, m0, false);      // no slot at all
    return;
  }
  e = __builtin_amdgcn_readfirstlane(e);
  __syncthreads();
  constexpr int ES = I8 ? 1 : 2;
  const int chunks = (n + 16 * FN - 1) / (16 * FN);
  const char* const w0 = reinterpret_cast<const char*>(a.w_down) + (size_t)e * a.d * a.ff * ES;
  stream_tiles<T, I8, WAVES, FM, FN>(
      chunks, a.ff, reinterpret_cast<const char*>(a.h), wave, lane,
      [&](int t, __amdgpu_buffer_rsrc_t (&rw)[FM], uint32_t (&vw)[FM], uint32_t (&xo)[FN]) {
        const int c0 = t * 16 * FN;
#pragma unroll
        for (int i = 0; i < FM; ++i) {
          rw[i] = make_rsrc(w0 + (size_t)(m0 + 16 * i) * a.ff * ES, (uint32_t)OOB);
          vw[i] = l16 < a.d - m0 - 16 * i ? (uint32_t)l16 * (uint32_t)(a.ff * ES) + lg * 16u : OOB;
        }
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const int c = c0 + 16 * j + l16;
          xo[j] = c < n ? (uint32_t)s_slot[c] * (uint32_t)(a.ff * 2) : OOB;
        }
      },
      [&](int t, const f32x4 (&acc)[FM][FN]) {
        f32x4(*const parts_of)[FM * FN][64] = s_sum[t & 1];
        put_parts<FM, FN>(acc, parts_of, wave, lane);
        const int c0 = t * 16 * FN;
        for (int f = wave; f < FM * FN; f += WAVES) {
          const int c = c0 + 16 * (f % FN) + l16, o = m0 + 16 * (f / FN) + 4 * lg;
          f32x4 sum = sum_parts<WAVES, FM * FN>(parts_of, f, lane);
          if (c >= n || o >= a.d) continue;
          const int s = s_slot[c];
          const float g = a.w[s];
          if constexpr (I8) sum *= scales4(a.s_down + (size_t)e * a.d, o, a.d);
          float* z = a.z + (size_t)s * a.d + o;   // d % 8 == 0
#pragma unroll
          for (int v = 0; v < 4; ++v) __hip_atomic_store(z + v, sum[v] * g, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
      });
  // z is written through to where every XCD sees it (stores of agent scope) and
  // has arrived there before the count goes out; the last workgroup reads it
  // from there.  (A release fence instead writes back an XCD's whole L2,
  // for every workgroup: 32 tokens through 60 experts took 1595 us.)  The wait
  // is no memory operation to the compiler: the empty asm keeps the stores ahead
  // of it, as the one in the barrier keeps the count behind it.
  asm volatile("" ::: "memory");
  wait_vm<0>();
  bar_nofence();
  if (threadIdx.x == 0)
    s_last = __hip_atomic_fetch_add(a.done + m, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == hit - 1;
  __syncthreads();
  if (s_last != 0) add_slots<WAVES, 16 * FM>(a, m0, true);
}

// The down product of a single token: 16 outputs over all of its slots, one after
// the other in one run of steps, so that no workgroup waits for another's sums.
template <typename T, bool I8, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void experts_down_one_kernel(ExpertsArgs a) {
  __shared__ f32x4 s_sum[WAVES][1][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, lg = lane >> 4, m0 = blockIdx.x * 16, o = m0 + 4 * lg;
  const int bytes = a.ff * (I8 ? 1 : 2), nstep = (bytes + 127) >> 7, total = nstep * a.topk;
  const uint32_t row = l16 < a.d - m0 ? (uint32_t)l16 * (uint32_t)bytes + lg * 16u : OOB;
  // (slot, step of its k) of a step of the run; an id outside reads zeros
  auto fetch = [&](int st, int j, Step<T, I8, 1, 1>& r) {
    const int e = sload(a.ids, j);
    const bool live = e >= 0 && e < a.experts;
    const __amdgpu_buffer_rsrc_t rw[1] = {make_rsrc(
        reinterpret_cast<const char*>(a.w_down) + ((size_t)(live ? e : 0) * a.d + m0) * bytes, (uint32_t)OOB)};
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(reinterpret_cast<const char*>(a.h) + (size_t)j * a.ff * 2, (uint32_t)OOB);
    const uint32_t vw[1] = {live ? row : OOB}, xo[1] = {live && l16 == 0 ? 0u : OOB};
    r.fetch(st - j * nstep, bytes, lg, rw, vw, rx, xo);
  };
  f32x4 acc[1][1] = {{f32x4{0.f, 0.f, 0.f, 0.f}}}, sum[1][1] = {{f32x4{0.f, 0.f, 0.f, 0.f}}};
  // a slot's part of this wave, times its weight and scales
  auto close = [&](int j) {
    const int e = sload(a.ids, j);
    if (e >= 0 && e < a.experts) {
      f32x4 v = acc[0][0];
      if constexpr (I8) v *= scales4(a.s_down + (size_t)e * a.d, o, a.d);
      sum[0][0] += v * a.w[j];
    }
    acc[0][0] = f32x4{0.f, 0.f, 0.f, 0.f};
  };
  Step<T, I8, 1, 1> r0, r1;
  int st = wave, j0 = wave / nstep, j1 = 0, at = j0;      // slots of r0, of r1 and of acc
  if (st < total) fetch(st, j0, r0);
  for (; st < total; st += 2 * WAVES) {
    if (st + WAVES < total) fetch(st + WAVES, j1 = (st + WAVES) / nstep, r1);
    if (j0 != at) close(at), at = j0;
    r0.multiply(acc);
    if (st + WAVES >= total) break;
    if (st + 2 * WAVES < total) fetch(st + 2 * WAVES, j0 = (st + 2 * WAVES) / nstep, r0);
    if (j1 != at) close(at), at = j1;
    r1.multiply(acc);
  }
  if (wave < total) close(at);
  put_parts<1, 1>(sum, s_sum, wave, lane);
  if (wave > 0 || l16 > 0) return;
  const f32x4 y = sum_parts<WAVES, 1>(s_sum, 0, lane);
#pragma unroll
  for (int v = 0; v < 4; ++v)
    if (o + v < a.d) put_y(a, 0, o + v, y[v]);
}

static int units_of(const ExpertsArgs& a) { return a.T * a.topk <= a.experts ? a.T * a.topk : a.experts; }

template <typename T, bool I8, int WAVES, int P, int FN, bool ONE = false>
static void go_up(const ExpertsArgs& a, hipStream_t s) {
  const int mtile = (a.ff + 16 * P - 1) / (16 * P);
  hipLaunchKernelGGL((experts_up_kernel<T, I8, WAVES, P, FN, ONE>),
                     dim3((unsigned)(ONE ? mtile * a.topk : mtile * units_of(a) + 1)), dim3(64 * WAVES), 0, s, a, mtile);
}
template <typename T, bool I8, int WAVES, int FM, int FN>
static void go_down(const ExpertsArgs& a, hipStream_t s) {
  const int mtile = (a.d + 16 * FM - 1) / (16 * FM);
  hipLaunchKernelGGL((experts_down_kernel<T, I8, WAVES, FM, FN>), dim3((unsigned)(mtile * units_of(a))), dim3(64 * WAVES),
                     0, s, a, mtile);
}

// A workgroup's outputs and waves, by what was measured (us of a call, bf16, k in
// steps of 128 bytes; the kernel that is taken first, then the others on the same
// inputs; "large": experts of 4096 -> 14336, "small": of 2048 -> 1408):
//   one   a single token: no slots to look for, and the down kernel takes 16 outputs
//         of all its slots (8-bit, 4 of 60 small experts: 15.7, by the kernels below
//         17.7; 8 of 16 of 5120 -> 1536: 49.6, 57.1; one of 32 of 4096 -> 4096 in 16 bits:
//         24.7, 29.8).  Up 8 waves from 32 steps (2 of 8 large ones in 16 bits: 121, 4
//         waves 125; 4 of 60 small ones 21.0, 20.3), else 4 (8-bit, the 60 small: 15.7,
//         8 waves 16.1); down 8 waves from 256 workgroups (5120: 49.5, 16 waves 51.8;
//         large ones 71.3, 70.9), else 16 (8-bit small: 15.7, 8 waves 16.6)
//   up    from 64 steps 16 outputs, 8 waves (2 of 8 large ones, 8 tokens: 375; 4 waves
//         386, 32 outputs 400); from 32 steps 32 outputs, 4 waves (8-bit, the same: 213,
//         16 outputs 206; 32 tokens 278, 286), 8 waves below 512 workgroups (2 of 8
//         small ones, 8 tokens: 34.8; 4 waves 33.2, 16 outputs and 4 waves 31.4: the
//         slower way since a wave goes over all its products in one loop); below 16
//         outputs, 4 waves (8-bit small ones, 4 of 60, 32 tokens: 120.2, 32 outputs
//         118.9; 6 of 64, 64 tokens: 178, 168; 8 waves 147 and 208)
//   down  from 64 steps or below 512 workgroups 32 outputs, 8 waves (large ones, 32
//         tokens: 489, 4 waves 490, 64 outputs 489; in 8 bits 278, 279, 272; 2 of 8 of
//         1024 -> 1408, 8 tokens: 19.2, 16 outputs 19.7); else 4 waves and 16 outputs
//         (4 of 60 small ones, 32 tokens: 178, 32 outputs 180, 8 waves 195) or, in 8
//         bits, 32 (120, 16 outputs 125, 8 waves 135)
// Columns: 16 up to 10 slots an expert on average (large ones, 40 tokens: 507, with 32
// columns 517; 48 tokens: 574, 524; for small ones 16 stay the faster up to some 14:
// 160 tokens through 4 of 60: 276, 291), 32 up to 24 (large ones, 96 tokens: 592, with
// 64 columns 653, with 16 940), else 64 (112 tokens: 680, with 32 columns 701; 128: 707,
// 913; in 8 bits 473, 414 and 489, 497).  An expert with more slots goes over its
// weights again.  The workgroups there: 32 outputs and 4 waves up, 64 and 8 (with 64
// columns 4) down.  (From 13 to 32 slots an expert on, by the sizes, the grouped
// products take less: large ones, 80 tokens 563 against 608, 128 tokens 604 and 708; one
// of four large ones for 128 tokens 363 against 353 here.)
ExpertsPick choose_experts(const ExpertsArgs& a, bool int8) {
  const int units = units_of(a), S = a.T * a.topk, ES = int8 ? 1 : 2;
  const int up_steps = (a.d * ES + 127) / 128, down_steps = (a.ff * ES + 127) / 128;
  if (a.T == 1) return {1, {16, up_steps >= 32 ? 8 : 4}, {16, experts_tiles(a.d) >= 256 ? 8 : 16}};
  if (a.T > 32 && S > 24 * a.experts) return {64, {32, 4}, {64, 4}};
  if (a.T > 16 && S > 10 * a.experts) return {32, {32, 4}, {64, 8}};
  ExpertsPick p{16, {32, 4}, {int8 ? 32 : 16, 4}};
  if (up_steps >= 64) p.up = {16, 8};
  else if (up_steps < 32) p.up = {16, 4};
  else if (units * ((a.ff + 31) / 32) < 512) p.up = {32, 8};
  if (down_steps >= 64 || units * ((a.d + 31) / 32) < 512) p.down = {32, 8};
  return p;
}

template <typename T, bool I8>
static void go_layer(const ExpertsArgs& a, hipStream_t s) {
  const ExpertsPick p = choose_experts(a, I8);
  if (p.columns == 1) {
    if (p.up.waves == 8) go_up<T, I8, 8, 1, 1, true>(a, s);
    else go_up<T, I8, 4, 1, 1, true>(a, s);
    const dim3 grid((unsigned)experts_tiles(a.d));
    if (p.down.waves == 8) hipLaunchKernelGGL((experts_down_one_kernel<T, I8, 8>), grid, dim3(512), 0, s, a);
    else hipLaunchKernelGGL((experts_down_one_kernel<T, I8, 16>), grid, dim3(1024), 0, s, a);
  } else if (p.columns == 64) {
    go_up<T, I8, 4, 2, 4>(a, s);
    go_down<T, I8, 4, 4, 4>(a, s);
  } else if (p.columns == 32) {
    go_up<T, I8, 4, 2, 2>(a, s);
    go_down<T, I8, 8, 4, 2>(a, s);
  } else {
    if (p.up.outputs == 16) p.up.waves == 8 ? go_up<T, I8, 8, 1, 1>(a, s) : go_up<T, I8, 4, 1, 1>(a, s);
    else p.up.waves == 8 ? go_up<T, I8, 8, 2, 1>(a, s) : go_up<T, I8, 4, 2, 1>(a, s);
    if (p.down.waves == 8) go_down<T, I8, 8, 2, 1>(a, s);
    else go_down<T, I8, 4, I8 ? 2 : 1, 1>(a, s);
  }
}

void launch_experts(const ExpertsArgs& a, int act, bool int8, hipStream_t s) {
  if (act == 0) {
    if (int8) go_layer<half_t, true>(a, s);
    else go_layer<half_t, false>(a, s);
  } else {
    if (int8) go_layer<__bf16, true>(a, s);
    else go_layer<__bf16, false>(a, s);
  }
}

}  // namespace tq
