// Products grouped by expert: rows off[g] .. off[g+1]-1 meet the matrix W_g.
//
//   Y:  y[r][o]  = sum_i W_g[o][i] x[s(r)][i]
//   DX: dx[r][i] = sum_o W_g[o][i] dy[r][o]
//   DW: dW_g[o][i] = sum_{r in g} dy[r][o] x[s(r)][i]
//
// All three are C[n][m] = sum_k A[m][k] B[n][k] with m the dimension that is
// contiguous in the output, so that a lane's four accumulators of an MFMA
// (four neighbouring rows of the A operand) are four neighbouring outputs:
//        A                     B                  m     n     k
//   Y    W_g, k contiguous     x,  k contiguous   out   row   in
//   DX   W_g, m contiguous     dy, k contiguous   in    row   out
//   DW   x,   m contiguous     dy, n contiguous   in    out   row
// An operand whose k is contiguous is staged as rows of 128 bytes of k and
// read with 16-byte LDS reads.  An operand whose k is strided is staged as it
// lies in memory (k rows of MT elements) and transposed on the way out of the
// LDS by the 16 x 4 transposing reads, so no operand is ever copied to
// another layout in memory.
//
// A workgroup computes an MT x NT tile of one group.  Stages of 128 bytes of
// k per row (64 16-bit values, or 128 8-bit values) arrive by buffer loads
// with the LDS destination in rings of three stages of A and two of B.  Rows and k past the
// group, the matrix or the row are never read: their lanes get an offset out
// of the buffer's range, which loads zeros.  Groups are found from `off` in
// the kernel (no host read back); offsets are clamped to 0 .. rows, so no
// content of `off` or `src` leads to an access outside the arrays.
//
// Tile 256 x 256, 8 waves of 128 x 64: per stage 64 KB come in for 4.2 (e4m3:
// 8.4) million products, at most 64 bytes a clock and CU, in 1024 of the 2048
// clocks that its MFMAs take; a smaller tile moves more bytes per product
// (128 x 128: 0.95 PFLOP/s where this one has 1.28).  16x16x32 MFMA reaches 1.9
// PFLOP/s here on random values (the clock falls under load), 32x32x16 1.3.
// Measured, bf16, 32768 rows of 8 experts, 4096 -> 14336: 3.06 ms, 1.26 PFLOP/s
// (a dense library product of the size: 1.57); without its loads it takes 2.58
// ms, without its MFMAs 2.49: memory and matrix unit are used to two thirds
// each (MFMA busy 67 % of the cycles, no LDS bank conflicts) and do not overlap
// fully.  24960 rows of 64 ragged experts, 2048 -> 1408, f16: 183 us, DX (128 x
// 128) 219 us, DW 282 us; there a round of workgroups that is not full, and 6 us
// of start and end for each tile, count as much.  e4m3, 16384 x 4096 -> 14336:
// 1.09 ms, 1.77 PFLOP/s.  A stage of it takes 2.6 us where one of 16 bits, with
// the same bytes and MFMA clocks, takes 1.6: not the loads hold it.  6.2 vector
// instructions go with each MFMA (16 bits: 1.1), four of them the fma that need
// its result: 25 clocks of the vector unit and 32 of the matrix unit in the 88
// that one MFMA of a SIMD takes (busy 38 % with the MFMAs' issue, and 36 %).
#include "group_body.h"

namespace tq {

// The i-th group in the order of work, and its rows [lo, hi): first the groups
// with more than twice the average of rows, so that long sums do not start
// last, then the others; in plain order above 64 groups, where each one's
// share is small.
__device__ __forceinline__ int work_order(const GroupArgs& a, int lane, int i, int* lo, int* hi) {
  if (a.groups > 64) {
    group_span(a, i, lo, hi);
    return i;
  }
  int l = 0, h = 0;
  if (lane < a.groups) group_span(a, lane, &l, &h);
  const bool mine = lane < a.groups, heavy = mine && (long)(h - l) * a.groups > 2L * a.rows;
  const uint64_t first = __ballot(heavy), rest = __ballot(mine && !heavy);
  const uint64_t below = lane == 0 ? 0ull : ~0ull >> (64 - lane);
  const int rank = heavy ? __popcll(first & below) : __popcll(first) + __popcll(rest & below);
  const int g = __builtin_amdgcn_readfirstlane(
      __ffsll((unsigned long long)__ballot(mine && rank == i)) - 1);
  *lo = __builtin_amdgcn_readlane(l, g);
  *hi = __builtin_amdgcn_readlane(h, g);
  return g;
}

// Two neighbouring fragments of a column hold, in lane group g, outputs 4g ..
// 4g+3 of 16 each.  Exchanged between the groups (rows of 16 lanes, two swaps a
// register) group g holds 8 neighbours: 8g .. 8g+7 of the 32, and 64 bytes of
// a 16-bit output row are written by one instruction.
__device__ __forceinline__ void join_rows(uint32_t& x, uint32_t& y) {
  const auto r = __builtin_amdgcn_permlane32_swap(x, y, false, false);
  const auto q = __builtin_amdgcn_permlane16_swap(r[0], r[1], false, false);
  x = q[0];
  y = q[1];
  // pinned here: the exchange needs every lane, and must not move behind a
  // caller's branch over the lanes that store
  asm volatile("" : "+v"(x), "+v"(y));
}

template <bool BF>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const f32x2 v = {a, b};
  if constexpr (BF) return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
  else return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, half2v));
}

// outputs at .. at+7 of fragments v, w (joined), `left` of which exist
template <bool BF>
__device__ __forceinline__ void store8_16(const GroupArgs& a, size_t at, const f32x4& v, const f32x4& w, int left) {
  uint32_t x0 = pack2<BF>(v[0], v[1]), x1 = pack2<BF>(v[2], v[3]);
  uint32_t y0 = pack2<BF>(w[0], w[1]), y1 = pack2<BF>(w[2], w[3]);
  join_rows(x0, y0);
  join_rows(x1, y1);
  if (left <= 0) return;
  uint16_t* p = reinterpret_cast<uint16_t*>(a.out) + at;
  const u32x4 o = {x0, x1, y0, y1};
  if (a.vec_out && left >= 8) {
    *reinterpret_cast<u32x4*>(p) = o;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = (uint16_t)(o[i >> 1] >> (16 * (i & 1)));
  }
}

__device__ __forceinline__ void store8_32(const GroupArgs& a, size_t at, const f32x4& v, const f32x4& w, int left) {
  uint32_t x[4], y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float vi = v[i], wi = w[i];
    x[i] = __builtin_bit_cast(uint32_t, vi);
    y[i] = __builtin_bit_cast(uint32_t, wi);
    join_rows(x[i], y[i]);
  }
  if (left <= 0) return;
  uint32_t* p = reinterpret_cast<uint32_t*>(a.out) + at;
  if (a.vec_out && left >= 8) {
    *reinterpret_cast<u32x4*>(p) = u32x4{x[0], x[1], x[2], x[3]};
    *reinterpret_cast<u32x4*>(p + 4) = u32x4{y[0], y[1], y[2], y[3]};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = i < 4 ? x[i] : y[i - 4];
  }
}

// One operand's tile of R rows (its m or n) in LDS.
//   k contiguous (KC): row r at r * 128, its 16-byte chunk c of k at position
//     c ^ ((r >> 1) & 7): the 16 rows of a fragment read the same chunk from
//     all 64 banks once.
//   k strided: k row at k * R * 2, its 32-byte piece p (16 elements) at
//     position p ^ ((k & 3) | (k >> 3 & 1) << 2): the 8 k rows that half a
//     wave's transposing read touches lie in different banks.
template <bool KC, int R, int NTHR>
struct Operand {
  static constexpr int BYTES = R * 128;
  static constexpr int NLD = BYTES / (NTHR * 16);       // loads per lane and stage
  static_assert(NLD * NTHR * 16 == BYTES, "loads split evenly");
};

template <typename T, int MODE, int MT, int NT, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void group_tile_kernel(GroupArgs a) {
  constexpr bool F8 = sizeof(T) == 1;
  constexpr bool AKC = MODE == GROUP_Y, BKC = MODE != GROUP_DW;
  constexpr int ES = Elem<T>::BYTES;
  constexpr int KS = 128 / ES;                  // k per stage
  constexpr int WAVES = WM * WN, NTHR = 64 * WAVES;
  constexpr int FM = MT / WM / 16, FN = NT / WN / 16;
  typedef Operand<AKC, MT, NTHR> OA;
  typedef Operand<BKC, NT, NTHR> OB;
  static_assert(3 * OA::BYTES + 2 * OB::BYTES <= 160 * 1024, "LDS budget");
  static_assert(AKC || MT >= 128, "strided tile rows hold 8 pieces");
  static_assert(BKC || NT >= 128, "strided tile rows hold 8 pieces");
  // One array per buffer: the compiler then knows that the loads in flight do
  // not touch the buffer being read (with one array it waits for all of them).
  // Three stages of A and two of B: 160 KB in a 256 x 256 tile.
  __shared__ __attribute__((aligned(128))) char a0[OA::BYTES];
  __shared__ __attribute__((aligned(128))) char a1[OA::BYTES];
  __shared__ __attribute__((aligned(128))) char a2[OA::BYTES];
  __shared__ __attribute__((aligned(128))) char b0[OB::BYTES];
  __shared__ __attribute__((aligned(128))) char b1[OB::BYTES];
  char* const ra_[3] = {a0, a1, a2};
  char* const rb_[2] = {b0, b1};

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, lg = lane >> 4;
  const int wm = wave % WM, wn = wave / WM;

  // ---- the tile ----
  int g, m0, n0, row0 = 0, nrow, K, mdim, ndim;
  if constexpr (MODE == GROUP_DW) {
    mdim = a.d_in;
    ndim = a.d_out;
    const int mtile = (mdim + MT - 1) / MT, ntile = (ndim + NT - 1) / NT;
    // XCD x takes the m columns x, x + 8, ... of all groups in turn, each with
    // all its n tiles: a group's work, which grows with its rows, is spread
    // over the XCDs, and the workgroups together on an XCD share columns of x
    const int li = blockIdx.x >> 3;
    const int c = (li / ntile) * 8 + (blockIdx.x & 7);
    if (c >= a.groups * mtile) return;
    const int gi = c / mtile;
    m0 = (c - gi * mtile) * MT;
    n0 = (li % ntile) * NT;
    int lo, hi;
    g = work_order(a, lane, gi, &lo, &hi);
    row0 = __builtin_amdgcn_readfirstlane(lo);
    K = __builtin_amdgcn_readfirstlane(hi - lo);
    nrow = min(NT, ndim - n0);
  } else {
    mdim = MODE == GROUP_Y ? a.d_out : a.d_in;
    K = MODE == GROUP_Y ? a.d_in : a.d_out;
    int m;
    if (!locate_row_tile<NT>(a, lane, (mdim + MT - 1) / MT, &m, &g, &row0, &nrow)) return;
    m0 = m * MT;
    n0 = 0;
  }
  const int nstage = (K + KS - 1) / KS;

  // ---- operand addressing ----
  // byte offsets of this lane's loads from the operand's base, without k
  const char* wg = reinterpret_cast<const char*>(a.w) + (size_t)g * a.d_out * a.d_in * ES;
  uint32_t va[OA::NLD], vb[OB::NLD];
  __amdgpu_buffer_rsrc_t ra, rb;
  if constexpr (MODE == GROUP_Y) {
    ra = make_rsrc(wg + (size_t)m0 * a.d_in * ES, (uint32_t)OOB);
#pragma unroll
    for (int i = 0; i < OA::NLD; ++i) {
      const int r = (wave * OA::NLD + i) * 8 + (lane >> 3);
      const int c = (lane & 7) ^ ((r >> 1) & 7);
      va[i] = m0 + r < mdim ? (uint32_t)r * a.d_in * ES + c * 16u : OOB;
    }
  }
  if constexpr (BKC) {
    const bool gather = MODE == GROUP_Y && a.src != nullptr;
    const char* base = reinterpret_cast<const char*>(MODE == GROUP_Y ? a.x : a.dy);
    const long ld = MODE == GROUP_Y ? a.ldx : a.ldy;
    rb = make_rsrc(gather ? base : base + (size_t)row0 * ld * ES, (uint32_t)OOB);
#pragma unroll
    for (int i = 0; i < OB::NLD; ++i) {
      const int r = (wave * OB::NLD + i) * 8 + (lane >> 3);
      const int c = (lane & 7) ^ ((r >> 1) & 7);
      int row = r;
      if (r >= nrow) row = -1;
      else if (gather) row = source_row(a, a.src[row0 + r]);
      vb[i] = row >= 0 ? (uint32_t)row * (uint32_t)(ld * ES) + c * 16u : OOB;
    }
  }
  // Strided operands: k row and column (16-byte half piece) of load i of this
  // lane, and the operand's first k row.  The base moves with the stage (64
  // bit), the lane offsets inside a stage stay; gathered rows are addressed
  // from x itself.
  auto strided = [&](int R, int i, int nld, int* k, int* col) {
    const int byte = (wave * nld + i) * 1024 + lane * 16;
    *k = byte / (2 * R);
    const int p = (byte % (2 * R)) >> 5;
    const int sw = (*k & 3) | ((*k >> 3 & 1) << 2);
    *col = ((p ^ sw) << 4) + (lane & 1) * 8;
  };
  const bool gather_k = MODE == GROUP_DW && a.src != nullptr;
  const char* sa = nullptr;
  const char* sb = nullptr;
  long lda = 0, ldb = 0;
  if constexpr (MODE == GROUP_DX) {
    sa = wg + (size_t)m0 * ES;
    lda = (long)a.d_in * ES;
  } else if constexpr (MODE == GROUP_DW) {
    lda = a.ldx * ES;
    ldb = a.ldy * ES;
    sa = reinterpret_cast<const char*>(a.x) + (gather_k ? 0 : (size_t)row0 * lda) + (size_t)m0 * ES;
    sb = reinterpret_cast<const char*>(a.dy) + (size_t)row0 * ldb + (size_t)n0 * ES;
  }
  // Gathered k rows: a load of this wave covers KR of them.  Their indices come
  // by scalar loads (wave-uniform, counted apart from the loads in flight) a
  // stage ahead of their use.
  constexpr int KR = MODE == GROUP_DW ? 512 / MT : 1, NIDX = OA::NLD * KR;
  int sidx[NIDX], sidx1[NIDX], sidx2[NIDX];     // (the last two at the start only)
  auto want_rows_in = [&](int st, int* sidx) {
    if constexpr (MODE == GROUP_DW) {
      if (!gather_k) return;
      const int k = st * KS + wave * NIDX;
      if (k + NIDX <= K) {
#pragma unroll
        for (int q = 0; q < NIDX; ++q) sidx[q] = sload(a.src, row0 + k + q);
      } else {
#pragma unroll
        for (int q = 0; q < NIDX; ++q) sidx[q] = k + q < K ? sload(a.src, row0 + k + q) : -1;
      }
    }
  };
  auto want_rows = [&](int st) { want_rows_in(st, sidx); };

  // load i of A (B) of stage st
  auto issue_a = [&](int st, char* buf, int i) {
    const int k0 = st * KS;
    const bool live = st < nstage;
    char* to = buf + (wave * OA::NLD + i) * 1024;
    if constexpr (AKC) {
      const int r = (wave * OA::NLD + i) * 8 + (lane >> 3);
      const int c = (lane & 7) ^ ((r >> 1) & 7);
      const bool ok = live && k0 + c * (16 / ES) < K;
      dma16(ra, to, ok ? va[i] : OOB, live ? st * 128u : 0u);
    } else {
      const __amdgpu_buffer_rsrc_t r = make_rsrc(live && !gather_k ? sa + (size_t)k0 * lda : sa, (uint32_t)OOB);
      int k, col;
      strided(MT, i, OA::NLD, &k, &col);
      bool ok = k0 + k < K && m0 + col < mdim;
      int row = k;
      if constexpr (MODE == GROUP_DW) {
        if (gather_k) {
          row = source_row(a, sidx[i * KR]);
#pragma unroll
          for (int q = 1; q < KR; ++q) {
            const int rq = source_row(a, sidx[i * KR + q]);
            row = lane >= q * (64 / KR) ? rq : row;
          }
          ok = ok && row >= 0;
        }
      }
      dma16(r, to, ok ? (uint32_t)row * (uint32_t)lda + col * ES : OOB, 0);
    }
  };
  auto issue_b = [&](int st, char* buf, int i) {
    const int k0 = st * KS;
    const bool live = st < nstage;
    char* to = buf + (wave * OB::NLD + i) * 1024;
    if constexpr (BKC) {
      const int r = (wave * OB::NLD + i) * 8 + (lane >> 3);
      const int c = (lane & 7) ^ ((r >> 1) & 7);
      const bool ok = live && k0 + c * (16 / ES) < K;
      dma16(rb, to, ok ? vb[i] : OOB, live ? st * 128u : 0u);
    } else {
      const __amdgpu_buffer_rsrc_t r = make_rsrc(live ? sb + (size_t)k0 * ldb : sb, (uint32_t)OOB);
      int k, col;
      strided(NT, i, OB::NLD, &k, &col);
      const bool ok = k0 + k < K && n0 + col < ndim;
      dma16(r, to, ok ? (uint32_t)k * (uint32_t)ldb + col * ES : OOB, 0);
    }
  };
  auto issue_all = [&](int st, char* ab, char* bb) {
    if (bb != nullptr) {
#pragma unroll
      for (int i = 0; i < OB::NLD; ++i) issue_b(st, bb, i);
    }
    if (ab != nullptr) {
#pragma unroll
      for (int i = 0; i < OA::NLD; ++i) issue_a(st, ab, i);
    }
  };
  // Ring: A runs three stages ahead and B two, since 160 KB hold no third B: with
  // both two ahead only one stage of loads is in flight (a buffer is free when
  // the next stage has landed), and a stage then takes as long as a trip to
  // memory.  Order of the loads: A0 B0 A1 B1 A2 | B2 A3 | B3 A4 | ...
  want_rows(0);
  want_rows_in(1, sidx1);
  want_rows_in(2, sidx2);
  issue_all(0, ra_[0], nullptr);
  issue_all(0, nullptr, rb_[0]);
#pragma unroll
  for (int q = 0; q < NIDX; ++q) sidx[q] = sidx1[q];
  issue_all(1, ra_[1], nullptr);
  issue_all(1, nullptr, rb_[1]);
#pragma unroll
  for (int q = 0; q < NIDX; ++q) sidx[q] = sidx2[q];
  issue_all(2, ra_[2], nullptr);
  want_rows(3);

  // fragment f (16 rows) of an operand for half h of the stage
  const int kc_at = l16 * 128 + ((lg ^ ((l16 >> 1) & 7)) << 4);
  auto frag_kc = [&](const char* op, int f, int h) {
    return *reinterpret_cast<const u32x4*>(op + f * 2048 + (opaque(kc_at) ^ (h * 64)));
  };
  // (strided: lane j = l16 of a group of 16 points at 4 elements of k row j/4
  // and receives column j of the 4 rows; f0 is the wave's first fragment, a
  // multiple of the fragments it reads, so that only i meets the swizzle)
  const int st_k = 8 * lg + (l16 >> 2);
  const int st_at = ((l16 >> 2) | ((lg & 1) << 2)) << 5 | (l16 & 3) << 3;
  auto frag_st = [&](const char* op, int R, int f0, int i, int h) {
    const char* p = op + (32 * h + st_k) * (2 * R) + ((((f0 + i) & ~7) << 5) + (opaque(st_at) ^ (((f0 + i) & 7) << 5)));
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * 2 * R));
    return __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };

  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // a wave whose part lies past the tile's rows or outputs only loads
  const bool idle = wn * (NT / WN) >= nrow || m0 + wm * (MT / WM) >= mdim;
  if (idle) {
    wait_vm<F8 ? 0 : 2 * OA::NLD + OB::NLD>();
    bar_nofence();
    for (int t = 0; t < nstage; t += 6) {
#pragma unroll
      for (int u = 0; u < 6; ++u) {
        if (t + u >= nstage) break;
        wait_vm<OA::NLD>();
        bar_nofence();
        issue_all(t + u + 2, nullptr, rb_[u % 2]);
        issue_all(t + u + 3, ra_[u % 3], nullptr);
        want_rows(t + u + 4);
      }
    }
    wait_vm<0>();
    return;
  }

  if constexpr (F8) {
    // A stage is one k step of 128, one block of scales: the product of a row
    // i of A's fragments with B comes out of the MFMA by itself and enters the
    // sums times fl32(xs ws).  A's registers hold 4 rows: after row i they take
    // row i + 4; in the last row, B's take the next stage.  The barrier
    // (buffers of stage t free, stage t + 1 landed) follows row FM - 4.
    static_assert(!F8 || (MT / WM <= 128 && 128 % (MT / WM) == 0), "wave inside a scale block");
    constexpr int RA = FM < 4 ? FM : 4;           // rows of A in registers
    constexpr int RB = FM - RA;                   // the row with the barrier
    const int nkb = (a.d_in + 127) >> 7;
    // scale of this lane's row for each n fragment, and of the wave's outputs
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(
        a.src != nullptr ? a.xs : a.xs + (size_t)row0 * nkb, (uint32_t)OOB);
    uint32_t xo[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int n = wn * (NT / WN) + 16 * j + l16;
      int row = n < nrow ? n : -1;
      if (row >= 0 && a.src != nullptr) row = source_row(a, a.src[row0 + n]);
      xo[j] = row >= 0 ? (uint32_t)row * nkb * 4u : OOB;
    }
    const int ob = min((m0 + wm * (MT / WM)) >> 7, ((a.d_out + 127) >> 7) - 1);
    const float* wsp = a.ws + ((size_t)g * ((a.d_out + 127) >> 7) + ob) * nkb;
    float xs[2][FN], ws[2];
    auto get_scales = [&](int st, int set) {      // (the last scale again past the end)
      const int k = min(st, nstage - 1);
      ws[set] = __builtin_bit_cast(float, sload(reinterpret_cast<const int*>(wsp), k));
#pragma unroll
      for (int j = 0; j < FN; ++j)
        xs[set][j] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, xo[j], k * 4u, 0));
    };
    u32x4 fa[RA][2], fb[FN][2];
    // (both halves of a fragment from one address, 64 bytes apart by the swizzle)
    const int at_a = kc_at + wm * (MT / WM) * 128, at_b = kc_at + wn * (NT / WN) * 128;
    auto get_a = [&](const char* op, int i) {
      const int at = opaque(at_a);
      fa[i % RA][0] = *reinterpret_cast<const u32x4*>(op + i * 2048 + at);
      fa[i % RA][1] = *reinterpret_cast<const u32x4*>(op + i * 2048 + (at ^ 64));
    };
    auto get_b = [&](const char* op, int j) {
      const int at = opaque(at_b);
      fb[j][0] = *reinterpret_cast<const u32x4*>(op + j * 2048 + at);
      fb[j][1] = *reinterpret_cast<const u32x4*>(op + j * 2048 + (at ^ 64));
    };
    get_scales(0, 0);
    get_scales(1, 1);
    wait_vm<0>();
    bar_nofence();
#pragma unroll
    for (int i = 0; i < RA; ++i) get_a(ra_[0], i);
#pragma unroll
    for (int j = 0; j < FN; ++j) get_b(rb_[0], j);
    for (int t = 0; t < nstage; t += 6) {
#pragma unroll
      for (int u = 0; u < 6; ++u) {
        if (t + u >= nstage) break;
        float sc[FN];
#pragma unroll
        for (int j = 0; j < FN; ++j) sc[j] = xs[u % 2][j] * ws[u % 2];
#pragma unroll
        for (int i = 0; i < FM; ++i) {
#pragma unroll
          for (int j = 0; j < FN; ++j) {
            const f32x4 p = mfma_e4m3(fa[i % RA][0], fa[i % RA][1], fb[j][0], fb[j][1]);
            if (i == FM - 1) get_b(rb_[(u + 1) % 2], j);
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[i][j][v] = __builtin_fmaf(p[v], sc[j], acc[i][j][v]);
          }
          if (i == RB) {
            __builtin_amdgcn_sched_barrier(0);
            wait_lgkm0();
            wait_vm<OA::NLD>();
            bar_nofence();
            __builtin_amdgcn_sched_barrier(0);
            get_scales(t + u + 2, u % 2);
          }
          if (i < RB) get_a(ra_[u % 3], i + RA);
          else get_a(ra_[(u + 1) % 3], i - RB);
          if (i >= RB) {
            constexpr int NI = OA::NLD + OB::NLD;
#pragma unroll
            for (int p = (i - RB) * NI / RA; p < (i - RB + 1) * NI / RA; ++p) {
              if (p < OB::NLD) issue_b(t + u + 2, rb_[u % 2], p);
              else issue_a(t + u + 3, ra_[u % 3], p - OB::NLD);
            }
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
    wait_vm<0>();
  } else {
    // Half a stage is one k step of 32.  A row i of A's fragments meets all of
    // B's in turn; as soon as its MFMAs are issued, its registers take row i of
    // the next half, and B's two sets alternate, so that LDS reads run half a
    // stage ahead of their use.  One barrier a stage, after the first row of
    // the second half: then every wave holds the rest of stage t in registers
    // (its buffers are free), and stage t + 1 has landed (all but the loads of
    // A for stage t + 2).  The loads of a stage are spread over the rows.
    u32x4 fa[FM], fb[2][FN];
    auto get_a = [&](const char* op, int h, int i) {
      fa[i] = AKC ? frag_kc(op + wm * (MT / WM) * 128, i, h) : frag_st(op, MT, wm * FM, i, h);
    };
    auto get_b = [&](const char* op, int h, int j) {
      fb[h][j] = BKC ? frag_kc(op + wn * (NT / WN) * 128, j, h) : frag_st(op, NT, wn * FN, j, h);
    };
    auto row = [&](int h, int i) {
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = mfma_half<T>(fa[i], fb[h][j], acc[i][j]);
    };
    // what follows row i of a half: row i of A and a share of B for half h
    // (B complete by the middle of the rows)
    constexpr int BR = FM > 1 ? (FM + 1) / 2 : 1;
    auto refill = [&](const char* ab, const char* bb, int h, int i) {
      get_a(ab, h, i);
      if (i < BR) {
#pragma unroll
        for (int j = i * FN / BR; j < (i + 1) * FN / BR; ++j) get_b(bb, h, j);
      }
    };
    wait_vm<2 * OA::NLD + OB::NLD>();
    bar_nofence();
#pragma unroll
    for (int i = 0; i < FM; ++i) refill(ra_[0], rb_[0], 0, i);
    for (int t = 0; t < nstage; t += 6) {
#pragma unroll
      for (int u = 0; u < 6; ++u) {
        if (t + u >= nstage) break;
#pragma unroll
        for (int i = 0; i < FM; ++i) {
          row(0, i);
          refill(ra_[u % 3], rb_[u % 2], 1, i);
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < FM; ++i) {
          row(1, i);
          if (i == 0) {
            __builtin_amdgcn_sched_barrier(0);
            wait_lgkm0();
            wait_vm<OA::NLD>();
            bar_nofence();
            __builtin_amdgcn_sched_barrier(0);
          }
          refill(ra_[(u + 1) % 3], rb_[(u + 1) % 2], 0, i);
          constexpr int NI = OA::NLD + OB::NLD;
#pragma unroll
          for (int p = i * NI / FM; p < (i + 1) * NI / FM; ++p) {
            if (p < OB::NLD) issue_b(t + u + 2, rb_[u % 2], p);
            else issue_a(t + u + 3, ra_[u % 3], p - OB::NLD);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        want_rows(t + u + 4);
      }
    }
    wait_vm<0>();
  }

  // ---- outputs ----
  // (every lane takes part in the exchange; rows and columns past the end
  // write nothing)
  static_assert(FM % 2 == 0, "fragments are stored in pairs");
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int n = n0 + wn * (NT / WN) + 16 * j + l16;
    const size_t base = MODE == GROUP_DW ? ((size_t)g * a.d_out + n) * a.d_in : (size_t)(row0 + n) * a.ldo;
    const bool have = n - n0 < nrow;
#pragma unroll
    for (int i = 0; i < FM; i += 2) {
      const int m = m0 + wm * (MT / WM) + 16 * i + 8 * lg;
      const int left = have ? mdim - m : 0;
      if (a.out_dtype == 2) store8_32(a, base + m, acc[i][j], acc[i + 1][j], left);
      else if (a.out_dtype == 1) store8_16<true>(a, base + m, acc[i][j], acc[i + 1][j], left);
      else store8_16<false>(a, base + m, acc[i][j], acc[i + 1][j], left);
    }
  }
}

// ---- launch ------------------------------------------------------------------

void group_tile_shape(GroupTile t, int* mt, int* nt) {
  *mt = t == TILE_256x256 ? 256 : 128;
  *nt = t == TILE_256x256 ? 256 : (t == TILE_128x128 ? 128 : 32);
}

long group_tile_grid(const GroupArgs& a, GroupMode mode, GroupTile t) {
  int mt, nt;
  group_tile_shape(t, &mt, &nt);
  const long mdim = mode == GROUP_Y ? a.d_out : a.d_in;
  const long mtile = (mdim + mt - 1) / mt;
  long ntile;
  if (mode == GROUP_DW) {
    return (a.groups * mtile + 7) / 8 * 8 * ((a.d_out + nt - 1) / nt);
  } else if (a.groups == 1) {
    ntile = ((long)a.rows + nt - 1) / nt;
  } else {
    // every group adds at most one tile that is not full
    ntile = (long)a.rows / nt + (a.groups < a.rows ? a.groups : a.rows);
  }
  return (mtile * ntile + 7) / 8 * 8;
}

// Expected tiles of mt x nt (the host does not know the offsets: a group ends
// in the middle of a tile on average, and has one at least).
static double tiles(const GroupArgs& a, GroupMode mode, int mt, int nt) {
  const long mdim = mode == GROUP_Y ? a.d_out : a.d_in;
  const double m = (double)((mdim + mt - 1) / mt);
  if (mode == GROUP_DW) return m * a.groups * ((a.d_out + nt - 1) / nt);
  if (a.groups == 1) return m * (double)(((long)a.rows + nt - 1) / nt);
  const double some = a.groups < a.rows ? a.groups : a.rows;
  const double n = (double)a.rows / nt + 0.5 * some;
  return m * (n > some ? n : some);
}

// The kernel with the least expected time, in us, from what each measured over
// products of 1 .. 64 groups, 32 .. 8192 rows and 256 .. 14336 inputs and
// outputs in bf16 (e4m3 in brackets; a stage is 128 bytes of k; 256 CUs).
// Forward:
//   rows kernels   all operands come through the L2, at 9.5 and 8 TB/s (7, 6)
//   128 x 32       0.42 a stage (0.36) while all workgroups run at once (512),
//                  2 (2.8) times that for each 512 otherwise
//   128 x 128      0.58 a stage (0.75) with one workgroup a CU, 0.68 (1.0) for
//                  each 256 workgroups beyond
//   256 x 256      1.6 a stage (2.6) and round of 256 workgroups, 0.8 (1.25)
//                  when few run; a last round that is not full costs half
// plus 4 to 8 for start and end, and at least the time to read the experts'
// weights: 5.5 TB/s without LDS, 4.6 through it.  Both sides of some borders,
// bf16, us: one group of 64 rows, 4096 -> 4096: 32 x 32 rows kernel 19, 128 x 32
// 30; 128 rows: 35, 30, 128 x 128 41; 1024 rows: 128 x 32 67, 128 x 128 46, 256 x
// 256 80; 290 rows in 3 groups, 5824 -> 640: 32 x 32 rows kernel 25, 128 x 32 41;
// two rows for each of 60 experts, 2048 -> 1408: 16 x 16 rows kernel 56, 128 x 32
// 75; 16 for each of 8, 4096 -> 4096: 92, 42; 24960 rows in 64 ragged groups,
// 2048 -> 1408: 128 x 128 222, 256 x 256 183.
// Input gradient (its A is read by transposing reads, twice as many):
//   128 x 32       as forward
//   128 x 128      0.64 a stage with one workgroup a CU, 0.51 for each 256 beyond
//                  (two a CU cover each other's starts)
//   256 x 256      1.25 a stage and 0.4 more as the round of 256 fills, then 1.65
//                  and 8 for start and end in each round
// Both sides, bf16, us, as 128 x 32, 128 x 128, 256 x 256: d_in and d_out 4096, one
// group of 1 row 29, 43, 74; 512 rows 38, 46, 94; 1024: 69, 51, 95; 2048: 136,
// 73, 100; 4096: 257, 134, 112; 8192: 491, 261, 219; 2048 rows in 8 groups 192,
// 87, 119; 8192 in 8: 610, 290, 252; 64 ragged groups, d_in 2048, d_out 1408,
// 4096 rows: 107, 94, 120; 24960 rows 413, 212, 232 (eight routings of a skewed
// router: 128 x 128 216 .. 228, 256 x 256 203 .. 260, by whether its tiles just fill
// four rounds or start a fifth).  (40 products of 1 .. 79
// groups, 77 .. 24434 rows and 256 .. 8000 inputs and outputs in f16 that the
// constants were not taken from: the choice is the fastest or within 2 % for 36,
// within 14 % for all.)
// Weight gradient, for each round of workgroups that run at once:
//   128 x 128      8 and 1.36 a stage of 64 rows (512 workgroups)
//   256 x 256      8 and 1.7 (256)
// Both sides, bf16, us, as 128 x 128, 256 x 256: 2048 x 2048, one group of 1024
// rows 21, 31; 8192 rows 104, 170; 4096 x 4096, one group of 256 rows 24, 19;
// 16384 rows 660, 423; 2048 rows in 2 groups 97, 72; 8192 in 8: 385, 285; 1024 x
// 2048, 2048 rows in 8 groups 26, 19; 2048 x 1408, 2100 rows in 16 ragged groups 48,
// 42; 24960 in 64: 299, 255.  The host does not know how uneven the groups are: where
// one holds a third of 24960 rows and there are few tiles (64 groups, 1024 x 512),
// its tiles bound the time and the rule is wrong, 81 against 133.
GroupPick choose_group(const GroupArgs& a, GroupMode mode, GroupType type) {
  const bool f8 = type == GROUP_E4M3;
  const double K = mode == GROUP_Y ? a.d_in : (mode == GROUP_DX ? a.d_out : (double)a.rows / a.groups);
  const double stages = mode == GROUP_DW ? K / 64 + 1 : (double)(long)((K * (f8 ? 1 : 2) + 127) / 128);
  GroupPick best{false, ROWS_16x16, TILE_256x256};
  double least = 0;
  auto offer = [&](const GroupPick& p, double us) {
    if (least == 0 || us < least) {
      best = p;
      least = us;
    }
  };
  const double g256 = tiles(a, mode, 256, 256), g128 = tiles(a, mode, 128, 128);
  const double r256 = g256 / 256;
  if (mode == GROUP_DW) {
    // each tile starts and ends by itself: 8 us a round
    const auto up = [](double v) { return (double)(long)(v + 0.999); };
    offer({false, ROWS_16x16, TILE_256x256}, up(r256) * (8 + 1.7 * stages));
    offer({false, ROWS_16x16, TILE_128x128}, up(g128 / 512) * (8 + 1.36 * stages));
    return best;
  }
  const double weights = (double)(a.groups < a.rows ? a.groups : a.rows) * a.d_in * a.d_out * (f8 ? 1 : 2);
  const auto least_of = [](double us, double memory) { return us > memory ? us : memory; };
  const double by_lds = weights / 4.6e6, direct = weights / 5.5e6;
  if (mode == GROUP_DX) {
    offer({false, ROWS_16x16, TILE_256x256},
          least_of(r256 <= 1 ? 8 + stages * (1.25 + 0.4 * r256) : 8 * r256 + stages * 1.65 * (r256 + 0.25), by_lds + 8));
    offer({false, ROWS_16x16, TILE_128x128},
          least_of(8 + stages * (g128 <= 256 ? 0.64 : 0.51 * g128 / 256), by_lds + 4));
  } else {
    offer({false, ROWS_16x16, TILE_256x256},
          least_of(8 + stages * (r256 <= 1 ? (f8 ? 1.25 : 0.8) * (1 + r256) : (f8 ? 2.6 : 1.6) * (r256 + 0.5)), by_lds + 8));
    offer({false, ROWS_16x16, TILE_128x128},
          least_of(8 + stages * (g128 <= 256 ? (f8 ? 0.75 : 0.58) : (f8 ? 1.0 : 0.68) * g128 / 256), by_lds + 4));
  }
  const double g32 = tiles(a, mode, 128, 32) / 512;
  offer({false, ROWS_16x16, TILE_128x32},
        least_of(6 + stages * (f8 ? 0.36 : 0.42) * (g32 <= 1 ? 1 : (f8 ? 2.8 : 2) * g32), by_lds));
  if (mode == GROUP_Y) {
    const double row = (double)a.d_in * (f8 ? 1 : 2), avg = (double)a.rows / a.groups;
    const double n16 = avg < 16 ? avg : 16, n32 = avg < 32 ? avg : 32;     // rows that a tile reads
    offer({true, ROWS_16x16, TILE_256x256},
          least_of(4 + tiles(a, mode, 16, 16) * (16 + n16) * row / (f8 ? 7e6 : 9.5e6), direct));
    offer({true, ROWS_32x32, TILE_256x256},
          least_of(4 + tiles(a, mode, 32, 32) * (32 + n32) * row / (f8 ? 6e6 : 8e6), direct));
  }
  return best;
}

template <typename T, int MODE, int MT, int NT, int WM, int WN>
static void go(const GroupArgs& a, long grid, hipStream_t s) {
  hipLaunchKernelGGL((group_tile_kernel<T, MODE, MT, NT, WM, WN>), dim3((unsigned)grid),
                     dim3(64 * WM * WN), 0, s, a);
}

template <typename T, int MODE>
static void go_tile(const GroupArgs& a, GroupTile t, long grid, hipStream_t s) {
  if (t == TILE_256x256) go<T, MODE, 256, 256, 2, 4>(a, grid, s);
  else if (t == TILE_128x128 || MODE == GROUP_DW) go<T, MODE, 128, 128, 2, 2>(a, grid, s);
  else if constexpr (MODE != GROUP_DW) go<T, MODE, 128, 32, 4, 1>(a, grid, s);
}

void launch_group_tile(const GroupArgs& a, GroupMode mode, GroupType type, GroupTile t, hipStream_t s) {
  const long grid = group_tile_grid(a, mode, t);
  if (grid <= 0) return;
  if (type == GROUP_E4M3) {
    go_tile<e4m3_t, GROUP_Y>(a, t, grid, s);
  } else if (type == GROUP_F16) {
    if (mode == GROUP_Y) go_tile<half_t, GROUP_Y>(a, t, grid, s);
    else if (mode == GROUP_DX) go_tile<half_t, GROUP_DX>(a, t, grid, s);
    else go_tile<half_t, GROUP_DW>(a, t, grid, s);
  } else {
    if (mode == GROUP_Y) go_tile<__bf16, GROUP_Y>(a, t, grid, s);
    else if (mode == GROUP_DX) go_tile<__bf16, GROUP_DX>(a, t, grid, s);
    else go_tile<__bf16, GROUP_DW>(a, t, grid, s);
  }
}

}  // namespace tq
