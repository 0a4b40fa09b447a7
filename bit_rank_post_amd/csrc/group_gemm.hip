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
// with the LDS destination in a ring of NBUF buffers.  Rows and k past the
// group, the matrix or the row are never read: their lanes get an offset out
// of the buffer's range, which loads zeros.  Groups are found from `off` in
// the kernel (no host read back); offsets are clamped to 0 .. rows, so no
// content of `off` or `src` leads to an access outside the arrays.
#include "group_gemm.h"
#include "tq_device.h"

namespace tq {

struct e4m3_t { uint8_t v; };

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

template <typename T> struct Elem { static constexpr int BYTES = 2; };
template <> struct Elem<e4m3_t> { static constexpr int BYTES = 1; };

// 16 elements of k for 16 rows of the A or B operand of one stage half: the
// 16 bytes of each lane.  16-bit: the operand of one 16x16x32 MFMA.  8-bit:
// two of them make the operand of one 16x16x128 MFMA (which 32 bytes of k a
// lane holds is free, as long as A and B agree).
template <typename T>
__device__ __forceinline__ f32x4 mfma_half(u32x4 a, u32x4 b, f32x4 c) {
  typedef typename Vec8<T>::type V8;
  return mfma16(__builtin_bit_cast(V8, a), __builtin_bit_cast(V8, b), c);
}

// The 8-bit matrix instructions add 8 neighbouring products at a time, each
// cut at 2^-13 of the power of two below the largest of the 8 (measured: a
// product 2^-14 of its neighbour is lost, 2^-13 is kept, across eights all is
// kept in f32).  That is the one rounding below 32 bits here: about 2^-16 of a
// result of random values, against 2^-9 of its rounding to bf16; the way
// around it, exact conversion to f16 and 16-bit MFMA, runs at half the rate.
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
  for (int i = 0; i < 4; ++i)
    h[i] = a.out_dtype == 0 ? __builtin_bit_cast(uint16_t, (half_t)v[i])
                            : __builtin_bit_cast(uint16_t, (__bf16)v[i]);
  uint16_t* p = reinterpret_cast<uint16_t*>(a.out) + at;
  if (a.vec_out && left >= 4)
    *reinterpret_cast<u32x2*>(p) = u32x2{h[0] | ((uint32_t)h[1] << 16), h[2] | ((uint32_t)h[3] << 16)};
  else
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) p[i] = h[i];
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

template <typename T, int MODE, int MT, int NT, int WM, int WN, int NBUF>
__global__ __launch_bounds__(64 * WM * WN) void group_tile_kernel(GroupArgs a) {
  constexpr bool F8 = sizeof(T) == 1;
  constexpr bool AKC = MODE == GROUP_Y, BKC = MODE != GROUP_DW;
  constexpr int ES = Elem<T>::BYTES;
  constexpr int KS = 128 / ES;                  // k per stage
  constexpr int WAVES = WM * WN, NTHR = 64 * WAVES;
  constexpr int FM = MT / WM / 16, FN = NT / WN / 16;
  typedef Operand<AKC, MT, NTHR> OA;
  typedef Operand<BKC, NT, NTHR> OB;
  constexpr int SB = OA::BYTES + OB::BYTES;
  static_assert(NBUF * SB <= 160 * 1024, "LDS budget");
  static_assert(AKC || MT >= 128, "strided tile rows hold 8 pieces");
  static_assert(BKC || NT >= 128, "strided tile rows hold 8 pieces");
  // one array per buffer: the compiler then knows that the loads in flight do
  // not touch the buffer being read (with one array it waits for all of them)
  __shared__ __attribute__((aligned(128))) char s0[SB];
  __shared__ __attribute__((aligned(128))) char s1[SB];
  __shared__ __attribute__((aligned(128))) char s2[NBUF > 2 ? SB : 16];
  char* const ring[3] = {s0, s1, s2};

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
    int it, m;
    if (!take_item(a.groups * ntile, mtile, &it, &m)) return;
    g = it / ntile;
    n0 = (it - g * ntile) * NT;
    m0 = m * MT;
    int lo, hi;
    group_span(a, g, &lo, &hi);
    row0 = __builtin_amdgcn_readfirstlane(lo);
    K = __builtin_amdgcn_readfirstlane(hi - lo);
    nrow = min(NT, ndim - n0);
  } else {
    mdim = MODE == GROUP_Y ? a.d_out : a.d_in;
    K = MODE == GROUP_Y ? a.d_in : a.d_out;
    const int mtile = (mdim + MT - 1) / MT;
    const int ntile = count_row_tiles<NT>(a, lane);
    int it, m;
    if (!take_item(ntile, mtile, &it, &m)) return;
    find_row_tile<NT>(a, lane, it, &g, &row0, &nrow);
    g = __builtin_amdgcn_readfirstlane(g);
    row0 = __builtin_amdgcn_readfirstlane(row0);
    nrow = __builtin_amdgcn_readfirstlane(nrow);
    m0 = m * MT;
    n0 = 0;
    if (nrow <= 0) return;
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
  // indices of the gathered k rows, requested one stage ahead of their loads
  int sidx[OA::NLD];
  auto want_rows = [&](int st) {
    if constexpr (MODE == GROUP_DW) {
      if (gather_k) {
#pragma unroll
        for (int i = 0; i < OA::NLD; ++i) {
          int k, col;
          strided(MT, i, OA::NLD, &k, &col);
          const int r = st * KS + k;
          sidx[i] = r < K ? a.src[row0 + r] : -1;
        }
      }
    }
  };

  auto issue = [&](int st, char* buf) {
    const int k0 = st * KS;
    const bool live = st < nstage;
    if constexpr (AKC) {
#pragma unroll
      for (int i = 0; i < OA::NLD; ++i) {
        const int r = (wave * OA::NLD + i) * 8 + (lane >> 3);
        const int c = (lane & 7) ^ ((r >> 1) & 7);
        const bool ok = live && k0 + c * (16 / ES) < K;
        dma16(ra, buf + (wave * OA::NLD + i) * 1024, ok ? va[i] : OOB, live ? st * 128u : 0u);
      }
    } else {
      const __amdgpu_buffer_rsrc_t r = make_rsrc(
          live && !gather_k ? sa + (size_t)k0 * lda : sa, (uint32_t)OOB);
#pragma unroll
      for (int i = 0; i < OA::NLD; ++i) {
        int k, col;
        strided(MT, i, OA::NLD, &k, &col);
        bool ok = k0 + k < K && m0 + col < mdim;
        int row = k;
        if constexpr (MODE == GROUP_DW) {
          if (gather_k) {
            row = source_row(a, sidx[i]);
            ok = ok && row >= 0;
          }
        }
        dma16(r, buf + (wave * OA::NLD + i) * 1024, ok ? (uint32_t)row * (uint32_t)lda + col * ES : OOB, 0);
      }
    }
    char* bb = buf + OA::BYTES;
    if constexpr (BKC) {
#pragma unroll
      for (int i = 0; i < OB::NLD; ++i) {
        const int r = (wave * OB::NLD + i) * 8 + (lane >> 3);
        const int c = (lane & 7) ^ ((r >> 1) & 7);
        const bool ok = live && k0 + c * (16 / ES) < K;
        dma16(rb, bb + (wave * OB::NLD + i) * 1024, ok ? vb[i] : OOB, live ? st * 128u : 0u);
      }
    } else {
      const __amdgpu_buffer_rsrc_t r = make_rsrc(live ? sb + (size_t)k0 * ldb : sb, (uint32_t)OOB);
#pragma unroll
      for (int i = 0; i < OB::NLD; ++i) {
        int k, col;
        strided(NT, i, OB::NLD, &k, &col);
        const bool ok = k0 + k < K && n0 + col < ndim;
        dma16(r, bb + (wave * OB::NLD + i) * 1024, ok ? (uint32_t)k * (uint32_t)ldb + col * ES : OOB, 0);
      }
    }
    want_rows(st + 1);
  };

  // fragment f (16 rows) of an operand for half h of the stage
  const int kc_at = l16 * 128 + ((lg ^ ((l16 >> 1) & 7)) << 4);
  auto frag_kc = [&](const char* op, int f, int h) {
    return *reinterpret_cast<const u32x4*>(op + f * 2048 + (kc_at ^ (h * 64)));
  };
  auto frag_st = [&](const char* op, int R, int f, int h) {
    const int j = l16, k = 32 * h + 8 * lg + (j >> 2);
    const int sw = (j >> 2) | ((lg & 1) << 2);
    const char* p = op + k * (2 * R) + ((f ^ sw) << 5) + (j & 3) * 8;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * 2 * R));
    return __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };

  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // 8-bit operands: scales of this lane's rows (one per n fragment) and of
  // the wave's 128-output block, for k block st
  const int nkb = (a.d_in + 127) >> 7;
  const float* xsp[FN];
  const float* wsp = nullptr;
  if constexpr (F8) {
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int n = wn * (NT / WN) + 16 * j + l16;
      int row = n < nrow ? row0 + n : -1;
      if (row >= 0 && a.src != nullptr) row = source_row(a, a.src[row]);
      xsp[j] = row >= 0 ? a.xs + (size_t)row * nkb : nullptr;
    }
    // a wave's outputs lie in one block of 128
    static_assert(!F8 || (MT / WM <= 128 && 128 % (MT / WM) == 0), "wave inside a scale block");
    const int ob = min((m0 + wm * (MT / WM)) >> 7, ((a.d_out + 127) >> 7) - 1);
    wsp = a.ws + ((size_t)g * ((a.d_out + 127) >> 7) + ob) * nkb;
  }

  auto compute = [&](const char* buf, int st) {
    const char* pa = buf + (AKC ? wm * (MT / WM) * 128 : 0);
    const char* pb = buf + OA::BYTES + (BKC ? wn * (NT / WN) * 128 : 0);
    if constexpr (F8) {
      float sc[FN];
      const float w = wsp[st];
#pragma unroll
      for (int j = 0; j < FN; ++j) sc[j] = xsp[j] != nullptr ? xsp[j][st] * w : 0.f;
      u32x4 b0[FN], b1[FN];
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        b0[j] = frag_kc(pb, j, 0);
        b1[j] = frag_kc(pb, j, 1);
      }
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const u32x4 a0 = frag_kc(pa, i, 0), a1 = frag_kc(pa, i, 1);
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const f32x4 p = mfma_e4m3(a0, a1, b0[j], b1[j]);
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[i][j][v] = __builtin_fmaf(p[v], sc[j], acc[i][j][v]);
        }
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        u32x4 fa[FM], fb[FN];
#pragma unroll
        for (int j = 0; j < FN; ++j)
          fb[j] = BKC ? frag_kc(pb, j, h) : frag_st(pb, NT, wn * FN + j, h);
#pragma unroll
        for (int i = 0; i < FM; ++i)
          fa[i] = AKC ? frag_kc(pa, i, h) : frag_st(pa, MT, wm * FM + i, h);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j) acc[i][j] = mfma_half<T>(fa[i], fb[j], acc[i][j]);
      }
    }
  };

  // ring: stage t + NBUF - 1 is requested as soon as every wave is done with
  // the buffer it goes to (that of stage t - 1); whole rounds always run,
  // stages past the end only wait and request nothing
  want_rows(0);
#pragma unroll
  for (int b = 0; b < NBUF - 1; ++b) issue(b, ring[b]);
  for (int t = 0; t < nstage; t += NBUF) {
#pragma unroll
    for (int u = 0; u < NBUF; ++u) {
      wait_vm<(NBUF - 2) * (OA::NLD + OB::NLD)>();
      wait_lgkm0();
      bar_nofence();
      issue(t + u + NBUF - 1, ring[(u + NBUF - 1) % NBUF]);
      if (t + u < nstage) compute(ring[u], t + u);
    }
  }
  wait_vm<0>();

  // ---- outputs ----
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int n = n0 + wn * (NT / WN) + 16 * j + l16;
    if (n - n0 >= nrow) continue;
    const size_t base = MODE == GROUP_DW ? ((size_t)g * a.d_out + n) * a.d_in : (size_t)(row0 + n) * a.ldo;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int m = m0 + wm * (MT / WM) + 16 * i + 4 * lg;
      if (m < mdim) store4(a, base + m, acc[i][j], mdim - m);
    }
  }
}

// ---- launch ------------------------------------------------------------------

static void tile_shape(GroupTile t, int* mt, int* nt) {
  *mt = t == TILE_256x256 ? 256 : 128;
  *nt = t == TILE_256x256 ? 256 : (t == TILE_128x128 ? 128 : 32);
}

long group_tile_grid(const GroupArgs& a, GroupMode mode, GroupTile t) {
  int mt, nt;
  tile_shape(t, &mt, &nt);
  const long mdim = mode == GROUP_Y ? a.d_out : a.d_in;
  const long mtile = (mdim + mt - 1) / mt;
  long ntile;
  if (mode == GROUP_DW) {
    ntile = (long)a.groups * ((a.d_out + nt - 1) / nt);
  } else if (a.groups == 1) {
    ntile = ((long)a.rows + nt - 1) / nt;
  } else {
    // every group adds at most one tile that is not full
    ntile = (long)a.rows / nt + (a.groups < a.rows ? a.groups : a.rows);
  }
  return (mtile * ntile + 7) / 8 * 8;
}

GroupTile choose_group_tile(const GroupArgs& a, GroupMode mode, GroupType) {
  const long avg = a.rows / a.groups;
  if (mode != GROUP_DW && avg <= 48) return TILE_128x32;
  if (mode != GROUP_DW && avg < 512) return TILE_128x128;
  return group_tile_grid(a, mode, TILE_256x256) >= 256 ? TILE_256x256 : TILE_128x128;
}

template <typename T, int MODE, int MT, int NT, int WM, int WN, int NBUF>
static void go(const GroupArgs& a, long grid, hipStream_t s) {
  hipLaunchKernelGGL((group_tile_kernel<T, MODE, MT, NT, WM, WN, NBUF>), dim3((unsigned)grid),
                     dim3(64 * WM * WN), 0, s, a);
}

template <typename T, int MODE>
static void go_tile(const GroupArgs& a, GroupTile t, long grid, hipStream_t s) {
  if (t == TILE_256x256) go<T, MODE, 256, 256, 2, 4, 2>(a, grid, s);
  else if (t == TILE_128x128 || MODE == GROUP_DW) go<T, MODE, 128, 128, 2, 2, 2>(a, grid, s);
  else if constexpr (MODE != GROUP_DW) go<T, MODE, 128, 32, 4, 1, 3>(a, grid, s);
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
