// C ABI of the operators around a layer of experts (include/tileq.h): products
// grouped by expert, 8-bit products with block scales, norms around a block.
// Every check runs on the host before any launch; the calls only enqueue
// kernels on the caller's stream.
#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "group_gemm.h"
#include "norm_ops.h"
#include "tileq.h"
#include "tq_internal.h"

using namespace tq;

namespace {

tq_status fail(tq_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  set_last_error(buf);
  return st;
}

#define TRY(expr)                       \
  do {                                  \
    const tq_status st_ = (expr);       \
    if (st_ != TQ_OK) return st_;       \
  } while (0)

bool is_float(tq_dtype t) { return t == TQ_F16 || t == TQ_BF16 || t == TQ_F32; }
size_t size_of(tq_dtype t) { return t == TQ_F32 ? 4 : 2; }
bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

tq_status launched() {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(TQ_EHIP, "launch failed: %s", hipGetErrorString(e));
  return TQ_OK;
}

// ---- grouped products --------------------------------------------------------

// a workgroup of 512 threads at most; HIP counts a grid's threads in 32 bits
constexpr long GRID_MAX = 0xFFFFFFFFL / 512 / 8 * 8;

tq_status check_group(const tq_group_desc* d, bool e4m3, GroupMode mode, tq_dtype out_dtype, GroupArgs* a) {
  if (!d) return fail(TQ_EINVAL, "descriptor is NULL");
  if (!e4m3 && d->act != TQ_F16 && d->act != TQ_BF16) return fail(TQ_EINVAL, "act must be TQ_F16 or TQ_BF16");
  if (!is_float(out_dtype)) return fail(TQ_EINVAL, "unknown output dtype %d", (int)out_dtype);
  if (d->groups < 1 || d->groups > 1024) return fail(TQ_ESHAPE, "groups = %d outside [1, 1024]", d->groups);
  if (d->rows < 0) return fail(TQ_ESHAPE, "rows = %d", d->rows);
  if (d->rows > 1 << 30) return fail(TQ_EUNSUPPORTED, "rows = %d > 2^30", d->rows);
  const int step = e4m3 ? 16 : 8;
  if (d->d_in < step || d->d_in % step)
    return fail(TQ_ESHAPE, "d_in = %d must be a positive multiple of %d", d->d_in, step);
  if (d->d_out < 1) return fail(TQ_ESHAPE, "d_out = %d", d->d_out);
  if (mode != GROUP_Y && d->d_out % 8)
    return fail(TQ_ESHAPE, "d_out = %d must be a multiple of 8 for the gradients", d->d_out);
  if (d->groups > 1 && !d->off) return fail(TQ_EINVAL, "off is NULL with %d groups", d->groups);
  a->groups = d->groups;
  a->rows = d->rows;
  a->d_in = d->d_in;
  a->d_out = d->d_out;
  a->off = d->off;
  a->ldx = d->ldx ? d->ldx : d->d_in;
  a->ldy = d->ldy ? d->ldy : d->d_out;
  if (a->ldx < d->d_in) return fail(TQ_ESHAPE, "ldx = %ld < d_in = %d", a->ldx, d->d_in);
  if (a->ldy < d->d_out) return fail(TQ_ESHAPE, "ldy = %ld < d_out = %d", a->ldy, d->d_out);
  // rows of a tile are addressed with 32-bit offsets
  if (a->ldx > (1 << 21) || a->ldy > (1 << 21))
    return fail(TQ_EUNSUPPORTED, "row stride of more than 2^21 elements");
  const bool reads_x = mode != GROUP_DX, reads_dy = mode != GROUP_Y;
  if (reads_x && a->ldx % step) return fail(TQ_ESHAPE, "ldx = %ld must be a multiple of %d", a->ldx, step);
  if (reads_dy && a->ldy % 8) return fail(TQ_ESHAPE, "ldy = %ld must be a multiple of 8", a->ldy);
  a->src = nullptr;
  a->x_rows = d->rows;
  a->div_mul = 0;
  a->div_shift = -1;
  if (d->src && mode == GROUP_DX) return fail(TQ_EINVAL, "the input gradient takes no src (one row per grouped row)");
  if (d->src) {
    if (d->src_div < 1) return fail(TQ_ESHAPE, "src_div = %d", d->src_div);
    if (d->x_rows < 0) return fail(TQ_ESHAPE, "x_rows = %d", d->x_rows);
    const long bytes = (long)d->x_rows * a->ldx * (e4m3 ? 1 : 2);
    if (bytes >= 0x7FFFFFF0L)
      return fail(TQ_EUNSUPPORTED, "gathered x of %ld bytes >= 2^31", bytes);
    a->src = d->src;
    a->x_rows = d->x_rows;
    if (d->src_div > 1) {
      // floor(v / div) for v < 2^31 is (v ceil(2^(31+l) / div)) >> (31+l), 2^l >= div
      int l = 0;
      while ((1LL << l) < d->src_div) ++l;
      a->div_mul = (uint32_t)((((unsigned long long)1 << (31 + l)) + d->src_div - 1) / d->src_div);
      a->div_shift = l - 1;
    }
  }
  a->out_dtype = (int)out_dtype;
  return TQ_OK;
}

tq_status check_apart(const void* out, const void* a, const void* b) {
  if (out && (out == a || out == b)) return fail(TQ_EINVAL, "the output is one of the operands");
  return TQ_OK;
}

// the stride and alignment rule of 16-byte stores
void set_out(GroupArgs* a, void* out, long ldo) {
  a->out = out;
  a->ldo = ldo;
  a->vec_out = ldo % (a->out_dtype == 2 ? 4 : 8) == 0 && aligned(out, 16) ? 1 : 0;
}

// the kernel for a product and its workgroups
tq_status pick_group(const GroupArgs& a, GroupMode mode, GroupType type, GroupPick* p) {
  *p = choose_group(a, mode, type);
  // (HIP counts a launch's threads in 32 bits; rows kernels have up to 1024)
  if (p->rows && group_rows_grid(a, p->shape) > GRID_MAX / 2) *p = {false, p->shape, TILE_128x32};
  if (p->rows) return TQ_OK;
  if (group_tile_grid(a, mode, p->tile) > GRID_MAX) p->tile = TILE_256x256;
  const long grid = group_tile_grid(a, mode, p->tile);
  if (grid > GRID_MAX)
    return fail(TQ_EUNSUPPORTED, "%ld workgroups: more than one launch takes", grid);
  return TQ_OK;
}

tq_status run_group(const GroupArgs& a, GroupMode mode, GroupType type, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  GroupPick p;
  TRY(pick_group(a, mode, type, &p));
  if (p.rows) launch_group_rows(a, type, p.shape, s);
  else launch_group_tile(a, mode, type, p.tile, s);
  return launched();
}

// ---- norms -------------------------------------------------------------------

// one operand of rows: present or not, its stride, its alignment
tq_status check_rows(const tq_rows& r, const char* name, bool need, int d, tq_dtype t, long* ld) {
  *ld = d;
  if (!r.p) return need ? fail(TQ_EINVAL, "%s is NULL", name) : TQ_OK;
  *ld = r.ld ? r.ld : d;
  const int step = t == TQ_F32 ? 4 : 8;
  if (*ld < d || *ld % step)
    return fail(TQ_ESHAPE, "row stride %ld of %s must be a multiple of %d and at least d", *ld, name, step);
  if (!aligned(r.p, 16)) return fail(TQ_EINVAL, "%s not 16-byte aligned", name);
  return TQ_OK;
}

// An output in place of an input: its rows must lie where the input's do, or a
// row is written while another, not yet read, lies there.
tq_status check_in_place(const tq_rows& out, long ldo, const char* out_name, const tq_rows& in, long ldi,
                         const char* in_name, int T) {
  if (T > 1 && out.p && out.p == in.p && ldo != ldi)
    return fail(TQ_EINVAL, "%s in place of %s with another row stride (%ld, %ld)", out_name, in_name, ldo, ldi);
  return TQ_OK;
}

tq_status check_norm(int T, int d, tq_dtype st, tq_dtype act, tq_dtype w, int gate, float alpha) {
  if (T < 0) return fail(TQ_ESHAPE, "T = %d", T);
  if (d < 8 || d % 8 || d > NORM_D_MAX)
    return fail(TQ_ESHAPE, "d = %d must be a multiple of 8 from 8 to %d", d, NORM_D_MAX);
  if (!is_float(st) || !is_float(act) || !is_float(w)) return fail(TQ_EINVAL, "unknown dtype");
  if (gate < TQ_GATE_NONE || gate > TQ_GATE_FULL) return fail(TQ_EINVAL, "unknown gate kind %d", gate);
  if (!std::isfinite(alpha)) return fail(TQ_EINVAL, "alpha is not finite");
  return TQ_OK;
}

tq_status check_gate(const tq_rows& g, const char* name, int gate, int d, tq_dtype act, bool need, long* ld) {
  if (gate == TQ_GATE_FULL) return check_rows(g, name, need, d, act, ld);
  *ld = g.ld ? g.ld : 1;
  if (gate == TQ_GATE_TOKEN && need && !g.p) return fail(TQ_EINVAL, "%s is NULL", name);
  if (gate == TQ_GATE_TOKEN && *ld < 1) return fail(TQ_ESHAPE, "stride %ld of %s", *ld, name);
  if (gate == TQ_GATE_TOKEN && !aligned(g.p, 4)) return fail(TQ_EINVAL, "%s not 4-byte aligned", name);
  return TQ_OK;
}

tq_status check_vec(const void* p, const char* name) {
  if (!aligned(p, 16)) return fail(TQ_EINVAL, "%s not 16-byte aligned", name);
  return TQ_OK;
}

tq_status check_norm_forward(const tq_norm_desc* d, NormArgs* a) {
  if (!d) return fail(TQ_EINVAL, "descriptor is NULL");
  TRY(check_norm(d->T, d->d, d->stream_dtype, d->act, d->w_dtype, d->gate, d->alpha));
  if (!(d->eps >= 0.f) || !std::isfinite(d->eps)) return fail(TQ_EINVAL, "eps must be finite and >= 0");
  const bool has_b = d->b.p != nullptr, has_n = d->n.p != nullptr;
  if (has_b != (d->y.p != nullptr))
    return fail(TQ_EINVAL, "b and y go together (y = x + alpha gate p(b))");
  if (!has_b && !has_n && d->T > 0) return fail(TQ_EINVAL, "neither y nor n is asked for");
  if (!has_b && (d->w_post || d->gate != TQ_GATE_NONE)) return fail(TQ_EINVAL, "w_post and gate need b");
  if (has_n && !d->w_next) return fail(TQ_EINVAL, "w_next is NULL");
  if (d->rstd_post && !d->w_post) return fail(TQ_EINVAL, "rstd_post needs w_post");
  if (d->rstd_next && !has_n) return fail(TQ_EINVAL, "rstd_next needs n");
  TRY(check_rows(d->x, "x", d->T > 0, d->d, d->stream_dtype, &a->ld_x));
  TRY(check_rows(d->y, "y", false, d->d, d->stream_dtype, &a->ld_y));
  TRY(check_rows(d->b, "b", false, d->d, d->act, &a->ld_b));
  TRY(check_rows(d->n, "n", false, d->d, d->act, &a->ld_n));
  TRY(check_in_place(d->y, a->ld_y, "y", d->x, a->ld_x, "x", d->T));
  TRY(check_in_place(d->n, a->ld_n, "n", d->b, a->ld_b, "b", d->T));
  TRY(check_gate(d->gate_v, "gate", d->gate, d->d, d->act, d->T > 0, &a->ld_gate));
  TRY(check_vec(d->w_post, "w_post"));
  TRY(check_vec(d->w_next, "w_next"));
  if (!aligned(d->rstd_post, 4) || !aligned(d->rstd_next, 4)) return fail(TQ_EINVAL, "rstd not 4-byte aligned");
  // one workgroup of up to 1024 threads a row
  if (d->T > 0x3FFFFF) return fail(TQ_EUNSUPPORTED, "T = %d >= 2^22", d->T);
  return TQ_OK;
}

}  // namespace

namespace tq {
tq_status check_norm_residual(const tq_norm_desc* d) {
  NormArgs a{};
  return check_norm_forward(d, &a);
}
}  // namespace tq

extern "C" {

tq_status tq_group_gemm(const tq_group_desc* d, const void* x, const void* w, void* y, tq_dtype y_dtype,
                        void* stream) {
  GroupArgs a{};
  TRY(check_group(d, false, GROUP_Y, y_dtype, &a));
  if (a.rows == 0) return TQ_OK;
  if ((!x && a.x_rows > 0) || !w || !y) return fail(TQ_EINVAL, "NULL buffer");
  if (!aligned(x, 16) || !aligned(w, 16)) return fail(TQ_EINVAL, "x and w must be 16-byte aligned");
  TRY(check_apart(y, x, w));
  a.x = x;
  a.w = w;
  set_out(&a, y, a.ldy);
  return run_group(a, GROUP_Y, d->act == TQ_F16 ? GROUP_F16 : GROUP_BF16, stream);
}

tq_status tq_group_gemm_dx(const tq_group_desc* d, const void* dy, const void* w, void* dx, tq_dtype dx_dtype,
                           void* stream) {
  GroupArgs a{};
  TRY(check_group(d, false, GROUP_DX, dx_dtype, &a));
  if (a.rows == 0) return TQ_OK;
  if (!dy || !w || !dx) return fail(TQ_EINVAL, "NULL buffer");
  if (!aligned(dy, 16) || !aligned(w, 16)) return fail(TQ_EINVAL, "dy and w must be 16-byte aligned");
  TRY(check_apart(dx, dy, w));
  a.dy = dy;
  a.w = w;
  set_out(&a, dx, a.ldx);
  return run_group(a, GROUP_DX, d->act == TQ_F16 ? GROUP_F16 : GROUP_BF16, stream);
}

tq_status tq_group_gemm_dw(const tq_group_desc* d, const void* dy, const void* x, void* dw, tq_dtype dw_dtype,
                           void* stream) {
  GroupArgs a{};
  TRY(check_group(d, false, GROUP_DW, dw_dtype, &a));
  if (!dw) return fail(TQ_EINVAL, "dw is NULL");
  if (a.rows > 0 && (!dy || (!x && a.x_rows > 0))) return fail(TQ_EINVAL, "NULL buffer");
  if (!aligned(dy, 16) || !aligned(x, 16)) return fail(TQ_EINVAL, "dy and x must be 16-byte aligned");
  TRY(check_apart(dw, dy, x));
  a.dy = dy;
  a.x = x;
  set_out(&a, dw, a.d_in);
  return run_group(a, GROUP_DW, d->act == TQ_F16 ? GROUP_F16 : GROUP_BF16, stream);
}

tq_status tq_fp8_gemm(const tq_group_desc* d, const void* x, const float* x_scale, const void* w,
                      const float* w_scale, void* y, tq_dtype y_dtype, void* stream) {
  GroupArgs a{};
  TRY(check_group(d, true, GROUP_Y, y_dtype, &a));
  if (a.rows == 0) return TQ_OK;
  if ((a.x_rows > 0 && (!x || !x_scale)) || !w || !w_scale || !y) return fail(TQ_EINVAL, "NULL buffer");
  if (!aligned(x, 16) || !aligned(w, 16)) return fail(TQ_EINVAL, "x and w must be 16-byte aligned");
  if (!aligned(x_scale, 4) || !aligned(w_scale, 4)) return fail(TQ_EINVAL, "scales must be 4-byte aligned");
  TRY(check_apart(y, x, w));
  a.x = x;
  a.w = w;
  a.xs = x_scale;
  a.ws = w_scale;
  set_out(&a, y, a.ldy);
  return run_group(a, GROUP_Y, GROUP_E4M3, stream);
}

tq_status tq_debug_group_kernel(const tq_group_desc* d, int32_t product, int32_t* outputs, int32_t* rows,
                                int32_t* staged) {
  if (product < 0 || product > 3) return fail(TQ_EINVAL, "product = %d outside [0, 3]", product);
  if (!outputs || !rows || !staged) return fail(TQ_EINVAL, "outputs, rows or staged is NULL");
  const bool e4m3 = product == 3;
  const GroupMode mode = product == 1 ? GROUP_DX : product == 2 ? GROUP_DW : GROUP_Y;
  GroupArgs a{};
  TRY(check_group(d, e4m3, mode, TQ_F32, &a));
  GroupPick p;
  TRY(pick_group(a, mode, e4m3 ? GROUP_E4M3 : d->act == TQ_F16 ? GROUP_F16 : GROUP_BF16, &p));
  *staged = p.rows ? 0 : 1;
  if (p.rows) group_rows_shape(p.shape, outputs, rows);
  else group_tile_shape(p.tile, outputs, rows);
  return TQ_OK;
}

tq_status tq_fp8_quant_rows(const void* x, tq_dtype x_dtype, int32_t rows, int32_t d, int64_t ldx, void* q,
                            float* scale, void* stream) {
  if (!is_float(x_dtype)) return fail(TQ_EINVAL, "unknown x_dtype %d", (int)x_dtype);
  if (rows < 0) return fail(TQ_ESHAPE, "rows = %d", rows);
  if (d < 16 || d % 16) return fail(TQ_ESHAPE, "d = %d must be a positive multiple of 16", d);
  const long ld = ldx ? ldx : d;
  if (ld < d || ld % (x_dtype == TQ_F32 ? 4 : 8))
    return fail(TQ_ESHAPE, "ldx = %ld must be at least d and keep rows 16-byte aligned", ld);
  if (rows == 0) return TQ_OK;
  if (!x || !q || !scale) return fail(TQ_EINVAL, "NULL buffer");
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scale, 4)) return fail(TQ_EINVAL, "x and q must be 16-byte aligned");
  if ((long)rows * ((d + 127) / 128) / 16 > 0xFFFFFFFFL / 256 - 1)
    return fail(TQ_EUNSUPPORTED, "%d rows of %d: more than one launch takes", rows, d);
  launch_quant_rows(x, (int)x_dtype, rows, d, ld, q, scale, reinterpret_cast<hipStream_t>(stream));
  return launched();
}

tq_status tq_fp8_quant_blocks(const void* w, tq_dtype w_dtype, int32_t groups, int32_t d_out, int32_t d_in,
                              void* q, float* scale, void* stream) {
  if (!is_float(w_dtype)) return fail(TQ_EINVAL, "unknown w_dtype %d", (int)w_dtype);
  if (groups < 1 || d_out < 1) return fail(TQ_ESHAPE, "groups = %d, d_out = %d", groups, d_out);
  if (d_in < 16 || d_in % 16) return fail(TQ_ESHAPE, "d_in = %d must be a positive multiple of 16", d_in);
  if (!w || !q || !scale) return fail(TQ_EINVAL, "NULL buffer");
  if (!aligned(w, 16) || !aligned(q, 16) || !aligned(scale, 4)) return fail(TQ_EINVAL, "w and q must be 16-byte aligned");
  if ((double)groups * ((d_out + 127) / 128) * ((d_in + 127) / 128) > 0xFFFFFFFFL / 256 - 1)
    return fail(TQ_EUNSUPPORTED, "%d matrices of %d x %d: more than one launch takes", groups, d_out, d_in);
  launch_quant_blocks(w, (int)w_dtype, groups, d_out, d_in, q, scale, reinterpret_cast<hipStream_t>(stream));
  return launched();
}

tq_status tq_norm_residual(const tq_norm_desc* d, void* stream) {
  NormArgs a{};
  TRY(check_norm_forward(d, &a));
  if (d->T == 0) return TQ_OK;
  a.T = d->T;
  a.d = d->d;
  a.wdt = (int)d->w_dtype;
  a.gate = d->gate;
  a.alpha = d->alpha;
  a.eps = d->eps;
  a.x = d->x.p;
  a.b = d->b.p;
  a.y = d->y.p;
  a.n = d->n.p;
  a.w_post = d->w_post;
  a.w_next = d->w_next;
  a.gate_p = d->gate_v.p;
  a.rstd_post = d->rstd_post;
  a.rstd_next = d->rstd_next;
  launch_norm_forward(a, (int)d->stream_dtype, (int)d->act, reinterpret_cast<hipStream_t>(stream));
  return launched();
}

tq_status tq_norm_grad_workspace_size(int32_t T, int32_t d, size_t* bytes) {
  if (!bytes) return fail(TQ_EINVAL, "bytes is NULL");
  TRY(check_norm(T, d, TQ_F32, TQ_F32, TQ_F32, TQ_GATE_NONE, 0.f));
  *bytes = (size_t)2 * norm_parts(T, d) * d * sizeof(float);
  return TQ_OK;
}

tq_status tq_norm_residual_grad(const tq_norm_grad_desc* d, void* ws, size_t ws_bytes, void* stream) {
  if (!d) return fail(TQ_EINVAL, "descriptor is NULL");
  TRY(check_norm(d->T, d->d, d->stream_dtype, d->act, d->w_dtype, d->gate, d->alpha));
  const bool rows = d->T > 0;
  const bool has_b = d->b.p != nullptr, has_dn = d->dn.p != nullptr;
  if (rows && !d->dy.p && !has_dn) return fail(TQ_EINVAL, "neither dy nor dn is given");
  if (has_dn && (!d->y.p || !d->w_next || !d->rstd_next))
    return fail(TQ_EINVAL, "dn needs y, w_next and rstd_next");
  if (rows && !has_b && (d->w_post || d->db.p || d->dw_post || d->dgate.p || d->gate != TQ_GATE_NONE))
    return fail(TQ_EINVAL, "w_post, gate, db, dw_post and dgate need b");
  if (d->w_post && rows && !d->rstd_post) return fail(TQ_EINVAL, "w_post needs rstd_post");
  if (d->dw_post && !d->w_post) return fail(TQ_EINVAL, "dw_post needs w_post");
  if (d->dw_next && rows && !has_dn) return fail(TQ_EINVAL, "dw_next needs dn");
  if (d->dgate.p && d->gate == TQ_GATE_NONE) return fail(TQ_EINVAL, "dgate needs a gate");
  NormArgs a{};
  TRY(check_rows(d->y, "y", false, d->d, d->stream_dtype, &a.ld_y));
  TRY(check_rows(d->dy, "dy", false, d->d, d->stream_dtype, &a.ld_dy));
  TRY(check_rows(d->dx, "dx", false, d->d, d->stream_dtype, &a.ld_dx));
  TRY(check_rows(d->dn, "dn", false, d->d, d->act, &a.ld_dn));
  TRY(check_rows(d->b, "b", false, d->d, d->act, &a.ld_b));
  TRY(check_rows(d->db, "db", false, d->d, d->act, &a.ld_db));
  TRY(check_in_place(d->dx, a.ld_dx, "dx", d->dy, a.ld_dy, "dy", d->T));
  TRY(check_in_place(d->dx, a.ld_dx, "dx", d->y, a.ld_y, "y", d->T));
  TRY(check_in_place(d->db, a.ld_db, "db", d->dn, a.ld_dn, "dn", d->T));
  TRY(check_in_place(d->db, a.ld_db, "db", d->b, a.ld_b, "b", d->T));
  TRY(check_gate(d->gate_v, "gate", d->gate, d->d, d->act, rows, &a.ld_gate));
  TRY(check_gate(d->dgate, "dgate", d->gate, d->d, d->act, false, &a.ld_dgate));
  TRY(check_vec(d->w_post, "w_post"));
  TRY(check_vec(d->w_next, "w_next"));
  if (!aligned(d->rstd_post, 4) || !aligned(d->rstd_next, 4) || !aligned(d->dw_post, 4) || !aligned(d->dw_next, 4))
    return fail(TQ_EINVAL, "rstd, dw_post and dw_next must be 4-byte aligned");
  a.nparts = norm_parts(d->T, d->d);
  if (d->dw_post || d->dw_next) {
    size_t need = 0;
    TRY(tq_norm_grad_workspace_size(d->T, d->d, &need));
    if (!ws) return fail(TQ_EINVAL, "ws is NULL");
    if (!aligned(ws, 256)) return fail(TQ_EINVAL, "ws not 256-byte aligned");
    if (ws_bytes < need) return fail(TQ_ESHAPE, "ws_bytes = %zu < %zu", ws_bytes, need);
  } else if (!rows) {
    return TQ_OK;
  }
  a.T = d->T;
  a.d = d->d;
  a.wdt = (int)d->w_dtype;
  a.gate = d->gate;
  a.alpha = d->alpha;
  a.y = d->y.p;
  a.dy = d->dy.p;
  a.dn = d->dn.p;
  a.b = d->b.p;
  a.dx = d->dx.p;
  a.db = d->db.p;
  a.dgate = d->dgate.p;
  a.gate_p = d->gate_v.p;
  a.w_post = d->w_post;
  a.w_next = d->w_next;
  a.rstd_post = const_cast<float*>(d->rstd_post);
  a.rstd_next = const_cast<float*>(d->rstd_next);
  a.dw_post = d->dw_post;
  a.dw_next = d->dw_next;
  a.part = reinterpret_cast<float*>(ws);
  launch_norm_backward(a, (int)d->stream_dtype, (int)d->act, reinterpret_cast<hipStream_t>(stream));
  return launched();
}

}  // extern "C"
