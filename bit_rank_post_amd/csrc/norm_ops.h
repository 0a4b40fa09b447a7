// Arguments and launchers of the norms around a block (norm.hip) and of the
// 8-bit quantisation (quant8.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace tq {

// dtypes: 0 f16, 1 bf16, 2 f32
struct NormArgs {
  int T, d;
  int wdt;                       // dtype of the weights
  int gate;                      // 0 none, 1 one f32 per row, 2 a value for each element (act)
  float alpha, eps;
  // forward: x, b in; y, n out.  backward: y, dy, dn, b in; dx, db out.
  // absent: nullptr
  const void* x;
  const void* b;
  void* y;
  void* n;
  const void* w_post;            // [d] or nullptr: p(b) = b
  const void* w_next;            // [d]
  const void* gate_p;
  float* rstd_post;              // [T] written by the forward (or nullptr), read by the backward
  float* rstd_next;
  const void* dy;
  const void* dn;
  void* dx;
  void* db;
  void* dgate;
  float* dw_post;                // [d]
  float* dw_next;
  float* part;                   // [2][nparts][d] partial weight gradients
  int nparts;
  long ld_x, ld_b, ld_y, ld_n, ld_gate, ld_dy, ld_dn, ld_dx, ld_db, ld_dgate;
};
// sdt: dtype of x, y, dy, dx; adt: dtype of b, n, dn, db and a full gate
void launch_norm_forward(const NormArgs& a, int sdt, int adt, hipStream_t s);
void launch_norm_backward(const NormArgs& a, int sdt, int adt, hipStream_t s);
int norm_parts(int T, int d);

void launch_quant_rows(const void* x, int dtype, int rows, int d, long ldx, void* q, float* scale,
                       hipStream_t s);
void launch_quant_blocks(const void* w, int dtype, int groups, int d_out, int d_in, void* q, float* scale,
                         hipStream_t s);

constexpr int NORM_D_MAX = 16384;

}  // namespace tq
