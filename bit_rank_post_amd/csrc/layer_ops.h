// Arguments and launchers of what lies between and after the products of a
// layer of experts (swiglu.hip, slots.hip) and of the whole layer for a few
// tokens (experts.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace tq {

// dtypes: 0 f16, 1 bf16, 2 f32
struct SwigluArgs {
  int rows, ff;
  const int* off;                // [groups + 1]: rows off[0] .. off[groups]-1 only; or nullptr: all
  int groups;
  const void* a;                 // [rows][lda]: gate, up
  void* h;                       // [rows][ldh]
  const void* dh;                // gradient: [rows][lddh]
  void* da;                      // [rows][ldda]
  long lda, ldh, lddh, ldda;
};
// adt: dtype of a and da; hdt: of h (swiglu) or dh (gradient, whose h is of adt)
void launch_swiglu(const SwigluArgs& a, int adt, int hdt, hipStream_t s);
void launch_swiglu_grad(const SwigluArgs& a, int adt, int hdt, hipStream_t s);

// 8-bit integers with a scale for each row: of x [rows][ldx] (d values), or of
// silu(gate) up with x = a [rows][ldx] (2 d values)
struct Int8RowsArgs {
  int rows, d;
  const int* off;
  int groups;
  const void* x;
  long ldx;
  int8_t* q;                     // [rows][d]
  float* scale;                  // [rows]
};
void launch_int8_rows(const Int8RowsArgs& a, int xdt, bool swiglu, hipStream_t s);

struct SlotSumArgs {
  int T, topk, d, rows;          // rows of z and dz
  const int* inv;                // [T * topk]
  const float* w;                // [T][topk] or nullptr: 1
  const void* z;
  const void* add;               // [T][ld_add] of y's type, or nullptr
  void* y;
  const void* dy;
  void* dz;
  float* dw;                     // [T][topk] or nullptr
  long ldz, ldy, ld_add, ld_dy, ld_dz;
};
// zdt: dtype of z and dz; ydt: of y, add and dy
void launch_slot_sum(const SlotSumArgs& a, int zdt, int ydt, hipStream_t s);
void launch_slot_sum_grad(const SlotSumArgs& a, int zdt, int ydt, hipStream_t s);

struct ExpertsArgs {
  int T, topk, experts, d, ff;
  const int* ids;                // [T][topk]
  const float* w;                // [T][topk]
  const void* x;                 // [T][ldx], act
  const void* w_up;              // [experts][2 ff][d], act or 8-bit integers
  const void* w_down;            // [experts][d][ff]
  const float* s_up;             // 8-bit integers: [experts][2 ff]
  const float* s_down;           // [experts][d]
  const void* add;               // [T][ld_add] of y's type, or nullptr
  void* y;                       // [T][ldy]
  long ldx, ldy, ld_add;
  int ydt;
  int* done;                     // [experts_tiles(d)] workgroups of the second kernel that are done
  int* hit;                      // experts that have a slot
  void* h;                       // [T * topk][ff] act
  float* z;                      // [T * topk][d]
};
constexpr int EXPERTS_SLOTS = 1024;      // slots that a call may have
__host__ __device__ inline int experts_tiles(int d) { return (d + 15) / 16; }
// The kernels of a call (by sizes alone): columns that a workgroup takes at a time
// (1: those of a single token), outputs and waves of a workgroup of either.
struct ExpertsKernel { int outputs, waves; };
struct ExpertsPick {
  int columns;
  ExpertsKernel up, down;
};
ExpertsPick choose_experts(const ExpertsArgs& a, bool int8);
// act: 0 f16, 1 bf16; int8: weights in 8-bit integers
void launch_experts(const ExpertsArgs& a, int act, bool int8, hipStream_t s);

}  // namespace tq
