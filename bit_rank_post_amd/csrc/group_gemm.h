// Arguments and launchers of the products grouped by expert (group_gemm.hip,
// group_rows.hip): 16-bit operands in three directions, e4m3 operands with a
// scale for each block of 128 and 8-bit integers with a scale for each row.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace tq {

// Y  (forward):  y[r]  = W_g x[s(r)]            r in the rows of group g
// DX (gradient): dx[r] = W_g^T dy[r]
// DW (gradient): dW_g  = sum_r dy[r] x[s(r)]^T
enum GroupMode { GROUP_Y = 0, GROUP_DX = 1, GROUP_DW = 2 };
enum GroupType { GROUP_F16 = 0, GROUP_BF16 = 1, GROUP_E4M3 = 2, GROUP_I8 = 3 };

struct GroupArgs {
  int groups, rows, d_in, d_out;
  const int* off;                // [groups + 1], or nullptr: one group of all rows
  const int* src;                // [rows] index of each row, or nullptr
  int x_rows;                    // rows of x
  uint32_t div_mul;              // s(r) = src[r] / div: (src * div_mul) >> 32 >> div_shift,
  int div_shift;                 // or src itself when div_shift < 0 (div 1)
  const void* x;                 // [x_rows][ldx]
  const void* w;                 // [groups][d_out][d_in]
  const void* dy;                // [rows][ldy]
  void* out;                     // Y [rows][ldo], DX [rows][ldo], DW [groups][d_out][d_in]
  long ldx, ldy, ldo;            // row strides in elements
  int out_dtype;                 // 0 f16, 1 bf16, 2 f32
  int vec_out;                   // eight neighbouring outputs may be stored as 16-byte words
  int vec_scales;                // I8: ws may be read as 16-byte words
  const float* xs;               // E4M3: [x_rows][ceil(d_in/128)] scales of x; I8: [x_rows]
  const float* ws;               // E4M3: [groups][ceil(d_out/128)][ceil(d_in/128)]; I8: [groups][d_out]
};

// Y by waves over k without LDS staging (outputs x rows per workgroup): few
// rows per group (decode), or few tiles
enum GroupRows { ROWS_16x16 = 0, ROWS_32x32 = 1 };
void launch_group_rows(const GroupArgs& a, GroupType type, GroupRows shape, hipStream_t s);
long group_rows_grid(const GroupArgs& a, GroupRows shape);
void group_rows_shape(GroupRows shape, int* outputs, int* rows);

// Tile shapes of the LDS kernel (outputs x rows per workgroup).
enum GroupTile { TILE_256x256 = 0, TILE_128x128 = 1, TILE_128x32 = 2 };

void launch_group_tile(const GroupArgs& a, GroupMode mode, GroupType type, GroupTile tile, hipStream_t s);
// the kernel for a product, by sizes and type alone
struct GroupPick {
  bool rows;                     // launch_group_rows with shape, else launch_group_tile with tile
  GroupRows shape;
  GroupTile tile;
};
GroupPick choose_group(const GroupArgs& a, GroupMode mode, GroupType type);
// workgroups that launch_group_tile would start
long group_tile_grid(const GroupArgs& a, GroupMode mode, GroupTile tile);
void group_tile_shape(GroupTile tile, int* outputs, int* rows);

}  // namespace tq
