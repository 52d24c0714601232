// Parameter blocks of the products with bias, activation and residual (mb_linear) between their C entries
// (mb_linear_api.cu) and the kernels (mb_linear.cu, mb_linear_rows.cu).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace mb {

constexpr int LINEAR_MAX_GROUPS = 1024;
constexpr int LINEAR_TILE = 256;         // rows of a pair's tile
constexpr int LINEAR_DEEP = 64;          // of the contraction in one stage

// One product D = A B^T over tiles of 256 rows x `wide` columns, by pairs of CTAs.
//   rows of a group (forward, dx):  D's rows are the group's, B is the group's matrix;
//   over a group's rows (dweight):  the contraction runs over them, D is the group's matrix.
struct LinearJob {
  CUtensorMap a, b;
  CUtensorMap d;           // the result in boxes of 32 rows x 64, where `bulk`
  int bulk;                // whole chunks are stored by TMA (of the forward pass: z too)
  int a_mn, b_mn;          // the operand's rows run along memory (boxes of 64 x 64), not the contraction
  int over_rows;
  int M;                   // over_rows: D's rows
  int N, K;                // D's columns; the contraction (not over_rows)
  int wide;                // 128 or 256
  int m_tiles, n_tiles;    // m_tiles: over_rows only
  int passes, pass_cols;   // 2: the A operand comes as two halves, the second pass_cols columns on: each has sums of its own
  int splits;              // parts of the contraction
  int access;              // bytes that D's rows allow to be stored at a time: 16, 4 or 2
  void* out;
  long long ld, group_stride;
  float* parts;            // splits > 1: fp32 sums of every (split, tile), laid out by the epilogue's warps
  long long part_tiles;    // tiles that it holds for each split
};

// dz = dy act'(z) and the sums of dz over slabs of rows.
struct LinearSlopeParams {
  const void* dy;
  long long dy_ld;
  const void* z;           // or null: dz = dy, not written
  long long z_ld;
  void* dz;                // [rows, dz_ld], 16-byte aligned rows
  long long dz_ld;
  int low;                 // 0, or the columns to dz's low halves: what its rounding left; zeros up to there past the last, rows of 2 low
  int act, rows, cols, groups;
  const int* ends;
  float* parts;            // or null
  int slab;                // rows of a slab
  int access;              // bytes that the rows allow to be read at a time: 16, 4 or 2
};

// The same as pieces that the products' epilogue warps take while they have nothing to store (LINEAR_PIECE_ROWS rows x 256
// columns, in the order in which the products need them).
constexpr int LINEAR_PIECE_ROWS = 32;
struct LinearAhead {
  LinearSlopeParams slope;
  unsigned* next;          // the next piece, zero at the launch; null: dz is there already
  unsigned* done;          // [slabs of LINEAR_PIECE_ROWS rows] column groups that are done, zero at the launch
  int slabs, column_groups;
  int ways, per_way;       // the pieces go through `ways` ranges of `per_way` slabs in turn
};

struct LinearParams {
  LinearJob job[2];
  int jobs;
  int extra;               // units of the second job for pairs that have one of the first less than others
  int rows, groups;
  const int* ends;         // [groups] or null: one group of all rows
  int status_from;         // whether this launch reports bad ends
  // forward
  const void* bias;        // [groups, out] or null
  int bias_f32, act;
  const void* residual;
  long long residual_ld;
  int residual_access;
  int residual_bulk;       // its chunks come by TMA
  CUtensorMap residual_map;
  void* z;
  long long z_ld;
  int z_access;
  CUtensorMap z_map;       // where job[0].bulk
  // dbias, from the sums over slabs of rows that the launch before made: [slabs + groups][db_cols]
  const float* db_parts;
  void* db;
  int db_f32, db_cols, slab;
  int* status;
  LinearAhead ahead;       // backward
};

// dbias from the sums over slabs of rows.
struct LinearBiasParams {
  const float* parts;      // [slabs + groups][cols]
  void* db;
  int f32, cols, slab, rows, groups;
  const int* ends;
};

// Rows of 2-byte elements into rows that start at 16-byte boundaries.
struct LinearPackParams {
  const uint16_t* src;
  long long src_ld;
  uint16_t* dst;
  long long dst_ld;
  long long rows;
  int cols;
  int pairs;               // rows and columns come in 4-byte pairs
};

// The product over a few rows: at most LINEAR_SOME_ROWS (LINEAR_SOME_GROUPED over groups) where W's and x's rows start at 16-byte
// boundaries, else LINEAR_FEW_ROWS.
constexpr int LINEAR_FEW_ROWS = 8, LINEAR_SOME_ROWS = 512, LINEAR_SOME_GROUPED = 64;
struct LinearFewParams {
  const void* x;
  long long x_ld;
  const void* w;           // [groups, out, in]
  const void* bias;        // [groups, out] or null
  int bias_f32, act;
  const void* residual;
  long long residual_ld;
  void* z;
  long long z_ld;
  void* y;
  long long y_ld;
  int rows, in, out, groups;
  const int* ends;
  int access;              // bytes that the rows of x and w allow to be read at a time
  int* status;
};
cudaError_t launch_linear_few(const LinearFewParams& p, int type, cudaStream_t s);

cudaError_t launch_linear(const LinearParams& p, int type, bool forward, int pairs_wanted, cudaStream_t s);
cudaError_t launch_linear_join(const LinearParams& p, int job, int type, bool forward, long long tiles, cudaStream_t s);
cudaError_t launch_linear_slope(const LinearSlopeParams& p, int type, cudaStream_t s);
cudaError_t launch_linear_bias(const LinearBiasParams& p, int type, cudaStream_t s);
cudaError_t launch_linear_pack(const LinearPackParams& p, int sms, cudaStream_t s);

}  // namespace mb
