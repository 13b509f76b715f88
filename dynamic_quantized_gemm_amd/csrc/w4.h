// w4.h -- what the translation units of the products with 4-bit weights
// share: the context, the packed layout and the kernels' arguments.
//
//   y[m, n] = sum_g s[n, g] (sum_{k in g} x[m, k] q[n, k]  -  z[n, g] sum_{k in g} x[m, k])
//
// The codes q (0 to 15) are exact in every operand type of the matrix cores,
// so each product of x and q is exact and the sums are fp32: nothing is
// rounded before the output but by those sums. The scales apply to a group's
// sum, not to its weights.
//
// Packed layout. The rows of W are taken 16 at a time (a tile: the columns of
// one 16x16 block of y) and K 128 at a time (a block). With gated != 0 the
// tiles alternate: 16 rows of the gate, the 16 rows of the values they gate.
// Rows are padded to whole tiles (their number to a multiple of 16), K to whole
// blocks; what is padded has code, scale and zero point 0.
//   codes  [experts][tiles][blocks][64 lanes][16 bytes]: a lane's 4 words are
//          the 4 k-steps of 32, for row lane % 16 and k = 8 (lane / 16) + i of
//          the step: byte b of the word holds i = b low and i = 4 + b high
//   scales [experts][tiles][blocks][16 rows][S], S = 4, 2 or 1 groups a block
//          (groups of 32, 64, or 128 and more: a larger group's is repeated)
//   zeros  the same with one byte each; none where every zero point is 8
// A wave reads 1 KiB of codes of a tile and block with one load a lane, in
// the order of the matrix operand.
#pragma once

#include "dq_device.h"

namespace dq {

constexpr int kW4Block = 128;  // k of a block
constexpr int kW4TilePad = 16;  // tiles of 16 rows are padded to a multiple of this

// the kernels' arguments; what they read has been checked against these sizes
struct W4Args {
    const void* x;            // rows of K elements, x_stride apart
    long long x_stride;
    const uint8_t* codes;
    const void* scales;       // 2 or 4 bytes each
    const uint8_t* zeros;     // NULL: 8
    const float* bias;        // [experts][tiles * 16] in the packed order; NULL: none
    void* y;                  // [rows, N]
    const int32_t* row_index; // NULL: row r of y comes from row r of x
    const int32_t* offsets;   // NULL: one expert has all rows
    int rows, x_rows, N, K, experts;
    int tiles, blocks;        // of an expert's weights
    int scale_type, y_type;
    int gated;
    int vec;                  // rows of x can be loaded 16 bytes at a time
    int col_groups;           // workgroups along the columns
    FastDiv per_row;          // by the pieces of 8 elements of a row, K padded to blocks
};

}  // namespace dq

struct dq_w4_ctx {
    int device = 0;
    int experts = 0, N = 0, K = 0, group = 0, gated = 0;
    int64_t max_rows = 0;
    dq_dtype x_type = DQ_BF16, scale_type = DQ_BF16, y_type = DQ_BF16;
    int tiles = 0, blocks = 0, S = 1;  // of the packed layout
    int cus = 256;
    bool ready = false, has_zeros = false, has_bias = false;
    uint8_t* codes = nullptr;
    void* scales = nullptr;
    uint8_t* zeros = nullptr;
    float* bias = nullptr;
    // many rows: sums of x's groups and rows prepared for sums_rows and copy_rows
    // rows at a time (0: the context takes few rows)
    float* sums = nullptr;
    uint16_t* copy = nullptr;
    int64_t sums_rows = 0, copy_rows = 0;
    char info[192] = "";
};

// What the files of each type of x offer: the kernels for few rows (w4_rows.h,
// and w4_any.h for rows that it cannot take) by rows and column tiles of 16 a
// workgroup, the kernel for many (w4_tile.h) by the workgroup's columns / 64,
// and the latter's preparation; S as above.
namespace dq {

struct W4TileArgs;
struct W4Prepare;
struct W4Kernels {
    void (*(*rows)(int rows, int col_tiles, int S, int scales))(W4Args);
    void (*(*any)(int rows, int col_tiles, int S))(W4Args);
    void (*(*tile)(int wide, int S, int scales, bool gather))(W4TileArgs);
    void (*prepare)(W4Prepare);
};
W4Kernels w4_kernels_bf16();
W4Kernels w4_kernels_f16();
W4Kernels w4_kernels_f32();

}  // namespace dq
