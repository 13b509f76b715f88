// w4_f32.hip -- the 4-bit weights' kernels for fp32 rows of x.
#include "w4_rows.h"

namespace dq {

W4RowsKernel w4_rows_f32(int row_tiles, int col_tiles, int S) { return w4_rows_pick<DQ_F32>(row_tiles, col_tiles, S); }

}  // namespace dq
