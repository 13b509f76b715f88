// w4_bf16.hip -- the 4-bit weights' kernels for bf16 rows of x.
#include "w4_rows.h"

namespace dq {

W4RowsKernel w4_rows_bf16(int row_tiles, int col_tiles, int S) { return w4_rows_pick<DQ_BF16>(row_tiles, col_tiles, S); }

}  // namespace dq
