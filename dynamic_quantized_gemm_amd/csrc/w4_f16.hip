// w4_f16.hip -- the 4-bit weights' kernels for fp16 rows of x.
#include "w4_rows.h"

namespace dq {

W4RowsKernel w4_rows_f16(int row_tiles, int col_tiles, int S) { return w4_rows_pick<DQ_F16>(row_tiles, col_tiles, S); }

}  // namespace dq
