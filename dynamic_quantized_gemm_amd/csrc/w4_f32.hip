// w4_f32.hip -- the 4-bit weights' kernels for fp32 rows of x.
#include "w4_any.h"
#include "w4_rows.h"
#include "w4_tile.h"

namespace dq {

W4Kernels w4_kernels_f32() {
    return {w4_rows_pick<DQ_F32>, w4_any_pick<DQ_F32>, w4_tile_pick<DQ_F32>, k_w4_prepare<DQ_F32>};
}

}  // namespace dq
