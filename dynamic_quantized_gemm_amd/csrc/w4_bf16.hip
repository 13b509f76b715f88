// w4_bf16.hip -- the 4-bit weights' kernels for bf16 rows of x.
#include "w4_any.h"
#include "w4_rows.h"
#include "w4_tile.h"

namespace dq {

W4Kernels w4_kernels_bf16() {
    return {w4_rows_pick<DQ_BF16>, w4_any_pick<DQ_BF16>, w4_tile_pick<DQ_BF16>, k_w4_prepare<DQ_BF16>};
}

}  // namespace dq
