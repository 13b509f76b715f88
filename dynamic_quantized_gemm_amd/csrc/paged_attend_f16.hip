// paged_attend_f16.hip -- the attention kernel's instances for this cache type
// (attend_kernel.h).
#include "attend_kernel.h"

namespace dq {

// pieces of fp16: 16-bit queries are one (bf16 ones after their scaling), an
// fp32 query is three
AttendKernel attend_f16(dq_dtype q, int D) {
    if (q == DQ_F32) return attend_pick<DQ_F16, 3, 2>(D);
    return attend_pick<DQ_F16, 1, 2>(D);
}

}  // namespace dq
