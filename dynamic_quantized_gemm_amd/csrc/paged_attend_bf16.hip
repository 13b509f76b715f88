// paged_attend_bf16.hip -- the attention kernel's instances for this cache type
// (attend_kernel.h).
#include "attend_kernel.h"

namespace dq {

// pieces of bf16: a bf16 query is one, an fp16 one (11 digits) two, an fp32
// one three; fp32 outputs keep the weights in three pieces
AttendKernel attend_bf16(dq_dtype q, int D) {
    if (q == DQ_F32) return attend_pick<DQ_BF16, 3, 3>(D);
    if (q == DQ_F16) return attend_pick<DQ_BF16, 2, 2>(D);
    return attend_pick<DQ_BF16, 1, 2>(D);
}

}  // namespace dq
