// attend_bf16.hip -- the kernels of the paged attention for bfloat16 queries, for gfx950.

#include <hip/hip_runtime.h>

#include "attend_kernel.h"

namespace detfold_impl {

AttendKernel attend_bf16(const AttendArgs &a)
{
    const bool wide = a.a.out_type == DETFOLD_F32;
    if (a.c.type == DETFOLD_E4M3)
        return wide ? pick_attend<e4m3, kBf16, kSplit>(a) : pick_attend<e4m3, kBf16, kBf16>(a);
    return wide ? pick_attend<bf16, kBf16, kF32>(a) : pick_attend<bf16, kBf16, kBf16>(a);
}

}  // namespace detfold_impl
