// attend_f32.hip -- the kernels of the paged attention for float32 queries, for gfx950.

#include <hip/hip_runtime.h>

#include "attend_kernel.h"

namespace detfold_impl {

AttendKernel attend_f32(const AttendArgs &a)
{
    if (a.c.type == DETFOLD_E4M3)
        return pick_attend<e4m3, kSplit, kSplit>(a);
    return a.c.type == DETFOLD_BF16 ? pick_attend<bf16, kF32, kF32>(a) : pick_attend<float, kF32, kF32>(a);
}

}  // namespace detfold_impl
