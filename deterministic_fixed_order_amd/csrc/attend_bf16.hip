// attend_bf16.hip -- the kernels of the paged attention for bfloat16 queries, for gfx950.

#include <hip/hip_runtime.h>

#include "attend_kernel.h"

namespace detfold_impl {

AttendKernel attend_bf16(int cache, bool wide, int dim, bool tiled, bool brief)
{
    if (cache == DETFOLD_E4M3)
        return wide ? pick_attend<e4m3, kBf16, kF32>(dim, tiled, brief) : pick_attend<e4m3, kBf16, kBf16>(dim, tiled, brief);
    return wide ? pick_attend<bf16, kBf16, kF32>(dim, tiled, brief) : pick_attend<bf16, kBf16, kBf16>(dim, tiled, brief);
}

}  // namespace detfold_impl
