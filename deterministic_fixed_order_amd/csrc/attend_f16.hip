// attend_f16.hip -- the kernels of the paged attention for float16 queries, for gfx950.

#include <hip/hip_runtime.h>

#include "attend_kernel.h"

namespace detfold_impl {

AttendKernel attend_f16(int cache, bool wide, int dim, bool tiled, bool brief)
{
    if (cache == DETFOLD_E4M3)
        return wide ? pick_attend<e4m3, kF16, kF32>(dim, tiled, brief) : pick_attend<e4m3, kF16, kF16>(dim, tiled, brief);
    return wide ? pick_attend<f16, kF16, kF32>(dim, tiled, brief) : pick_attend<f16, kF16, kF16>(dim, tiled, brief);
}

}  // namespace detfold_impl
