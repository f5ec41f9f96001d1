// attend_f32.hip -- the kernels of the paged attention for float32 queries, for gfx950.

#include <hip/hip_runtime.h>

#include "attend_kernel.h"

namespace detfold_impl {

AttendKernel attend_f32(int cache, int dim, bool tiled, bool brief)
{
    if (cache == DETFOLD_E4M3)
        return pick_attend<e4m3, kF32, kF32>(dim, tiled, brief);
    return cache == DETFOLD_BF16 ? pick_attend<bf16, kF32, kF32>(dim, tiled, brief) : pick_attend<float, kF32, kF32>(dim, tiled, brief);
}

}  // namespace detfold_impl
