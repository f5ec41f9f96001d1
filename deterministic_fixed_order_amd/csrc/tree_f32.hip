// tree_f32.hip -- the kernels of the attention of drafted tokens for float32 queries, for gfx950.

#include <hip/hip_runtime.h>

#include "tree_kernel.h"

namespace detfold_impl {

TreeKernel tree_f32(const TreeArgs &a)
{
    if (a.c.type == DETFOLD_E4M3)
        return pick_tree<e4m3, kSplit, kSplit>(a);
    return a.c.type == DETFOLD_BF16 ? pick_tree<bf16, kF32, kF32>(a) : pick_tree<float, kF32, kF32>(a);
}

}  // namespace detfold_impl
