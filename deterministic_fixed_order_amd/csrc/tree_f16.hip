// tree_f16.hip -- the kernels of the attention of drafted tokens for float16 queries, for gfx950.

#include <hip/hip_runtime.h>

#include "tree_kernel.h"

namespace detfold_impl {

TreeKernel tree_f16(const TreeArgs &a)
{
    const bool wide = a.a.out_type == DETFOLD_F32;
    if (a.c.type == DETFOLD_E4M3)
        return wide ? pick_tree<e4m3, kF16, kSplit>(a) : pick_tree<e4m3, kF16, kF16>(a);
    return wide ? pick_tree<f16, kF16, kF32>(a) : pick_tree<f16, kF16, kF16>(a);
}

}  // namespace detfold_impl
