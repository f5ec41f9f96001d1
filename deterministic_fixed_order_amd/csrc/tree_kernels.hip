// tree_kernels.hip -- the launch of the attention of drafted tokens and the join
// of the parts of long rows, for gfx950.

#include <hip/hip_runtime.h>

#include "tree_kernel.h"

namespace detfold_impl {
namespace {

constexpr int kBlock = 256;  // threads of the join

// The sums of each query of a row, or of the row that a share begins without
// ending it, joined in order.  A lane takes four dims, LANES lanes a part, and
// GROUPS groups of lanes every GROUPS-th part of a query; the loads of DEEP parts
// go out together.  Parts that are empty add zeros, so with the same GROUPS and DEEP a
// row's bits do not depend on how many follow its last one.  Nor do they on whether
// there are groups, where these have one part each and one group takes as many at a time:
// the same sums in the same order, each product added by one rounding.
template <int LANES, int GROUPS, int DEEP> __global__ __launch_bounds__(kBlock) void k_join_tree(TreeArgs p)
{
    constexpr int QUERIES = kBlock / (LANES * GROUPS);  // of a workgroup
    const detfold_attend &a = p.a;
    const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES % GROUPS, own = threadIdx.x / (LANES * GROUPS);
    const uint32_t y = divide(blockIdx.x, p.join_blocks);
    const int query = (int)(blockIdx.x - y * p.join_blocks.d) * QUERIES + own;
    const int64_t units = (int64_t)p.units.d * p.beside;
    int64_t b = p.row0 + y;
    int n = (int)p.parts.d;
    bool there = query < p.drafts * a.q_heads;
    int3 cut = {};
    if (p.shares.d) {
        cut = p.cut[y];
        if (cut.x < 0)
            return;
        b = cut.x;
        n = cut.z - cut.y + 1;
    }
    const int i = (int)((uint32_t)query / (uint32_t)a.q_heads), head = query - i * a.q_heads;
    there &= i < (p.counts ? p.counts[b] : p.drafts);
    const int h = (int)divide((uint32_t)head, p.heads_of), col = i * p.group + head - h * p.group;
    const int tile = col / (16 * p.tiles_of);
    const int64_t unit = h * (int64_t)p.tiles.d + tile;
    int64_t first, next, step;  // slots
    if (p.shares.d) {
        step = 2 * units;
        next = (cut.y * units + unit) * 2;
        first = next + 1;
    } else {
        step = units;
        first = next = b * n * step + unit;
    }
    auto slot = [&](int i) { return (i ? next + i * step : first) * p.slot_cols + (col - tile * 16 * p.tiles_of); };
    const int d0 = 4 * lane, d = min(d0, p.c.v_dim - 4);
    f4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    float m = -INFINITY, l = 0.0f;
    for (int i0 = group; there && i0 < n; i0 += DEEP * GROUPS) {
        f4 x[DEEP];
        float2 s[DEEP];
        float top = m;
#pragma unroll
        for (int j = 0; j < DEEP; ++j) {
            const int i = i0 + j * GROUPS;
            const int64_t at = slot(min(i, n - 1));
            s[j] = p.ml[at];
            __builtin_memcpy(&x[j], p.acc + at * p.c.v_dim + d, sizeof(f4));
            if (i >= n)
                s[j] = make_float2(-INFINITY, 0.0f), x[j] = f4{0.0f, 0.0f, 0.0f, 0.0f};
        }
#pragma unroll
        for (int j = 0; j < DEEP; ++j)
            top = fmaxf(top, s[j].x);
        const float origin = top == -INFINITY ? 0.0f : top, turn = weight2_of(m - origin);
        l *= turn;
        acc *= turn;
        m = top;
#pragma unroll
        for (int j = 0; j < DEEP; ++j) {
            const float w = weight2_of(s[j].x - origin);
            l = __builtin_fmaf(s[j].y, w, l);
            acc = __builtin_elementwise_fma(x[j], f4{w, w, w, w}, acc);
        }
    }
    float top = m;
    if constexpr (GROUPS > 1) {
        __shared__ f4 accs[QUERIES][GROUPS][LANES];
        __shared__ float2 mls[QUERIES][GROUPS];
        accs[own][group][lane] = acc;
        if (lane == 0)
            mls[own][group] = make_float2(m, l);
        __syncthreads();
        there &= group == 0;
        top = -INFINITY;
        for (int i = 0; i < GROUPS; ++i)
            top = fmaxf(top, mls[own][i].x);
        const float origin = top == -INFINITY ? 0.0f : top;
        acc = f4{0.0f, 0.0f, 0.0f, 0.0f}, l = 0.0f;
        for (int i = 0; i < GROUPS; ++i) {
            const float w = weight2_of(mls[own][i].x - origin);
            l = __builtin_fmaf(mls[own][i].y, w, l);
            acc = __builtin_elementwise_fma(accs[own][i][lane], f4{w, w, w, w}, acc);
        }
    }
    if (!there)
        return;
    const float by = out_scale(p.c.v_scale ? p.c.v_scale[h] : 1.0f, l), out[4] = {acc.x * by, acc.y * by, acc.z * by, acc.w * by};
    if (d0 < p.c.v_dim)
        put_out<4>(a, b * a.out_row + i * p.out_draft + (int64_t)head * a.out_head + d, out);
    if (a.lse && lane == 0)
        a.lse[(b * p.drafts + i) * a.q_heads + head] = log_sum2(top, l);
}

template <int GROUPS, int DEEP> const void *pick_join(int dim)
{
    if constexpr (GROUPS == 4 || DEEP == 4)
        if (dim > 128)
            return (const void *)k_join_tree<64, GROUPS, DEEP>;
    return dim <= 64 ? (const void *)k_join_tree<16, GROUPS, DEEP> : (const void *)k_join_tree<32, GROUPS, DEEP>;
}

}  // namespace

int launch_tree(const TreeArgs &a, void *stream)
{
    const TreeKernel k = a.a.type == DETFOLD_F32 ? tree_f32(a) : a.a.type == DETFOLD_BF16 ? tree_bf16(a) : tree_f16(a);
    TreeArgs copy = a;
    void *args[] = {&copy};
    auto launch = [&](const void *f, int64_t blocks, int threads, int lds) {
        return hipLaunchKernel(f, dim3((unsigned)blocks), dim3(threads), args, lds, static_cast<hipStream_t>(stream)) == hipSuccess;
    };
    // Some rows to a launch, whatever a row's workgroups.
    auto rows = [&](int64_t each, const void *f, int threads, int lds) {
        const int64_t some = each < kMaxBlocks ? kMaxBlocks / each : 1;
        for (copy.row0 = 0; copy.row0 < a.a.batch; copy.row0 += some)
            if (!launch(f, (a.a.batch - copy.row0 < some ? a.a.batch - copy.row0 : some) * each, threads, lds))
                return false;
        return true;
    };
    const int queries = k.staged_bytes + a.beside * k.unit_bytes + 4 * DETFOLD_MAX_DRAFTS, sums = a.waves * k.wave_bytes, lds = queries > sums ? queries : sums;
    if (!(a.shares.d ? launch(k.f, (int64_t)a.shares.d * a.units.d, 64 * a.waves, lds) : rows((int64_t)a.units.d * a.parts.d, k.f, 64 * a.waves, lds)))
        return DETFOLD_ELAUNCH;
    if (!a.shares.d && a.parts.d <= 1)
        return DETFOLD_OK;
    // Where rows have many parts, and few queries wait for them, several groups of
    // lanes take a query's.  With `split` a row's bits must not go by the number of parts,
    // which max_len sets: there groups begin where they have more than one part each, and
    // up to there one group takes all parts at once, which adds the same (16 x 64 tokens
    // over 2048 in 2 parts: 88 us, 128 with groups; 64 x 8 over 4096 in 8: 224 and 249).
    const int lanes = a.c.v_dim <= 64 ? 16 : a.c.v_dim <= 128 ? 32 : 64, most = 256 / lanes < 8 ? 4 : 8;
    const int64_t parts = a.shares.d ? a.shares.d / a.a.batch : a.parts.d, queries_all = (int64_t)a.drafts * a.a.q_heads;
    const int groups = parts > (a.a.split > 0 ? most : 8) ? most : 1, per = kBlock / (lanes * groups);
    const bool at_once = a.a.split > 0 && parts > 4;
    const int64_t each = (queries_all + per - 1) / per;
    copy.join_blocks = divider((uint32_t)each);
    const void *join = groups == 8 ? pick_join<8, 8>(a.c.v_dim) : groups == 4 ? pick_join<4, 8>(a.c.v_dim)
                       : at_once   ? pick_join<1, 8>(a.c.v_dim) : pick_join<1, 4>(a.c.v_dim);
    if (!(a.shares.d ? launch(join, (a.by_row ? a.a.batch : a.shares.d) * each, kBlock, 0) : rows(each, join, kBlock, 0)))
        return DETFOLD_ELAUNCH;
    return DETFOLD_OK;
}

}  // namespace detfold_impl
