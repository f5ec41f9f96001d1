// attend_kernels.hip -- the launch of the paged attention and the join of the
// parts of long rows, for gfx950.

#include <hip/hip_runtime.h>

#include "attend_kernel.h"

namespace detfold_impl {
namespace {

// One workgroup per query head and row, or share that a row may begin in without
// ending there.  A lane takes four dims, LANES lanes a part, and the groups of
// lanes every GROUPS-th part; their sums are added in order.  Parts that are
// empty add zeros, so a row's bits do not depend on how many follow its last one.
//
// A part is v_dim + 2 floats per query head, about 1% of the tokens it stands
// for, so this is latency: the loads of eight parts go out together.  4 to 5 us
// (one row of 131072 in 128 parts, 256 rows of 4096), of which a launch is 2.
template <int LANES, int WAVES> __global__ __launch_bounds__(64 * WAVES) void k_join_parts(AttendArgs p)
{
    constexpr int GROUPS = 64 * WAVES / LANES;
    const detfold_attend &a = p.a;
    const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
    const uint32_t y = blockIdx.x / a.q_heads;
    const int head = blockIdx.x - y * a.q_heads, h = head / p.group, in = head - h * p.group;
    const int64_t unit = h * (int64_t)p.tiles.d + in / 16, heads = min(16, p.group), units = (int64_t)p.units.d * p.beside;
    int64_t b = p.row0 + y;
    int n = (int)p.parts.d;
    int64_t first, next, step;  // slots
    if (p.shares.d) {
        const int3 cut = p.cut[y];
        if (cut.x < 0)
            return;
        b = cut.x;
        n = cut.z - cut.y + 1;
        step = 2 * units;
        next = (cut.y * units + unit) * 2;
        first = next + 1;
    } else {
        step = units;
        first = next = b * n * step + unit;
    }
    auto slot = [&](int i) { return (i ? next + i * step : first) * heads + in % 16; };
    const int d0 = 4 * lane, d = min(d0, p.c.v_dim - 4);
    f4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    float m = -INFINITY, l = 0.0f;
    for (int i0 = group; i0 < n; i0 += 8 * GROUPS) {  // eight parts' loads together
        f4 x[8];
        float2 s[8];
        float top = m;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = i0 + j * GROUPS;
            const int64_t at = slot(min(i, n - 1));
            s[j] = p.ml[at];
            __builtin_memcpy(&x[j], p.acc + at * p.c.v_dim + d, sizeof(f4));
            if (i >= n)
                s[j] = make_float2(-INFINITY, 0.0f), x[j] = f4{0.0f, 0.0f, 0.0f, 0.0f};
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            top = fmaxf(top, s[j].x);
        const float base = top == -INFINITY ? 0.0f : top, turn = weight_of(m - base);
        l *= turn;
        acc *= turn;
        m = top;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float w = weight_of(s[j].x - base);
            l += s[j].y * w;
            acc += x[j] * w;
        }
    }
    __shared__ f4 accs[GROUPS][LANES];
    __shared__ float2 mls[GROUPS];
    accs[group][lane] = acc;
    if (lane == 0)
        mls[group] = make_float2(m, l);
    __syncthreads();
    if (group > 0)
        return;
    float top = -INFINITY;
    for (int i = 0; i < GROUPS; ++i)
        top = fmaxf(top, mls[i].x);
    const float base = top == -INFINITY ? 0.0f : top;
    acc = f4{0.0f, 0.0f, 0.0f, 0.0f}, l = 0.0f;
    for (int i = 0; i < GROUPS; ++i) {
        const float w = weight_of(mls[i].x - base);
        l += mls[i].y * w;
        acc += accs[i][lane] * w;
    }
    const float by = out_scale(p.c.v_scale ? p.c.v_scale[h] : 1.0f, l), out[4] = {acc.x * by, acc.y * by, acc.z * by, acc.w * by};
    if (d0 < p.c.v_dim)
        put_out<4>(a, b * a.out_row + (int64_t)head * a.out_head + d, out);
    if (a.lse && lane == 0)
        a.lse[b * a.q_heads + head] = log_sum(top, l);
}

template <int WAVES> const void *pick_join(int dim)
{
    return dim <= 64 ? (const void *)k_join_parts<16, WAVES> : dim <= 128 ? (const void *)k_join_parts<32, WAVES> : (const void *)k_join_parts<64, WAVES>;
}

}  // namespace

int launch_attend(const AttendArgs &a, void *stream)
{
    const AttendKernel k = a.a.type == DETFOLD_F32 ? attend_f32(a) : a.a.type == DETFOLD_BF16 ? attend_bf16(a) : attend_f16(a);
    AttendArgs copy = a;
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
    const int heads = a.group < 16 ? a.group : 16;
    const int queries = a.beside * k.q_bytes, sums = a.waves * (128 + heads * k.head_bytes), lds = queries > sums ? queries : sums;
    if (a.shares.d) {
        // Where rows have few parts, what counts is how many waves look for one: the
        // join of 64 ragged rows takes 7 us with two a workgroup and 12 with eight,
        // of 256 rows 5 and 7, of 16 rows of eight parts each 5.2 and 6.4.  Rows of
        // many parts want the waves: 1 x 131072 over two key heads of e4m3 (256
        // parts) 28 us in all with two, 24 with eight; 2 rows (128) 24 and 22, 4
        // rows (64) 22.1 both, 8 rows (32) 21.2 and 22.3.
        const bool few = a.a.batch * 32 >= a.shares.d;
        return launch(k.f, (int64_t)a.shares.d * a.units.d, 64 * a.waves, lds) &&
                       launch(few ? pick_join<2>(a.c.v_dim) : pick_join<8>(a.c.v_dim), (a.by_row ? a.a.batch : a.shares.d) * a.a.q_heads,
                              few ? 128 : 512, 0)
                   ? DETFOLD_OK
                   : DETFOLD_ELAUNCH;
    }
    if (!rows((int64_t)a.units.d * a.parts.d, k.f, 64 * a.waves, lds))
        return DETFOLD_ELAUNCH;
    if (a.parts.d > 1 && !rows(a.a.q_heads, pick_join<8>(a.c.v_dim), 512, 0))
        return DETFOLD_ELAUNCH;
    return DETFOLD_OK;
}

}  // namespace detfold_impl
