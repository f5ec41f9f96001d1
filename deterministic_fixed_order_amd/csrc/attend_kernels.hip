// attend_kernels.hip -- the launch of the paged attention and the join of the
// parts of long rows, for gfx950.

#include <hip/hip_runtime.h>

#include "attend_kernel.h"

namespace detfold_impl {
namespace {

constexpr int kBlock = 256;
constexpr int64_t kMaxBlocks = (int64_t)1 << 22;  // of a launch: a grid holds at most 2^32 threads

// One workgroup per row and query head.  A wave takes every fourth part, a
// lane four dims (heads are at most 256), and the waves' sums are added in
// order: parts that are empty add zeros, so a row's bits do not depend on how
// many follow its last one.
__global__ __launch_bounds__(kBlock) void k_join_parts(AttendArgs p)
{
    const detfold_attend &a = p.a;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t b = p.row0 + blockIdx.x / a.q_heads;
    const int head = blockIdx.x % a.q_heads, n = (int)p.parts.d;
    const int64_t g = b * a.q_heads + head;
    const float2 *ml = p.ml + g * n;
    float m = -INFINITY;
    for (int i = lane; i < n; i += 64)
        m = fmaxf(m, ml[i].x);
#pragma unroll
    for (int i = 32; i > 0; i >>= 1)
        m = fmaxf(m, __shfl_xor(m, i));
    const float base = m == -INFINITY ? 0.0f : m;
    const int d0 = 4 * lane, d = min(d0, p.c.v_dim - 4);
    const float *o = p.acc + g * n * p.c.v_dim + d;
    f4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    float l = 0.0f;
#pragma unroll 8
    for (int i = wave; i < n; i += kBlock / 64) {
        const float2 s = ml[i];
        f4 x;
        __builtin_memcpy(&x, o + (int64_t)i * p.c.v_dim, sizeof(x));
        const float w = __builtin_amdgcn_exp2f(s.x - base);
        l += s.y * w;
        if (s.y == 0.0f)  // no token: its sums were not written
            x = f4{0.0f, 0.0f, 0.0f, 0.0f};
        acc += x * w;
    }
    __shared__ f4 accs[kBlock / 64][64];
    __shared__ float ls[kBlock / 64];
    accs[wave][lane] = acc;
    if (lane == 0)
        ls[wave] = l;
    __syncthreads();
    if (wave > 0)
        return;
#pragma unroll
    for (int i = 1; i < kBlock / 64; ++i) {
        acc += accs[i][lane];
        l += ls[i];
    }
    const float vs = p.c.v_scale ? p.c.v_scale[head / p.group] : 1.0f;
    const float out[4] = {attended(acc.x, vs, l), attended(acc.y, vs, l), attended(acc.z, vs, l), attended(acc.w, vs, l)};
    if (d0 < p.c.v_dim)
        put_out<4>(a, b * a.out_row + (int64_t)head * a.out_head + d, out);
    if (a.lse && lane == 0)
        a.lse[g] = log_sum(m, l);
}

}  // namespace

int launch_attend(const AttendArgs &a, void *stream)
{
    const bool wide = a.a.out_type == DETFOLD_F32;
    const int dim = a.c.dim > a.c.v_dim ? a.c.dim : a.c.v_dim;
    const AttendKernel k = a.a.type == DETFOLD_F32    ? attend_f32(a.c.type, dim, a.tiled)
                           : a.a.type == DETFOLD_BF16 ? attend_bf16(a.c.type, wide, dim, a.tiled)
                                                      : attend_f16(a.c.type, wide, dim, a.tiled);
    AttendArgs copy = a;
    void *args[] = {&copy};
    // Rows to a launch, whatever a row's workgroups.
    auto rows = [&](int64_t each, const void *f, int threads, int lds) {
        const int64_t some = each < kMaxBlocks ? kMaxBlocks / each : 1;
        for (copy.row0 = 0; copy.row0 < a.a.batch; copy.row0 += some) {
            const int64_t now = a.a.batch - copy.row0 < some ? a.a.batch - copy.row0 : some;
            if (hipLaunchKernel(f, dim3((unsigned)(now * each)), dim3(threads), args, lds, static_cast<hipStream_t>(stream)) != hipSuccess)
                return false;
        }
        return true;
    };
    const int threads = 64 * a.waves, lds = k.q_bytes + a.waves / 2 * k.save_bytes;
    if (!rows((int64_t)a.units.d * a.parts.d, k.f, threads, lds))
        return DETFOLD_ELAUNCH;
    if (a.parts.d > 1 && !rows(a.a.q_heads, (const void *)k_join_parts, kBlock, 0))
        return DETFOLD_ELAUNCH;
    return DETFOLD_OK;
}

}  // namespace detfold_impl
