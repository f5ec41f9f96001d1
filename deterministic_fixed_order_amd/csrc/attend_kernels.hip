// attend_kernels.hip -- attention of one new token per row over a paged
// key-value cache, for gfx950.

#include <hip/hip_runtime.h>

#include "decode_device.h"

namespace detfold_impl {
namespace {

constexpr int kBlock = 256;

// One workgroup per row and query head, tiles of 256 tokens: a thread scores
// one token of the tile, then sums one value of the output over the tile.
template <typename Q, typename C, typename O>
__global__ __launch_bounds__(kBlock) void k_attend(AttendArgs p)
{
    const detfold_attend &a = p.a;
    const detfold_paged_cache &c = p.c;
    const int64_t b = blockIdx.x / a.q_heads;
    const int g = (int)(blockIdx.x % a.q_heads), h = g / p.group, tid = threadIdx.x;
    __shared__ float q[DETFOLD_MAX_HEAD], w[kBlock], part[kBlock];
    __shared__ int64_t place[kBlock];
    for (int i = tid; i < c.dim; i += kBlock)
        q[i] = to_f32(((const Q *)a.q)[b * a.q_row + g * a.q_head + i]);
    const int64_t len = a.lens[b] > 0 ? a.lens[b] : 0;
    bool bad = len > a.max_len || len > a.table_width * c.page;
    const int64_t end = bad ? 0 : len, begin = a.window > 0 && end > a.window ? end - a.window : 0;
    const float by = a.scale * (c.k_scale ? c.k_scale[h] : 1.0f);
    float m = -INFINITY, l = 0.0f, acc = 0.0f;
    for (int64_t t0 = begin; t0 < end; t0 += kBlock) {
        const int64_t t = t0 + tid;
        float s = -INFINITY;
        __syncthreads();
        if (t < end) {
            const uint32_t at = divide((uint32_t)t, p.page);
            const int64_t pg = a.table[b * a.table_row + at], off = t - (int64_t)at * c.page;
            if (pg < 0 || pg >= c.pages) {
                s = __builtin_nanf("");
                place[tid] = 0;
            } else {
                const C *k = (const C *)c.k + pg * c.k_page + off * c.k_token + h * c.k_head;
                s = 0.0f;
                for (int i = 0; i < c.dim; ++i)
                    s += q[i] * to_f32(k[i]);
                s *= by;
                place[tid] = pg * c.v_page + off * c.v_token + h * c.v_head;
            }
        }
        part[tid] = s;
        __syncthreads();
        for (int n = kBlock / 2; n > 0; n >>= 1) {
            if (tid < n)
                part[tid] = fmaxf(part[tid], part[tid + n]);
            __syncthreads();
        }
        const float top = fmaxf(m, part[0]), base = top == -INFINITY ? 0.0f : top;
        const float turn = expf(m - base);
        w[tid] = expf(s - base);
        __syncthreads();
        part[tid] = w[tid];
        __syncthreads();
        for (int n = kBlock / 2; n > 0; n >>= 1) {
            if (tid < n)
                part[tid] += part[tid + n];
            __syncthreads();
        }
        l = l * turn + part[0];
        m = top;
        acc *= turn;
        const int64_t count = end - t0 < kBlock ? end - t0 : kBlock;
        if (tid < c.v_dim)
            for (int i = 0; i < count; ++i)
                acc += w[i] * to_f32(((const C *)c.v + place[i])[tid]);
    }
    if (bad)
        l = __builtin_nanf("");
    if (tid < c.v_dim) {
        const float o = l == 0.0f ? 0.0f : acc * (c.v_scale ? c.v_scale[h] : 1.0f) / l;
        ((O *)a.out)[b * a.out_row + g * a.out_head + tid] = from_f32<O>(o);
    }
    if (a.lse && tid == 0)
        a.lse[b * a.q_heads + g] = (m == -INFINITY ? 0.0f : m) + logf(l);
}

template <typename Q, typename O> const void *pick(int cache)
{
    if (cache == DETFOLD_E4M3)
        return (const void *)k_attend<Q, e4m3, O>;
    if (sizeof(Q) == 4 && cache == DETFOLD_BF16)
        return (const void *)k_attend<Q, bf16, O>;
    return (const void *)k_attend<Q, Q, O>;
}

}  // namespace

int launch_attend(const AttendArgs &a, void *stream)
{
    const bool wide = a.a.out_type == DETFOLD_F32;
    const void *k = a.a.type == DETFOLD_F32    ? pick<float, float>(a.c.type)
                    : a.a.type == DETFOLD_BF16 ? (wide ? pick<bf16, float>(a.c.type) : pick<bf16, bf16>(a.c.type))
                                               : (wide ? pick<f16, float>(a.c.type) : pick<f16, f16>(a.c.type));
    AttendArgs copy = a;
    void *args[] = {&copy};
    return hipLaunchKernel(k, dim3((unsigned)(a.a.batch * a.a.q_heads)), dim3(kBlock), args, 0,
                           static_cast<hipStream_t>(stream)) == hipSuccess
               ? DETFOLD_OK
               : DETFOLD_ELAUNCH;
}

}  // namespace detfold_impl
