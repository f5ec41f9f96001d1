// cache_kernels.hip -- the append to a paged cache with its position rotation,
// and the softmax-weighted fold of attention partials, for gfx950.

#include <hip/hip_runtime.h>

#include "decode_device.h"

namespace detfold_impl {
namespace {

constexpr int kBlock = 256;

// One thread per pair that turns together, or per value that does not.
template <typename T, typename C>
__global__ __launch_bounds__(kBlock) void k_append(AppendArgs p)
{
    const detfold_append &a = p.a;
    const detfold_paged_cache &c = p.c;
    const int64_t t = blockIdx.x;
    const int half = a.rot / 2, units = c.dim - half;
    const int64_t slot = a.slots[t];
    const bool stored = slot >= 0 && slot < c.pages * c.page;
    const uint32_t pg = stored ? divide((uint32_t)slot, p.page) : 0;
    const int64_t off = stored ? slot - (int64_t)pg * c.page : 0;
    const int64_t pos = half ? a.positions[t] : 0;
    const bool placed = pos >= 0 && pos < a.angles;
    for (int w = threadIdx.x; w < (a.q_heads + c.heads) * units; w += kBlock) {
        const int row = w / units, u = w % units;
        const bool is_q = row < a.q_heads;
        const int h = is_q ? row : row - a.q_heads;
        if (!is_q && !stored)
            continue;
        const T *x = is_q ? (const T *)a.q + t * a.q_token + h * a.q_head : (const T *)a.k + t * a.k_token + h * a.k_head;
        T *yq = (T *)a.q_out + t * a.out_token + h * a.out_head;
        C *yk = (C *)c.k + pg * c.k_page + off * c.k_token + h * c.k_head;
        const float by = !is_q && c.k_scale ? c.k_scale[h] : 1.0f;
        auto put = [&](int i, float v) {
            if (is_q)
                yq[i] = from_f32<T>(v);
            else
                yk[i] = from_f32<C>(c.k_scale ? v / by : v);
        };
        if (u >= half) {
            put(half + u, to_f32(x[half + u]));
            continue;
        }
        const int i = a.pairs ? 2 * u : u, j = a.pairs ? 2 * u + 1 : u + half;
        const float cs = placed ? a.cos[pos * half + u] : __builtin_nanf("");
        const float sn = placed ? a.sin[pos * half + u] : __builtin_nanf("");
        const float xi = to_f32(x[i]), xj = to_f32(x[j]);
        put(i, xi * cs - xj * sn);
        put(j, xj * cs + xi * sn);
    }
    if (!stored)
        return;
    for (int w = threadIdx.x; w < c.heads * c.v_dim; w += kBlock) {
        const int h = w / c.v_dim, i = w % c.v_dim;
        const float v = to_f32(((const T *)a.v)[t * a.v_token + h * a.v_head + i]);
        ((C *)c.v)[pg * c.v_page + off * c.v_token + h * c.v_head + i] = from_f32<C>(c.v_scale ? v / c.v_scale[h] : v);
    }
}

// One thread per element; every thread forms its row's weights itself.
template <typename T> __global__ __launch_bounds__(kBlock) void k_fold_softmax(SoftmaxArgs s)
{
    const int64_t n = s.rows * s.dim;
    for (int64_t e = (int64_t)blockIdx.x * kBlock + threadIdx.x; e < n; e += (int64_t)gridDim.x * kBlock) {
        const int64_t row = e / s.dim;
        float top = -INFINITY;
        for (int w = 0; w < s.w; ++w)
            top = fmaxf(top, s.lses[w * s.lses_pitch + row]);
        top = top == -INFINITY ? 0.0f : top;
        float acc = 0.0f, total = 0.0f;
        for (int w = 0; w < s.w; ++w) {
            const float lse = s.lses[w * s.lses_pitch + row];
            const float a = expf(lse - top);
            total = total + a;
            if (lse != -INFINITY)
                acc = acc + a * to_f32(((const T *)s.outs)[w * s.outs_pitch + e]);
        }
        ((T *)s.out)[e] = from_f32<T>(total == 0.0f ? 0.0f : acc / total);
        if (s.lse && e == row * s.dim)
            s.lse[row] = top + logf(total);
    }
}

template <typename T> const void *pick_append(int cache)
{
    if (cache == DETFOLD_E4M3)
        return (const void *)k_append<T, e4m3>;
    if (sizeof(T) == 4 && cache == DETFOLD_BF16)
        return (const void *)k_append<T, bf16>;
    return (const void *)k_append<T, T>;
}

}  // namespace

int launch_append(const AppendArgs &a, void *stream)
{
    const void *k = a.a.type == DETFOLD_F32    ? pick_append<float>(a.c.type)
                    : a.a.type == DETFOLD_BF16 ? pick_append<bf16>(a.c.type)
                                               : pick_append<f16>(a.c.type);
    AppendArgs copy = a;
    void *args[] = {&copy};
    return hipLaunchKernel(k, dim3((unsigned)a.a.tokens), dim3(kBlock), args, 0, static_cast<hipStream_t>(stream)) == hipSuccess
               ? DETFOLD_OK
               : DETFOLD_ELAUNCH;
}

int launch_softmax(const SoftmaxArgs &s, void *stream)
{
    const void *k = s.type == DETFOLD_F32    ? (const void *)k_fold_softmax<float>
                    : s.type == DETFOLD_BF16 ? (const void *)k_fold_softmax<bf16>
                                             : (const void *)k_fold_softmax<f16>;
    SoftmaxArgs copy = s;
    void *args[] = {&copy};
    const int64_t blocks = (s.rows * s.dim + kBlock - 1) / kBlock;
    return hipLaunchKernel(k, dim3((unsigned)(blocks < (1 << 30) ? blocks : (1 << 30))), dim3(kBlock), args, 0,
                           static_cast<hipStream_t>(stream)) == hipSuccess
               ? DETFOLD_OK
               : DETFOLD_ELAUNCH;
}

}  // namespace detfold_impl
