// cache_kernels.hip -- the append to a paged cache with its position rotation,
// and the softmax-weighted fold of attention partials, for gfx950.

#include <hip/hip_runtime.h>

#include "decode_device.h"

namespace detfold_impl {
namespace {

constexpr int kBlock = 256;
constexpr int64_t kMaxItems = (int64_t)1 << 30;  // threads of a launch: a grid holds at most 2^32

// N values at any alignment that their type allows, as one wide load or store.
template <typename T, int N> struct Vec {
    T x[N];
};
template <typename T, int N, bool ONCE = false> __device__ __forceinline__ Vec<T, N> load_vec(const T *p)
{
    constexpr int B = N * sizeof(T);
    Vec<T, N> v;
    if constexpr (ONCE && B % 4 == 0) {
        typedef uint32_t w __attribute__((ext_vector_type(B / 4), aligned(1)));
        const w y = __builtin_nontemporal_load((const w *)p);
        __builtin_memcpy(&v, &y, B);
    } else {
        __builtin_memcpy(&v, p, B);
    }
    return v;
}
template <typename T, int N> __device__ __forceinline__ void store_vec(T *p, const Vec<T, N> &v) { __builtin_memcpy(p, &v, sizeof(v)); }

__device__ __forceinline__ void turn(float &x, float &y, float c, float s)
{
    const float z = x * c - y * s;
    y = y * c + x * s;
    x = z;
}

// Heads that a thread turns by the same angles, and whose loads it issues
// together.
constexpr int kHeads = 4;

// The append.  A thread takes V pairs that turn together (or V values that do
// not turn) of kHeads heads of one token, so that the angles are read once for
// these; the values' heads are copied by the workgroups after the first `turn`.
template <typename T, typename C, int V> __global__ __launch_bounds__(kBlock) void k_append(AppendArgs p)
{
    const detfold_append &a = p.a;
    const detfold_paged_cache &c = p.c;
    const bool values = blockIdx.x >= p.turn;
    const uint32_t i = (blockIdx.x - (values ? p.turn : 0)) * kBlock + threadIdx.x;
    const Divider &per_row = values ? p.v_chunks : p.chunks, &per_token = values ? p.v_groups : p.groups;
    const uint32_t y = divide(i, per_row), u = i - y * per_row.d;
    const uint32_t in = divide(y, per_token), g = y - in * per_token.d;
    if (in >= p.tokens)
        return;
    const int64_t t = p.token0 + in;
    const bool query = !values && g < (uint32_t)p.q_groups;
    const int head0 = (int)(g - (query || values ? 0 : p.q_groups)) * kHeads, heads = query ? a.q_heads : c.heads;
    const int64_t slot = a.slots[t];
    const bool stored = slot >= 0 && slot < c.pages * c.page;
    if (!query && !stored)
        return;
    const uint32_t pg = stored ? divide((uint32_t)slot, p.page) : 0;
    const int64_t off = stored ? slot - (int64_t)pg * c.page : 0;
    if (values) {
        const T *x = (const T *)a.v + t * a.v_token + u * V;
        C *y = (C *)c.v + pg * c.v_page + off * c.v_token + u * V;
        Vec<T, V> v[kHeads];
#pragma unroll
        for (int j = 0; j < kHeads; ++j)
            v[j] = load_vec<T, V>(x + min(head0 + j, heads - 1) * a.v_head);
#pragma unroll
        for (int j = 0; j < kHeads; ++j) {
            const int h = head0 + j;
            if (h >= heads)
                break;
            const float by = c.v_scale ? c.v_scale[h] : 1.0f;
            Vec<C, V> o;
#pragma unroll
            for (int n = 0; n < V; ++n)
                o.x[n] = from_f32<C>(c.v_scale ? to_f32(v[j].x[n]) / by : to_f32(v[j].x[n]));
            store_vec(y + h * c.v_head, o);
        }
        return;
    }
    const int half = a.rot / 2, turned = half / V;  // the chunks of a head that turn come first
    const bool turns = u < (uint32_t)turned;
    const int i0 = turns ? (int)u * (a.pairs ? 2 * V : V) : a.rot + ((int)u - turned) * V;
    const int i1 = turns ? i0 + (a.pairs ? V : half) : i0;
    const T *x = query ? (const T *)a.q + t * a.q_token : (const T *)a.k + t * a.k_token;
    const int64_t x_head = query ? a.q_head : a.k_head;
    Vec<T, V> v0[kHeads], v1[kHeads];
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
        const T *from = x + min(head0 + j, heads - 1) * x_head;
        v0[j] = load_vec<T, V>(from + i0);
        v1[j] = load_vec<T, V>(from + i1);
    }
    Vec<float, V> cs = {}, sn = {};
    if (turns) {
        const int64_t pos = a.positions[t];
        if (pos >= 0 && pos < a.angles) {
            cs = load_vec<float, V>(a.cos + pos * half + u * V);
            sn = load_vec<float, V>(a.sin + pos * half + u * V);
        } else {
#pragma unroll
            for (int n = 0; n < V; ++n)
                cs.x[n] = sn.x[n] = __builtin_nanf("");
        }
    }
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
        const int h = head0 + j;
        if (h >= heads)
            break;
        float x01[2 * V];  // values i0 on, then i1 on
#pragma unroll
        for (int n = 0; n < V; ++n)
            x01[n] = to_f32(v0[j].x[n]), x01[V + n] = to_f32(v1[j].x[n]);
        if (turns && a.pairs) {
#pragma unroll
            for (int n = 0; n < V; ++n)
                turn(x01[2 * n], x01[2 * n + 1], cs.x[n], sn.x[n]);
        } else if (turns) {
#pragma unroll
            for (int n = 0; n < V; ++n)
                turn(x01[n], x01[V + n], cs.x[n], sn.x[n]);
        }
        if (query) {
            T *to = (T *)a.q_out + t * a.out_token + h * a.out_head;
            Vec<T, V> o;
#pragma unroll
            for (int n = 0; n < V; ++n)
                o.x[n] = from_f32<T>(x01[n]);
            store_vec(to + i0, o);
            if (turns) {
#pragma unroll
                for (int n = 0; n < V; ++n)
                    o.x[n] = from_f32<T>(x01[V + n]);
                store_vec(to + i1, o);
            }
        } else {
            C *to = (C *)c.k + pg * c.k_page + off * c.k_token + h * c.k_head;
            const float by = c.k_scale ? c.k_scale[h] : 1.0f;
            Vec<C, V> o;
#pragma unroll
            for (int n = 0; n < V; ++n)
                o.x[n] = from_f32<C>(c.k_scale ? x01[n] / by : x01[n]);
            store_vec(to + i0, o);
            if (turns) {
#pragma unroll
                for (int n = 0; n < V; ++n)
                    o.x[n] = from_f32<C>(c.k_scale ? x01[V + n] / by : x01[V + n]);
                store_vec(to + i1, o);
            }
        }
    }
}

// The softmax fold.  A thread takes V neighbouring values of a row, eight
// partials' loads at a time, and forms the row's weights itself: eight
// exponentials cost less than handing them round.
template <typename T, int V> __global__ __launch_bounds__(kBlock) void k_fold_softmax(SoftmaxArgs s)
{
    constexpr int N = 8;
    const uint32_t i = blockIdx.x * kBlock + threadIdx.x, in = divide(i, s.chunks), u = i - in * s.chunks.d;
    if (in >= s.count)
        return;
    const int64_t row = s.row0 + in, at = row * s.dim + u * V;
    const T *outs = (const T *)s.outs + at;
    const float *lses = s.lses + row;
    float top = -INFINITY, total = 0.0f, acc[V] = {};
    if (s.w > N)
        for (int w = 0; w < s.w; ++w)
            top = fmaxf(top, lses[w * s.lses_pitch]);
    for (int w0 = 0; w0 < s.w; w0 += N) {
        float lse[N];
        Vec<T, V> x[N];
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (w0 + j < s.w) {
                lse[j] = lses[(w0 + j) * s.lses_pitch];
                x[j] = load_vec<T, V, true>(outs + (w0 + j) * s.outs_pitch);
            }
        if (s.w <= N)
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (j < s.w)
                    top = fmaxf(top, lse[j]);
        const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (w0 + j < s.w) {
                const float a = __builtin_amdgcn_exp2f((lse[j] - base) * kLog2e);
                total = total + a;
#pragma unroll
                for (int n = 0; n < V; ++n)
                    acc[n] = acc[n] + (lse[j] == -INFINITY ? 0.0f : a * to_f32(x[j].x[n]));
            }
    }
    const float by = total == 0.0f ? 0.0f : 1.0f / total;
    Vec<T, V> o;
#pragma unroll
    for (int n = 0; n < V; ++n)
        o.x[n] = from_f32<T>(acc[n] * by);
    store_vec((T *)s.out + at, o);
    if (s.lse && u == 0)
        s.lse[row] = (top == -INFINITY ? 0.0f : top) + logf(total);
}

template <typename T, typename C> const void *append_width(int v)
{
    if constexpr (sizeof(T) == 2)
        if (v == 8)
            return (const void *)k_append<T, C, 8>;
    return v == 4 ? (const void *)k_append<T, C, 4> : v == 2 ? (const void *)k_append<T, C, 2> : (const void *)k_append<T, C, 1>;
}
template <typename T> const void *pick_append(int cache, int v)
{
    if (cache == DETFOLD_E4M3)
        return append_width<T, e4m3>(v);
    if constexpr (sizeof(T) == 4)
        if (cache == DETFOLD_BF16)
            return append_width<T, bf16>(v);
    return append_width<T, T>(v);
}
template <typename T> const void *pick_softmax(int v)
{
    if constexpr (sizeof(T) == 2)
        if (v == 8)
            return (const void *)k_fold_softmax<T, 8>;
    return v == 4 ? (const void *)k_fold_softmax<T, 4> : v == 2 ? (const void *)k_fold_softmax<T, 2> : (const void *)k_fold_softmax<T, 1>;
}

// The widest access of at most 16 bytes that divides every run of values.
int width(int type, int64_t a, int64_t b, int64_t c)
{
    int v = 16 / elem_size(type);
    while (a % v || b % v || c % v)
        v /= 2;
    return v;
}

bool launch(const void *k, int64_t blocks, void *args, void *stream)
{
    void *list[] = {args};
    return hipLaunchKernel(k, dim3((unsigned)blocks), dim3(kBlock), list, 0, static_cast<hipStream_t>(stream)) == hipSuccess;
}

}  // namespace

int launch_append(const AppendArgs &a, void *stream)
{
    AppendArgs p = a;
    const int v = width(a.a.type, a.a.rot / 2, a.c.dim - a.a.rot, a.c.v_dim);
    const void *k = a.a.type == DETFOLD_F32    ? pick_append<float>(a.c.type, v)
                    : a.a.type == DETFOLD_BF16 ? pick_append<bf16>(a.c.type, v)
                                               : pick_append<f16>(a.c.type, v);
    p.q_groups = (a.a.q_heads + kHeads - 1) / kHeads;
    p.groups = divider(p.q_groups + (a.c.heads + kHeads - 1) / kHeads);
    p.v_groups = divider((a.c.heads + kHeads - 1) / kHeads);
    p.chunks = divider((a.a.rot / 2 + a.c.dim - a.a.rot) / v);
    p.v_chunks = divider(a.c.v_dim / v);
    const int64_t each = (int64_t)p.groups.d * p.chunks.d, v_each = (int64_t)p.v_groups.d * p.v_chunks.d;
    const int64_t some = kMaxItems / (each + v_each);
    for (p.token0 = 0; p.token0 < a.a.tokens; p.token0 += some) {
        p.tokens = (uint32_t)(a.a.tokens - p.token0 < some ? a.a.tokens - p.token0 : some);
        p.turn = (uint32_t)((p.tokens * each + kBlock - 1) / kBlock);
        if (!launch(k, p.turn + (p.tokens * v_each + kBlock - 1) / kBlock, &p, stream))
            return DETFOLD_ELAUNCH;
    }
    return DETFOLD_OK;
}

int launch_softmax(const SoftmaxArgs &a, void *stream)
{
    SoftmaxArgs p = a;
    const int v = width(a.type, a.dim, 0, 0);
    const void *k = a.type == DETFOLD_F32 ? pick_softmax<float>(v) : a.type == DETFOLD_BF16 ? pick_softmax<bf16>(v) : pick_softmax<f16>(v);
    p.chunks = divider((uint32_t)(a.dim / v));
    const int64_t some = kMaxItems / p.chunks.d;
    for (p.row0 = 0; p.row0 < a.rows; p.row0 += some) {
        p.count = (uint32_t)(a.rows - p.row0 < some ? a.rows - p.row0 : some);
        if (!launch(k, ((int64_t)p.count * p.chunks.d + kBlock - 1) / kBlock, &p, stream))
            return DETFOLD_ELAUNCH;
    }
    return DETFOLD_OK;
}

}  // namespace detfold_impl
