// cache_kernels.hip -- the append to a paged cache with its position rotation,
// and the softmax-weighted fold of attention partials, for gfx950.

#include <hip/hip_runtime.h>

#include "decode_device.h"

namespace detfold_impl {
namespace {

constexpr int kBlock = 256;                      // threads of the append
constexpr int kFold = 128;                       // and of the fold
constexpr int64_t kOnceBytes = 8 << 20;          // of an output that is not kept in the caches
constexpr int kHeads = 2;
constexpr int64_t kFill = 1 << 18;               // threads that fill the device
constexpr int64_t kMaxItems = (int64_t)1 << 30;  // threads of a launch: a grid holds at most 2^32

// Workgroup b of n, of which each XCD takes runs of kRun neighbours (workgroups
// go to the XCDs round-robin): an XCD's share of a stream is then contiguous.
constexpr int kRun = 256;
__device__ __forceinline__ uint32_t in_runs(uint32_t b, uint32_t n)
{
    constexpr uint32_t span = 8 * kRun;
    const uint32_t r = b % span;
    return b - r + span <= n ? b - r + r % 8 * kRun + r / 8 : b;
}

// N values at any alignment that their type allows, as one wide load or store;
// once: not kept in the caches.
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
template <typename T, int N, bool ONCE = false> __device__ __forceinline__ void store_vec(T *p, const Vec<T, N> &v)
{
    constexpr int B = N * sizeof(T);
    if constexpr (ONCE && B % 4 == 0) {
        typedef uint32_t w __attribute__((ext_vector_type(B / 4), aligned(1)));
        w y;
        __builtin_memcpy(&y, &v, B);
        __builtin_nontemporal_store(y, (w *)p);
    } else {
        __builtin_memcpy(p, &v, B);
    }
}

__device__ __forceinline__ void turn(float &x, float &y, float c, float s)
{
    const float z = x * c - y * s;
    y = y * c + x * s;
    x = z;
}

// The append.  A thread takes V pairs that turn together (or V values that do
// not turn) of HEADS heads of one token, so that the angles are read once for
// these and their loads are in flight together; the values' heads are copied by
// the workgroups after the first `turn`.
//
// Bytes bound it: every value is read and written once, 3 flop to a turned one.
// 8192 tokens of 32 + 8 + 8 heads of 128 bfloat16: 37 us, 5.6 TB/s read and
// written, where a plain copy of 4 GiB runs at 4.8.  Few tokens are one thread's
// chain of loads, so they take one head a thread (1 token 2.9 us instead of 5.2,
// 64 into e4m3 3.5 instead of 7.5); more take two, and stores that bypass the
// caches (42 us without).
template <typename T, typename C, int V, int HEADS> __global__ __launch_bounds__(kBlock) void k_append(AppendArgs p)
{
    constexpr bool ONCE = HEADS > 1;
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
    const int head0 = (int)(g - (query || values ? 0 : p.q_groups)) * HEADS, heads = query ? a.q_heads : c.heads;
    const int64_t slot = a.slots[t];
    const bool stored = slot >= 0 && slot < c.pages * c.page;
    if (!query && !stored)
        return;
    const uint32_t pg = stored ? divide((uint32_t)slot, p.page) : 0;
    const int64_t off = stored ? slot - (int64_t)pg * c.page : 0;
    if (values) {
        const int i0 = min((int)u * V, c.v_dim - V);
        const T *x = (const T *)a.v + t * a.v_token + i0;
        C *y = (C *)c.v + pg * c.v_page + off * c.v_token + i0;
        Vec<T, V> v[HEADS];
#pragma unroll
        for (int j = 0; j < HEADS; ++j)
            v[j] = load_vec<T, V>(x + min(head0 + j, heads - 1) * a.v_head);
#pragma unroll
        for (int j = 0; j < HEADS; ++j) {
            const int h = head0 + j;
            if (h >= heads)
                break;
            const float by = c.v_scale ? c.v_scale[h] : 1.0f;
            Vec<C, V> o;
#pragma unroll
            for (int n = 0; n < V; ++n)
                o.x[n] = from_f32<C>(c.v_scale ? to_f32(v[j].x[n]) / by : to_f32(v[j].x[n]));
            store_vec<C, V, ONCE>(y + h * c.v_head, o);
        }
        return;
    }
    // The chunks of a head that turn come first.  The last one of a run starts
    // early enough to end with it.
    const int half = a.rot / 2, turned = (half + V - 1) / V;
    const bool turns = u < (uint32_t)turned;
    const int at = turns ? min((int)u * V, half - V) : a.rot + min(((int)u - turned) * V, c.dim - a.rot - V);
    const int i0 = turns && a.pairs ? 2 * at : at, i1 = !turns ? at : a.pairs ? 2 * at + V : half + at;
    const T *x = query ? (const T *)a.q + t * a.q_token : (const T *)a.k + t * a.k_token;
    const int64_t x_head = query ? a.q_head : a.k_head;
    Vec<T, V> v0[HEADS], v1[HEADS];
#pragma unroll
    for (int j = 0; j < HEADS; ++j) {
        const T *from = x + min(head0 + j, heads - 1) * x_head;
        v0[j] = load_vec<T, V>(from + i0);
        v1[j] = load_vec<T, V>(from + i1);
    }
    Vec<float, V> cs = {}, sn = {};
    if (turns) {
        const int64_t pos = a.positions[t];
        if (pos >= 0 && pos < a.angles) {
            cs = load_vec<float, V>(a.cos + pos * half + at);
            sn = load_vec<float, V>(a.sin + pos * half + at);
        } else {
#pragma unroll
            for (int n = 0; n < V; ++n)
                cs.x[n] = sn.x[n] = __builtin_nanf("");
        }
    }
#pragma unroll
    for (int j = 0; j < HEADS; ++j) {
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
            store_vec<T, V, ONCE>(to + i0, o);
            if (turns) {
#pragma unroll
                for (int n = 0; n < V; ++n)
                    o.x[n] = from_f32<T>(x01[V + n]);
                store_vec<T, V, ONCE>(to + i1, o);
            }
        } else {
            C *to = (C *)c.k + pg * c.k_page + off * c.k_token + h * c.k_head;
            const float by = c.k_scale ? c.k_scale[h] : 1.0f;
            Vec<C, V> o;
#pragma unroll
            for (int n = 0; n < V; ++n)
                o.x[n] = from_f32<C>(c.k_scale ? x01[n] / by : x01[n]);
            store_vec<C, V, ONCE>(to + i0, o);
            if (turns) {
#pragma unroll
                for (int n = 0; n < V; ++n)
                    o.x[n] = from_f32<C>(c.k_scale ? x01[V + n] / by : x01[V + n]);
                store_vec<C, V, ONCE>(to + i1, o);
            }
        }
    }
}

// exp(x), x <= 0.  For float32 partials to their own precision, where the product
// with log2 e alone would be off by up to |x| / 2 units of the result (0 to 2% of
// the time of large folds); for 16-bit ones the shorter form, 5% faster.
template <typename T> __device__ __forceinline__ float weight(float x)
{
    return sizeof(T) == 4 ? expf(x) : __builtin_amdgcn_exp2f(x * kLog2e);
}

// A sum over its weights' sum (by: that one's inverse): divided in float32; to 16
// bits, whose own rounding is 2^13 times that of another product, multiplied (1 to 5%
// of the time of large folds).
template <typename T> __device__ __forceinline__ float mean(float sum, float total, float by)
{
    return sizeof(T) == 4 ? sum / total : sum * by;
}

// The softmax fold.  A thread takes V neighbouring values of a row, eight
// partials' loads at a time, and forms the row's weights itself: eight
// exponentials cost less than handing them round.  Ascending in w throughout.
//
// Bytes bound it, W + 1 for W of arithmetic: 8 x 131072 x 128 float32 runs at 96
// us, 6.3 TB/s.  Workgroups of 128 threads in runs of 256 per XCD: 102 us with
// 256 in runs of 16, 109 without runs.  A thread's output is one wide store,
// past the caches where all outputs are 8 MiB or more: 131072 x 128 float32 33 us
// instead of 35 with 2 partials, 42 / 46 with 3, 53 / 55 with 4, 63.7 / 63.1 with 5, 74
// / 75 with 6, 85 / 86 with 7, 97 / 100 with 8; half the rows, 56 / 62 with 9, 72 / 80
// with 12, 95 / 104 with 16; bfloat16 18.5 / 19.1 with 2 to 58 / 63 with 16.  Below, a
// call of 32 rows takes 2.3 us instead of 2.4.
template <typename T, int V, bool ONCE> __global__ __launch_bounds__(kFold) void k_fold_softmax(SoftmaxArgs s)
{
    constexpr int N = 8;
    const uint32_t i = in_runs(blockIdx.x, gridDim.x) * kFold + threadIdx.x, in = divide(i, s.chunks), u = i - in * s.chunks.d;
    if (in >= s.count)
        return;
    const int64_t row = s.row0 + in, at = row * s.dim + min((int64_t)u * V, s.dim - V);
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
                const float a = weight<T>(lse[j] - base);
                total = total + a;
#pragma unroll
                for (int n = 0; n < V; ++n)
                    acc[n] = acc[n] + (lse[j] == -INFINITY ? 0.0f : a * to_f32(x[j].x[n]));
            }
    }
    const float some = total == 0.0f ? 1.0f : total, by = 1.0f / some;  // no partial had a token: the sums are zero
    Vec<T, V> o;
#pragma unroll
    for (int n = 0; n < V; ++n)
        o.x[n] = from_f32<T>(mean<T>(acc[n], some, by));
    store_vec<T, V, ONCE>((T *)s.out + at, o);
    if (s.lse && u == 0)
        s.lse[row] = (top == -INFINITY ? 0.0f : top) + logf(total);
}

template <typename T, typename C, int V> const void *append_heads(int heads)
{
    return heads == 1 ? (const void *)k_append<T, C, V, 1> : (const void *)k_append<T, C, V, kHeads>;
}
template <typename T, typename C> const void *append_width(int v, int heads)
{
    if constexpr (sizeof(T) == 2)
        if (v == 8)
            return append_heads<T, C, 8>(heads);
    return v == 4 ? append_heads<T, C, 4>(heads) : v == 2 ? append_heads<T, C, 2>(heads) : append_heads<T, C, 1>(heads);
}
template <typename T> const void *pick_append(int cache, int v, int heads)
{
    if (cache == DETFOLD_E4M3)
        return append_width<T, e4m3>(v, heads);
    if constexpr (sizeof(T) == 4)
        if (cache == DETFOLD_BF16)
            return append_width<T, bf16>(v, heads);
    return append_width<T, T>(v, heads);
}
template <typename T, int V> const void *softmax_once(bool once)
{
    return once ? (const void *)k_fold_softmax<T, V, true> : (const void *)k_fold_softmax<T, V, false>;
}
template <typename T> const void *pick_softmax(int v, bool once)
{
    if constexpr (sizeof(T) == 2)
        if (v == 8)
            return softmax_once<T, 8>(once);
    return v == 4 ? softmax_once<T, 4>(once) : v == 2 ? softmax_once<T, 2>(once) : softmax_once<T, 1>(once);
}

int chunks(int64_t n, int v) { return (int)((n + v - 1) / v); }

bool launch(const void *k, int64_t blocks, int threads, void *args, void *stream)
{
    void *list[] = {args};
    return hipLaunchKernel(k, dim3((unsigned)blocks), dim3(threads), list, 0, static_cast<hipStream_t>(stream)) == hipSuccess;
}

}  // namespace

int launch_append(const AppendArgs &a, void *stream)
{
    AppendArgs p = a;
    const int v = a.width;
    p.chunks = divider(chunks(a.a.rot / 2, v) + chunks(a.c.dim - a.a.rot, v));
    p.v_chunks = divider(chunks(a.c.v_dim, v));
    // One head a thread where there are not enough tokens to fill the device
    // otherwise: the time is then one thread's.
    const int heads = a.a.tokens * (a.a.q_heads + a.c.heads) * p.chunks.d / kHeads < kFill ? 1 : kHeads;
    const void *k = a.a.type == DETFOLD_F32    ? pick_append<float>(a.c.type, v, heads)
                    : a.a.type == DETFOLD_BF16 ? pick_append<bf16>(a.c.type, v, heads)
                                               : pick_append<f16>(a.c.type, v, heads);
    p.q_groups = (a.a.q_heads + heads - 1) / heads;
    p.groups = divider(p.q_groups + (a.c.heads + heads - 1) / heads);
    p.v_groups = divider((a.c.heads + heads - 1) / heads);
    const int64_t each = (int64_t)p.groups.d * p.chunks.d, v_each = (int64_t)p.v_groups.d * p.v_chunks.d;
    const int64_t some = kMaxItems / (each + v_each);
    for (p.token0 = 0; p.token0 < a.a.tokens; p.token0 += some) {
        p.tokens = (uint32_t)(a.a.tokens - p.token0 < some ? a.a.tokens - p.token0 : some);
        p.turn = (uint32_t)((p.tokens * each + kBlock - 1) / kBlock);
        if (!launch(k, p.turn + (p.tokens * v_each + kBlock - 1) / kBlock, kBlock, &p, stream))
            return DETFOLD_ELAUNCH;
    }
    return DETFOLD_OK;
}

int launch_softmax(const SoftmaxArgs &a, void *stream)
{
    SoftmaxArgs p = a;
    const int v = access_width(a.type, true, a.dim, 0, 0);
    const bool once = a.rows * a.dim * elem_size(a.type) >= kOnceBytes;
    const void *k = a.type == DETFOLD_F32 ? pick_softmax<float>(v, once) : a.type == DETFOLD_BF16 ? pick_softmax<bf16>(v, once) : pick_softmax<f16>(v, once);
    p.chunks = divider((uint32_t)chunks(a.dim, v));
    const int64_t some = kMaxItems / p.chunks.d;
    for (p.row0 = 0; p.row0 < a.rows; p.row0 += some) {
        p.count = (uint32_t)(a.rows - p.row0 < some ? a.rows - p.row0 : some);
        if (!launch(k, ((int64_t)p.count * p.chunks.d + kFold - 1) / kFold, kFold, &p, stream))
            return DETFOLD_ELAUNCH;
    }
    return DETFOLD_OK;
}

}  // namespace detfold_impl
