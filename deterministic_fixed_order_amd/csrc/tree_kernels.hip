// tree_kernels.hip -- the attention of drafted tokens over a paged cache, for gfx950.

#include <hip/hip_runtime.h>

#include "decode_device.h"
#include "draft.h"

namespace detfold_impl {
namespace {

constexpr int kBlock = 256;
constexpr int64_t kMaxBlocks = (int64_t)1 << 22;

// One workgroup per row, drafted query and query head; 256 tokens at a time.
template <typename T, typename C> __global__ __launch_bounds__(kBlock) void k_tree(TreeArgs p, int64_t block0)
{
    const detfold_attend &a = p.a;
    const detfold_paged_cache &c = p.c;
    const int64_t block = block0 + blockIdx.x;
    const int g = (int)(block % a.q_heads), i = (int)(block / a.q_heads % p.drafts), h = g / p.group;
    const int64_t b = block / a.q_heads / p.drafts;
    const int drafted = min(max(p.counts ? p.counts[b] : p.drafts, 0), p.drafts);
    if (i >= drafted)
        return;
    const int64_t n0 = max(a.lens[b], 0);
    bool bad = n0 > a.max_len || n0 > a.table_width * c.page;
    const int64_t n = bad ? 0 : n0, base = max(n - drafted, (int64_t)0);
    auto depth = [&](int64_t j) { return p.depths ? min(max(p.depths[b * p.drafts + j], 0), DETFOLD_MAX_DRAFTS - 1) : (int)j; };
    const uint64_t mask = p.masks ? (uint64_t)p.masks[b * p.drafts + i] : ~0ull >> (63 - i);
    const int64_t own = base + depth(i);
    const T *q = (const T *)a.q + b * a.q_row + i * p.q_draft + g * a.q_head;
    const float by = a.scale * (c.k_scale ? c.k_scale[h] : 1.0f), slope = p.slopes ? p.slopes[g] : 0.0f;
    const int32_t *table = a.table + b * a.table_row;

    __shared__ float weights[kBlock];
    __shared__ int64_t places[kBlock];
    __shared__ float red[kBlock];
    __shared__ int bads;
    if (threadIdx.x == 0)
        bads = bad;
    __syncthreads();
    float m = -INFINITY, l = 0.0f, acc = 0.0f;
    const int64_t begin = p.window > 0 ? max(base - p.window, (int64_t)0) : 0;
    for (int64_t t0 = begin; t0 < n; t0 += kBlock) {
        const int64_t t = t0 + threadIdx.x;
        float s = -INFINITY;
        int64_t at = -1;
        if (t < n) {
            const int64_t pos = t < base ? t : base + depth(t - base);
            const bool seen = (t < base || (mask >> (t - base) & 1)) && (p.window == 0 || own - pos < p.window);
            if (seen) {
                const int64_t id = table[t / c.page];
                if (id < 0 || id >= c.pages) {
                    bads = 1;
                } else {
                    const C *k = (const C *)c.k + id * c.k_page + t % c.page * c.k_token + h * c.k_head;
                    float dot = 0.0f;
                    for (int d = 0; d < c.dim; ++d)
                        dot += to_f32(q[d]) * to_f32(k[d]);
                    s = dot * by;
                    if (p.cap > 0.0f)
                        s = p.cap * tanhf(s / p.cap);
                    if (p.slopes)
                        s += slope * (float)(pos - own);
                    at = id * c.v_page + t % c.page * c.v_token + h * c.v_head;
                }
            }
        }
        red[threadIdx.x] = s;
        __syncthreads();
        float top = m;
        bool odd = false;
        for (int j = 0; j < kBlock; ++j)
            top = fmaxf(top, red[j]), odd |= __builtin_isnan(red[j]);
        const float origin = top == -INFINITY ? 0.0f : top, turn = expf(m - origin);
        weights[threadIdx.x] = at < 0 ? 0.0f : expf(s - origin);
        places[threadIdx.x] = at;
        __syncthreads();
        l *= turn, acc *= turn, m = top;
        for (int j = 0; j < kBlock; ++j) {
            l += weights[j];
            if (places[j] >= 0 && (int)threadIdx.x < c.v_dim)
                acc += weights[j] * to_f32(((const C *)c.v + places[j])[threadIdx.x]);
        }
        if (odd)
            l = __builtin_nanf("");
        __syncthreads();
    }
    __syncthreads();
    if (bads)
        l = __builtin_nanf("");
    const float out = (l == 0.0f ? 0.0f : 1.0f / l) * acc * (c.v_scale ? c.v_scale[h] : 1.0f);
    const int64_t to = b * a.out_row + i * p.out_draft + g * a.out_head + threadIdx.x;
    if ((int)threadIdx.x < c.v_dim) {
        if (a.out_type == DETFOLD_F32)
            ((float *)a.out)[to] = out;
        else if constexpr (sizeof(T) == 2)
            ((T *)a.out)[to] = (T)out;
    }
    if (a.lse && threadIdx.x == 0)
        a.lse[(b * p.drafts + i) * a.q_heads + g] = (m == -INFINITY ? 0.0f : m) + logf(l);
}

template <typename T> const void *pick(int cache)
{
    if (cache == DETFOLD_E4M3)
        return (const void *)k_tree<T, e4m3>;
    if constexpr (sizeof(T) == 4)
        if (cache == DETFOLD_BF16)
            return (const void *)k_tree<T, bf16>;
    return (const void *)k_tree<T, T>;
}

}  // namespace

int launch_tree(const TreeArgs &a, void *stream)
{
    TreeArgs copy = a;
    const void *f = a.a.type == DETFOLD_F32 ? pick<float>(a.c.type) : a.a.type == DETFOLD_BF16 ? pick<bf16>(a.c.type) : pick<f16>(a.c.type);
    const int64_t total = a.a.batch * a.drafts * a.a.q_heads;
    for (int64_t first = 0; first < total; first += kMaxBlocks) {
        void *args[] = {&copy, &first};
        if (hipLaunchKernel(f, dim3((unsigned)(total - first < kMaxBlocks ? total - first : kMaxBlocks)), dim3(kBlock), args, 0,
                            static_cast<hipStream_t>(stream)) != hipSuccess)
            return DETFOLD_ELAUNCH;
    }
    return DETFOLD_OK;
}

}  // namespace detfold_impl
