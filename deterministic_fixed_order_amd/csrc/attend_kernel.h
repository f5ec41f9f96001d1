// attend_kernel.h -- the kernel of the paged attention: one new token per row
// over a paged key-value cache.  Included by the attend_*.hip files, each of
// which instantiates the kernels of one compute type.
#ifndef DETFOLD_ATTEND_KERNEL_H
#define DETFOLD_ATTEND_KERNEL_H

#include "decode_device.h"

namespace detfold_impl {

enum Math { kBf16, kF16, kF32 };  // what the matrix units multiply

typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

// N bytes of the cache, read once: at any alignment that a head's start may
// have (one wide load all the same), and not kept in the caches.
template <int N> struct Words {
    uint32_t w[N / 4];
};
template <int N> __device__ __forceinline__ Words<N> load_words(const char *p)
{
    typedef uint32_t v4 __attribute__((ext_vector_type(4), aligned(1)));
    typedef uint32_t v2 __attribute__((ext_vector_type(2), aligned(1)));
    typedef uint32_t v1 __attribute__((aligned(1)));
    Words<N> r;
    if constexpr (N >= 16) {
#pragma unroll
        for (int i = 0; i < N / 16; ++i) {
            const v4 x = __builtin_nontemporal_load((const v4 *)p + i);
            r.w[4 * i] = x.x, r.w[4 * i + 1] = x.y, r.w[4 * i + 2] = x.z, r.w[4 * i + 3] = x.w;
        }
    } else if constexpr (N == 8) {
        const v2 x = __builtin_nontemporal_load((const v2 *)p);
        r.w[0] = x.x, r.w[1] = x.y;
    } else {
        r.w[0] = __builtin_nontemporal_load((const v1 *)p);
    }
    return r;
}

// Two neighbouring values of the cache as the 16-bit type of the matrix units
// (exact), and as floats.
template <typename C, int M> __device__ __forceinline__ uint32_t pair16(const uint32_t *w, int i)
{
    if constexpr (sizeof(C) == 2)
        return w[i];
    else if constexpr (M == kBf16)
        return __builtin_bit_cast(uint32_t, (i & 1) ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i / 2], 1.0f, true)
                                                    : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i / 2], 1.0f, false));
    else
        return __builtin_bit_cast(uint32_t, (i & 1) ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[i / 2], 1.0f, true)
                                                    : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[i / 2], 1.0f, false));
}
template <typename C> __device__ __forceinline__ float value32(const uint32_t *w, int i)
{
    if constexpr (sizeof(C) == 4)
        return __builtin_bit_cast(float, w[i]);
    else if constexpr (sizeof(C) == 1)
        return __builtin_amdgcn_cvt_f32_fp8((int)(w[i / 4] >> (8 * (i % 4))), 0);
    else if constexpr (__is_same(C, bf16))
        return __builtin_bit_cast(float, (i & 1) ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    else
        return (float)__builtin_bit_cast(f16x2, w[i / 2])[i & 1];
}

template <int M> __device__ __forceinline__ f4 mfma16(u4 a, u4 b, f4 c)
{
    if constexpr (M == kBf16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Over the four groups of 16 lanes, the same on all of them.
template <typename F> __device__ __forceinline__ float over_groups(float x, F f)
{
    const auto a = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
    x = f(__builtin_bit_cast(float, (uint32_t)a[0]), __builtin_bit_cast(float, (uint32_t)a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
    return f(__builtin_bit_cast(float, (uint32_t)b[0]), __builtin_bit_cast(float, (uint32_t)b[1]));
}

template <typename T> __device__ __forceinline__ float read_q(const void *q, int64_t i) { return to_f32(((const T *)q)[i]); }

// The ends of a row: its output from the sums, the logarithm of its weights'
// sum (m is in units of log 2), and the store of N values.
__device__ __forceinline__ float attended(float acc, float v_scale, float l) { return l == 0.0f ? 0.0f : acc * v_scale / l; }
__device__ __forceinline__ float log_sum(float m, float l) { return (m == -INFINITY ? 0.0f : m * kLn2) + logf(l); }
template <int N> __device__ __forceinline__ void put_out(const detfold_attend &a, int64_t at, const float (&o)[N])
{
    if (a.out_type == DETFOLD_F32) {
        float x[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            x[i] = o[i];
        __builtin_memcpy((float *)a.out + at, x, sizeof(x));
    } else if (a.out_type == DETFOLD_BF16) {
        bf16 x[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            x[i] = (bf16)o[i];
        __builtin_memcpy((bf16 *)a.out + at, x, sizeof(x));
    } else {
        f16 x[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            x[i] = (f16)o[i];
        __builtin_memcpy((f16 *)a.out + at, x, sizeof(x));
    }
}

template <typename C, int QK, int PV, int D, bool TILED> struct Attend {
    static constexpr int kSize = sizeof(C);
    static constexpr int kChunk = 16 / kSize;         // dims of one 16-byte load of a key
    static constexpr int kChunks = D / (4 * kChunk);  // of these per lane and key
    static constexpr int kTiles = kSize == 4 && D == 256 ? 1 : 2;  // tiles of 16 tokens in a step
    static constexpr int kStep = 16 * kTiles;
    static constexpr int kWide = D >= 128 ? 8 : 4;    // dims of a value that a lane holds together
    static constexpr int kParts = D / (16 * kWide);
    static constexpr int kTokens = 4 * kTiles;        // tokens whose values a lane loads
    static constexpr int kQ = (QK == kF32 ? 4 : 2) * D * 16;  // LDS bytes of the queries
    static constexpr int kAcc = D / 16;               // f4 of the output a lane holds
    static constexpr int kSave = kAcc * 1024 + 512;   // LDS bytes of one wave's state
    static constexpr int lds(int waves) { return kQ + waves / 2 * kSave; }

    static_assert(kTiles == 2 || PV == kF32, "the 16-bit products take 32 tokens");
};

template <typename C, int QK, int PV, int D, bool TILED>
__global__ __launch_bounds__(512) void k_attend(AttendArgs p)
{
    typedef Attend<C, QK, PV, D, TILED> S;
    constexpr int CS = S::kSize, E = S::kChunk, NC = S::kChunks, UT = S::kTiles, VW = S::kWide, NP = S::kParts, NT = S::kTokens;
    extern __shared__ __align__(16) char lds[];
    const detfold_attend &a = p.a;
    const detfold_paged_cache &c = p.c;
    const int lane = threadIdx.x & 63, col = lane & 15, grp = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const uint32_t per_row = divide(blockIdx.x, p.units), unit = blockIdx.x - per_row * p.units.d;
    const uint32_t row = divide(per_row, p.parts), part = per_row - row * p.parts.d;
    const uint32_t h = divide(unit, p.tiles), tile = unit - h * p.tiles.d;
    const int64_t b = p.row0 + row;
    const int head0 = (int)(h * p.group + 16 * tile);
    const int live = min(16, p.group - 16 * (int)tile);

    // The tokens of this part.
    const int32_t want = a.lens[b];
    const int64_t len = want > 0 ? want : 0;
    bool bad = len > a.max_len || len > a.table_width * c.page;
    const int64_t all = bad ? 0 : len, first = a.window > 0 && all > a.window ? all - a.window : 0;
    const uint32_t begin = (uint32_t)min(all, first + part * p.split), end = (uint32_t)min(all, first + (part + 1) * p.split);
    const uint32_t a0 = TILED ? begin & ~15u : begin, last = end > 0 ? end - 1 : 0;
    const uint32_t steps = end > begin ? (end - a0 + S::kStep - 1) / S::kStep : 0;

    // The queries as the operand of the score products, one lane's 16 bytes
    // after the other; a chunk that would pass the head's end starts earlier,
    // and what it repeats counts as zero.
    {
        constexpr int per = QK == kF32 ? 4 : 8;
        for (int i = threadIdx.x; i < D * 64 / (4 * per); i += blockDim.x) {
            const int l = i & 63, f = i >> 6;
            const int at = f * per / E, e0 = f * per % E, c0 = E * (4 * at + (l >> 4)), s = min(c0, c.dim - E);
            const int64_t q0 = b * a.q_row + (int64_t)(head0 + min(l & 15, live - 1)) * a.q_head + s + e0;
            float x[per];
#pragma unroll
            for (int e = 0; e < per; ++e) {
                const float v = QK == kF32 ? read_q<float>(a.q, q0 + e) : QK == kBf16 ? read_q<bf16>(a.q, q0 + e) : read_q<f16>(a.q, q0 + e);
                x[e] = s + e0 + e >= c0 && (l & 15) < live ? v : 0.0f;
            }
            if constexpr (QK == kF32)
                ((f4 *)lds)[i] = f4{x[0], x[1], x[2], x[3]};
            else if constexpr (QK == kBf16)
                ((bf16x8 *)lds)[i] = bf16x8{(bf16)x[0], (bf16)x[1], (bf16)x[2], (bf16)x[3], (bf16)x[4], (bf16)x[5], (bf16)x[6], (bf16)x[7]};
            else
                ((f16x8 *)lds)[i] = f16x8{(f16)x[0], (f16)x[1], (f16)x[2], (f16)x[3], (f16)x[4], (f16)x[5], (f16)x[6], (f16)x[7]};
        }
    }

    const int32_t *table = a.table + b * a.table_row;
    const char *k0 = (const char *)c.k + (int64_t)h * c.k_head * CS, *v0 = (const char *)c.v + (int64_t)h * c.v_head * CS;
    const int64_t k_page = c.k_page * CS, k_token = c.k_token * CS, v_page = c.v_page * CS, v_token = c.v_token * CS;
    const uint32_t pages = (uint32_t)c.pages;

    // Where a lane's loads lie within a key and a value.
    uint32_t k_at[NC], v_at[NP];
#pragma unroll
    for (int i = 0; i < NC; ++i)
        k_at[i] = (uint32_t)min(E * (4 * i + grp), c.dim - E) * CS + (TILED ? col * (uint32_t)k_token : 0);
#pragma unroll
    for (int i = 0; i < NP; ++i)
        v_at[i] = (uint32_t)min(VW * (16 * i + col), c.v_dim - VW) * CS + (TILED ? 4 * grp * (uint32_t)v_token : 0);

    // The table's entries of a step: one per tile where tiles lie within a
    // page, else one per token that this lane loads.  Tokens past the part are
    // taken from its last ones, and masked.
    int32_t id_k[UT], id_v[TILED ? 1 : NT];
    uint32_t off_k[UT], off_v[TILED ? 1 : NT];
    auto look_up = [&](uint32_t s) {
        const uint32_t t0 = a0 + s * S::kStep;
        if constexpr (TILED) {
#pragma unroll
            for (int u = 0; u < UT; ++u) {
                const uint32_t t = min(t0 + 16 * u, last & ~15u), n = divide(t, p.page);
                id_k[u] = table[n];
                off_k[u] = t - n * p.page.d;
            }
        } else {
#pragma unroll
            for (int u = 0; u < UT; ++u) {
                const uint32_t t = min(t0 + 16 * u + col, last), n = divide(t, p.page);
                id_k[u] = table[n];
                off_k[u] = t - n * p.page.d;
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const uint32_t t = min(t0 + 16 * (j / 4) + 4 * grp + j % 4, last), n = divide(t, p.page);
                id_v[j] = table[n];
                off_v[j] = t - n * p.page.d;
            }
        }
    };
    auto valid = [&](int32_t id) {  // the page, 0 for one that is none
        const bool no = (uint32_t)id >= pages;
        bad |= no;
        return (int64_t)(no ? 0 : id);
    };

    Words<16> kw[UT][NC];
    Words<VW * CS> vw[NT][NP];
    auto load_keys = [&] {
#pragma unroll
        for (int u = 0; u < UT; ++u) {
            const char *at = k0 + valid(id_k[u]) * k_page + off_k[u] * k_token;
#pragma unroll
            for (int i = 0; i < NC; ++i)
                kw[u][i] = load_words<16>(at + k_at[i]);
        }
    };
    auto load_values = [&] {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const char *at = TILED ? v0 + valid(id_k[j / 4]) * v_page + (off_k[j / 4] + j % 4) * v_token
                                   : v0 + valid(id_v[j]) * v_page + off_v[j] * v_token;
#pragma unroll
            for (int i = 0; i < NP; ++i)
                vw[j][i] = load_words<VW * CS>(at + v_at[i]);
        }
    };

    const float by = a.scale * (c.k_scale ? c.k_scale[h] : 1.0f) * kLog2e;
    const bool ragged = c.dim % (4 * E) != 0;
    // Weights of 16-bit floats are held 2^15 times larger, so that small ones
    // keep their digits; the sum is too, and both are put right at the end.
    constexpr float kLift = PV == kF16 ? 15.0f : 0.0f;
    float m = -INFINITY, l = 0.0f;
    f4 acc[NP][VW];
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int j = 0; j < VW; ++j)
            acc[i][j] = f4{0.0f, 0.0f, 0.0f, 0.0f};

    uint32_t s = wave;
    if (s < steps) {
        look_up(s);
        load_keys();
        load_values();
        if (s + waves < steps)
            look_up(s + waves);
    }
    __syncthreads();
    for (; s < steps; s += waves) {
        const uint32_t t0 = a0 + s * S::kStep;
        const bool more = s + waves < steps;
        // Scores: a row per token, a column per query head.
        f4 x[UT];
#pragma unroll
        for (int u = 0; u < UT; ++u) {
            x[u] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                if (CS != 1 && ragged) {  // what the last chunk repeats: zero times infinity would be NaN
                    const int drop = E * (4 * i + grp) - min(E * (4 * i + grp), c.dim - E);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int bits = 8 * CS * drop - 32 * j;
                        kw[u][i].w[j] &= bits >= 32 ? 0u : bits > 0 ? ~0u << bits : ~0u;
                    }
                }
                if constexpr (QK == kF32) {
#pragma unroll
                    for (int e = 0; e < E; e += 4) {
                        const f4 q = ((const f4 *)lds)[(i * (E / 4) + e / 4) * 64 + lane];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            x[u] = __builtin_amdgcn_mfma_f32_16x16x4f32(value32<C>(kw[u][i].w, e + j), q[j], x[u], 0, 0, 0);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < E; e += 8) {
                        const u4 q = ((const u4 *)lds)[(i * (E / 8) + e / 8) * 64 + lane];
                        const u4 k = {pair16<C, QK>(kw[u][i].w, e / 2), pair16<C, QK>(kw[u][i].w, e / 2 + 1),
                                      pair16<C, QK>(kw[u][i].w, e / 2 + 2), pair16<C, QK>(kw[u][i].w, e / 2 + 3)};
                        x[u] = mfma16<QK>(k, q, x[u]);
                    }
                }
            }
        }
        if (more)
            load_keys();
        // Weights, relative to the largest score so far.
        float top = -INFINITY;
        const bool edge = t0 < begin || t0 + S::kStep > end;
#pragma unroll
        for (int u = 0; u < UT; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[u][j] *= by;
                if (edge) {
                    const uint32_t t = t0 + 16 * u + 4 * grp + j;
                    x[u][j] = t < begin || t >= end ? -INFINITY : x[u][j];
                }
                top = fmaxf(top, x[u][j]);
            }
        top = fmaxf(m, over_groups(top, [](float y, float z) { return fmaxf(y, z); }));
        const float base = top == -INFINITY ? 0.0f : top;
        if (__any(top > m)) {
            const float turn = __builtin_amdgcn_exp2f(m - base);
            l *= turn;
#pragma unroll
            for (int i = 0; i < NP; ++i)
#pragma unroll
                for (int j = 0; j < VW; ++j)
                    acc[i][j] *= turn;
            m = top;
        }
#pragma unroll
        for (int u = 0; u < UT; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[u][j] = __builtin_amdgcn_exp2f((x[u][j] - base) + kLift);
                l += x[u][j];
            }
        // Values: the output's rows are its dims, its columns the query heads.
        if (edge) {  // what lies beyond the row's tokens may be anything
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const uint32_t t = t0 + 16 * (j / 4) + 4 * grp + j % 4;
                const bool out = t < begin || t >= end;
#pragma unroll
                for (int i = 0; i < NP; ++i)
#pragma unroll
                    for (int n = 0; n < VW * CS / 4; ++n)
                        vw[j][i].w[n] = out ? 0u : vw[j][i].w[n];
            }
        }
        if constexpr (PV == kF32) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < NP; ++i)
#pragma unroll
                    for (int n = 0; n < VW; ++n)
                        acc[i][n] = __builtin_amdgcn_mfma_f32_16x16x4f32(value32<C>(vw[j][i].w, n), x[j / 4][j % 4], acc[i][n], 0, 0, 0);
        } else {
            u4 w;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float y = x[j / 2][2 * (j % 2)], z = x[j / 2][2 * (j % 2) + 1];
                if constexpr (PV == kBf16)
                    w[j] = __builtin_bit_cast(uint32_t, bf16x2{(bf16)y, (bf16)z});
                else
                    w[j] = __builtin_bit_cast(uint32_t, f16x2{(f16)y, (f16)z});
            }
#pragma unroll
            for (int i = 0; i < NP; ++i)
#pragma unroll
                for (int n = 0; n < VW; n += 2) {
                    u4 lo, hi;  // dims n and n + 1 of the lane's eight tokens
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t y = pair16<C, PV>(vw[2 * j][i].w, n / 2), z = pair16<C, PV>(vw[2 * j + 1][i].w, n / 2);
                        lo[j] = __builtin_amdgcn_perm(z, y, 0x05040100u);
                        hi[j] = __builtin_amdgcn_perm(z, y, 0x07060302u);
                    }
                    acc[i][n] = mfma16<PV>(lo, w, acc[i][n]);
                    acc[i][n + 1] = mfma16<PV>(hi, w, acc[i][n + 1]);
                }
        }
        if (more) {
            load_values();
            if (s + 2 * waves < steps)
                look_up(s + 2 * waves);
        }
    }

    l = over_groups(l, [](float y, float z) { return y + z; });
    if (PV == kF16) {
        l *= 0x1p-15f;
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
            for (int j = 0; j < VW; ++j)
                acc[i][j] *= 0x1p-15f;
    }
    if (__any(bad))
        l = __builtin_nanf("");

    // The waves' states, joined pairwise in a fixed order.
    for (int n = waves / 2; n > 0; n >>= 1) {
        char *save = lds + S::kQ + (wave < n ? wave : wave - n) * S::kSave;
        if (wave >= n && wave < 2 * n) {
#pragma unroll
            for (int i = 0; i < S::kAcc; ++i)
                ((f4 *)save)[i * 64 + lane] = acc[i / VW][i % VW];
            ((f2 *)(save + S::kAcc * 1024))[lane] = f2{m, l};
        }
        __syncthreads();
        if (wave < n) {
            const f2 ml = ((const f2 *)(save + S::kAcc * 1024))[lane];
            const float top = fmaxf(m, ml.x), base = top == -INFINITY ? 0.0f : top;
            const float mine = __builtin_amdgcn_exp2f(m - base), theirs = __builtin_amdgcn_exp2f(ml.x - base);
            l = l * mine + ml.y * theirs;
            m = top;
#pragma unroll
            for (int i = 0; i < S::kAcc; ++i)
                acc[i / VW][i % VW] = acc[i / VW][i % VW] * mine + ((const f4 *)save)[i * 64 + lane] * theirs;
        }
        __syncthreads();
    }
    if (wave > 0 || col >= live)
        return;
    const int64_t g = b * a.q_heads + head0 + col;
    if (p.parts.d > 1) {
        const int64_t at = g * p.parts.d + part;
        if (grp == 0)
            p.ml[at] = make_float2(m, l);
        if (steps == 0)
            return;
        float *o = p.acc + at * c.v_dim;
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int d0 = VW * (16 * i + 4 * grp + j), d = min(d0, c.v_dim - VW);
                if (d0 < c.v_dim)
#pragma unroll
                    for (int n = 0; n < VW; ++n)
                        o[d + n] = acc[i][n][j];
            }
        return;
    }
    const float vs = c.v_scale ? c.v_scale[h] : 1.0f;
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int d0 = VW * (16 * i + 4 * grp + j), d = min(d0, c.v_dim - VW);
            float o[VW];
#pragma unroll
            for (int n = 0; n < VW; ++n)
                o[n] = attended(acc[i][n][j], vs, l);
            if (d0 < c.v_dim)
                put_out<VW>(a, b * a.out_row + (int64_t)(head0 + col) * a.out_head + d, o);
        }
    if (a.lse && grp == 0)
        a.lse[g] = log_sum(m, l);
}

// The kernel for a head size of at most D, if p says tiles lie within a page.
template <typename C, int QK, int PV, int D> AttendKernel pick_tiled(bool tiled)
{
    typedef Attend<C, QK, PV, D, true> S;
    return {tiled ? (const void *)k_attend<C, QK, PV, D, true> : (const void *)k_attend<C, QK, PV, D, false>, S::kQ, S::kSave};
}
template <typename C, int QK, int PV> AttendKernel pick_attend(int dim, bool tiled)
{
    return dim <= 64 ? pick_tiled<C, QK, PV, 64>(tiled) : dim <= 128 ? pick_tiled<C, QK, PV, 128>(tiled) : pick_tiled<C, QK, PV, 256>(tiled);
}

}  // namespace detfold_impl

#endif  // DETFOLD_ATTEND_KERNEL_H
