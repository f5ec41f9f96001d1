// attend_kernel.h -- the kernel of the paged attention: one new token per row
// over a paged key-value cache.  Included by the attend_*.hip files, each of
// which instantiates the kernels of one query type.
//
// Mathematics.  With s_t = scale * (q . k_t) a wave keeps, per query head, the
// largest score m so far, l = sum exp(s_t - m) and o = sum exp(s_t - m) v_t; a
// larger m' turns l and o by exp(m - m').  Two such states join the same way, so
// the tokens can be split over waves, workgroups and launches.  All is held in
// binary32; log2 e multiplies a score's distance from m, not the score, which
// could overflow.
//
// What bounds it.  Every key and value is read once from HBM and used for at
// most 16 query heads: 4 to 16 flop a byte, far below what the matrix units
// give.  So the design is about keeping the reads in flight:
// * Both products run on the matrix units with the cache as their first operand,
//   in the layout in which it is loaded: 16 tokens by 4 chunks of 16 bytes for
//   the scores.  The scores come out with a query head per lane column, which is
//   what the second product takes as its second operand, so the weights never
//   leave their lane; the values are transposed within a lane (two byte permutes
//   per two words), and nothing of the cache goes through LDS.
// * A wave's step is 64 tokens where the registers hold them (32 KiB of 128
//   bfloat16).  The next step's keys are loaded when this one's scores are done,
//   its values when this one's are used: 16 to 32 KiB in flight a wave, with 4
//   waves a compute unit (8 where a step is 16 KiB).
// * A workgroup's waves take different heads of the same tokens.  One head's 256
//   bytes at the 2 KiB stride of a token-major page fall on 2 of 16 L2 channels:
//   1 x 131072 bfloat16 took 101 us that way, 90 this way.
// * Workgroups take even shares of all rows' tokens, found from the lengths on
//   the device: 64 ragged rows took 281 us in parts of a fixed size, 160 so.
//
// Measured (MI355X, GPU time of the call with its join): 1 x 131072 bfloat16, 32
// heads over 8 of 128: 90 us, 6.0 TB/s; 64 ragged rows of up to 8192: 161 us, 6.3
// TB/s; 256 x 4096 e4m3: 328 us, 6.6 TB/s; 16 x 16384 float32: 316 us, 6.8 TB/s;
// one row of 1000: 11.5 us, of which the loads' dependent latencies are 6 and the
// join's launch 4.
//
// Weights are rounded to the cache's 16-bit type for the second product where
// the output is of 16 bits too: half a step of what the output itself is rounded
// to (0.0017 to 0.0019 relative against the definition, 0.0017 with float32 weights).  A
// float32 output takes them whole.
#ifndef DETFOLD_ATTEND_KERNEL_H
#define DETFOLD_ATTEND_KERNEL_H

#include "decode_device.h"

namespace detfold_impl {

// What the matrix units multiply.  kSplit: float32 queries or weights as the sum
// of three bfloat16 ones (24 bits in all, so exact), with keys or values of e4m3;
// three products of those take 3/8 of the time of one in float32.  Only where no
// key or value is infinite: a third part may be zero.
enum Math { kBf16, kF16, kF32, kSplit };

typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// N bytes of the cache at any alignment that a head's start may have (one wide
// load all the same); once: not kept in the caches.
template <int N> struct Words {
    uint32_t w[N / 4];
};
template <int N, bool ONCE> __device__ __forceinline__ Words<N> load_words(const char *p)
{
    typedef uint32_t v4 __attribute__((ext_vector_type(4), aligned(1)));
    typedef uint32_t v2 __attribute__((ext_vector_type(2), aligned(1)));
    typedef uint32_t v1 __attribute__((aligned(1)));
    Words<N> r;
    if constexpr (N >= 16) {
#pragma unroll
        for (int i = 0; i < N / 16; ++i) {
            const v4 x = ONCE ? __builtin_nontemporal_load((const v4 *)p + i) : ((const v4 *)p)[i];
            r.w[4 * i] = x.x, r.w[4 * i + 1] = x.y, r.w[4 * i + 2] = x.z, r.w[4 * i + 3] = x.w;
        }
    } else if constexpr (N == 8) {
        const v2 x = ONCE ? __builtin_nontemporal_load((const v2 *)p) : *(const v2 *)p;
        r.w[0] = x.x, r.w[1] = x.y;
    } else {
        r.w[0] = ONCE ? __builtin_nontemporal_load((const v1 *)p) : *(const v1 *)p;
    }
    return r;
}

// Two neighbouring values of the cache as the 16-bit type of the matrix units
// (exact), and as floats.
template <typename C, int M> __device__ __forceinline__ uint32_t pair16(const uint32_t *w, int i)
{
    if constexpr (sizeof(C) == 2)
        return w[i];
    else if constexpr (M != kF16)
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
    if constexpr (M != kF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// What a float32's upper half, a bfloat16, leaves of it: exact, and zero for an
// infinity, whose upper half is all of it.
__device__ __forceinline__ uint32_t below(uint32_t x)
{
    const float up = __builtin_bit_cast(float, x & 0xffff0000u), rest = __builtin_bit_cast(float, x) - up;
    return up - up == 0.0f ? __builtin_bit_cast(uint32_t, rest) : 0u;
}

// Over the four groups of 16 lanes, the same on all of them.
template <typename F> __device__ __forceinline__ float over_groups(float x, F f)
{
    const auto a = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
    x = f(__builtin_bit_cast(float, (uint32_t)a[0]), __builtin_bit_cast(float, (uint32_t)a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
    return f(__builtin_bit_cast(float, (uint32_t)b[0]), __builtin_bit_cast(float, (uint32_t)b[1]));
}

// A uniform read of what no kernel writes meanwhile.  As a vector load it
// would be counted with the loads of the cache, in order, and waiting for it
// would wait for them.
template <typename T> __device__ __forceinline__ T scalar_load(const T *p) { return *(const __attribute__((address_space(4))) T *)p; }

// The kernel's arguments, read anew: held across a loop they would fill the
// scalar registers, and then vector ones.
typedef const __attribute__((address_space(4))) AttendArgs *ArgsPtr;
__device__ __forceinline__ const AttendArgs &arguments()
{
    uint64_t p = (uint64_t)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *(const AttendArgs *)(ArgsPtr)p;
}

// The same value, of which the compiler knows nothing: what is computed from it
// in a loop is not held in registers across it.
template <typename T> __device__ __forceinline__ T anew(T x)
{
    asm volatile("" : "+v"(x));
    return x;
}

// The bits of the j-th of some words that lie n bytes or more from the start.
__device__ __forceinline__ uint32_t keep_from(int n, int j)
{
    const int bits = 8 * n - 32 * j;
    return bits >= 32 ? 0u : bits > 0 ? ~0u << bits : ~0u;
}

// exp of a score's distance from the largest one (-infinity: 0); times 2^lift.
template <int LIFT = 0> __device__ __forceinline__ float weight_of(float s)
{
    return __builtin_amdgcn_exp2f(LIFT ? __builtin_fmaf(s, kLog2e, (float)LIFT) : s * kLog2e);
}

// The ends of a row: what its sums are multiplied by (one division a row; a
// row without a token gives 0), the logarithm of its weights' sum, and the store
// of N values.
__device__ __forceinline__ float out_scale(float v_scale, float l) { return l == 0.0f ? 0.0f : v_scale / l; }
__device__ __forceinline__ float log_sum(float m, float l) { return (m == -INFINITY ? 0.0f : m) + logf(l); }
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

// The tokens of a row that are seen, in units from a0 on (a row without any
// counts as one, so that someone writes its output).
struct RowTokens {
    uint32_t begin, end, a0, units;
    bool bad;  // longer than the call or the table allows
};
__device__ __forceinline__ RowTokens row_tokens(const AttendArgs &p, int32_t len, bool tiled)
{
    const int64_t n = len > 0 ? len : 0;
    RowTokens r;
    r.bad = n > p.a.max_len || n > p.a.table_width * p.c.page;
    r.end = r.bad ? 0 : (uint32_t)n;
    r.begin = p.a.window > 0 && r.end > p.a.window ? (uint32_t)(r.end - p.a.window) : 0;
    r.a0 = tiled ? r.begin & ~15u : r.begin;
    r.units = r.end > r.begin ? (r.end - r.a0 + kUnit - 1) / kUnit : 1;
    return r;
}

// An even share of all rows' units, found by every wave from the lengths:
// share y has the units [y * each, (y + 1) * each) of the rows laid end to end.
struct Share {
    uint32_t left, at, row_at, each;  // units left, the next one, its row's first one, those of a share
    int32_t row, len;                 // that row and its length
};
__device__ __forceinline__ Share find_share(const AttendArgs &p, uint32_t y, bool tiled)
{
    const int lane = threadIdx.x & 63, batch = (int)p.a.batch;
    auto length = [&](int i) { return i < batch ? p.a.lens[i] : 0; };
    auto units = [&](int i, int32_t len) { return i < batch ? row_tokens(p, len, tiled).units : 0u; };
    int32_t len = length(lane);
    uint32_t total = 0;
    for (int i = lane + 64; i < batch; i += 64)
        total += units(i, length(i));
    Share w = {};
    uint32_t before = 0;
    for (int i = 0; i < batch; i += 64) {
        const uint32_t own = units(i + lane, len);
        uint32_t upto = own;
#pragma unroll
        for (int n = 1; n < 64; n <<= 1) {
            const uint32_t other = __shfl_up(upto, n);
            upto += lane >= n ? other : 0;
        }
        const uint32_t here = __builtin_amdgcn_readlane(upto, 63);
        if (i == 0) {
            if (batch > 64)
#pragma unroll
                for (int n = 32; n > 0; n >>= 1)
                    total += __shfl_xor(total, n);
            total = __builtin_amdgcn_readfirstlane(total) + here;
            w.each = divide(total + p.shares.d - 1, p.shares);
            w.at = y * w.each;
            if (w.at >= total)
                return w;
            w.left = min(w.each, total - w.at);
        }
        const uint64_t past = __ballot(before + upto > w.at);
        if (past) {
            const int at = __builtin_ctzll(past);
            w.row = i + at;
            w.row_at = before + __builtin_amdgcn_readlane(upto, at) - __builtin_amdgcn_readlane(own, at);
            w.len = __builtin_amdgcn_readlane(len, at);
            break;
        }
        before += here;
        len = length(i + 64 + lane);
    }
    return w;
}

template <bool B> struct Last {
    static constexpr bool value = B;
};

// What follows from the types C of the cache, QK and PV of the two products, and
// from the head class D.  TILED: 16 tokens lie within a page.  MOST: tiles of 16
// tokens in a step, at most.  KEEP: what the caches keep.
template <typename C, int QK, int PV, int D, bool TILED, int MOST, int KEEP> struct Attend {
    static constexpr int kSize = sizeof(C);
    static constexpr int kChunk = 16 / kSize;         // dims of one 16-byte load of a key
    static constexpr int kChunks = D / (4 * kChunk);  // of these per lane and key
    static constexpr int kFit = 1024 / (D * kSize);   // tiles of 16 tokens whose keys take 64 registers
    // Halves converted to float32 are held apart, in twice the registers.
    static constexpr bool kTwice = __is_same(C, f16) && PV == kF32;
    static constexpr int kMost = D < 256 ? (kTwice ? 2 : MOST) : PV == kF32 && (QK == kF32 || kTwice) ? 1 : 2;
    static constexpr int kTiles = kFit < kMost ? kFit : kMost;  // of a step
    static constexpr int kStep = 16 * kTiles;
    static constexpr int kWide = kChunk < D / 16 ? kChunk : D / 16;  // dims of a value that a lane loads together
    static constexpr int kParts = D / (16 * kWide);
    static constexpr int kTokens = 4 * kTiles;        // tokens whose values a lane loads
    static constexpr int kQ = (QK == kF32 ? 4 : QK == kSplit ? 6 : 2) * D * 16;  // LDS bytes of the queries
    static constexpr int kRow = D + 4;                // floats of a query head's sums in LDS: heads on other banks

    static_assert(kTiles % 2 == 0 || PV == kF32, "the 16-bit products take 32 tokens");
};

template <typename C, int QK, int PV, int D, bool TILED, int MOST, int KEEP>
__global__ __launch_bounds__(512) void k_attend(AttendArgs)
{
    typedef Attend<C, QK, PV, D, TILED, MOST, KEEP> S;
    constexpr int CS = S::kSize, E = S::kChunk, NC = S::kChunks, UT = S::kTiles, VW = S::kWide, NP = S::kParts, NT = S::kTokens;
    extern __shared__ __align__(16) char lds[];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const AttendArgs &p0 = arguments();
    const uint32_t y = divide(blockIdx.x, p0.units);
    // A wave takes one of the workgroup's units, or one of several turns at it.
    const int beside = p0.beside, in = wave & (beside - 1), turn = wave / beside, turns = waves / beside;
    const uint32_t unit = (blockIdx.x - y * p0.units.d) * beside + in;

    // The work of this workgroup: one part of one row, or its even share of the
    // steps of all rows, which may begin and end within one.
    int64_t b;
    uint32_t part = 0;
    Share mine = {};
    if (p0.shares.d) {
        mine = find_share(p0, y, TILED);
        if (mine.left == 0) {
            if (!p0.by_row && unit == 0 && threadIdx.x == 0)
                p0.cut[y] = make_int3(-1, 0, 0);
            return;
        }
        b = mine.row;
    } else {
        const uint32_t row = divide(y, p0.parts);
        part = y - row * p0.parts.d;
        b = p0.row0 + row;
        mine.len = scalar_load(p0.a.lens + b);
    }

    for (;;) {
        const AttendArgs &p = arguments();
        const detfold_attend &a = p.a;
        const detfold_paged_cache &c = p.c;
        const int lane = anew((int)threadIdx.x & 63), col = lane & 15, grp = lane >> 4;
        const uint32_t h = divide(unit, p.tiles), tile = unit - h * p.tiles.d;
        const int head0 = (int)(h * p.group + 16 * tile);
        const int live = min(16, p.group - 16 * (int)tile);
        const char *k0 = (const char *)c.k + (int64_t)h * c.k_head * CS, *v0 = (const char *)c.v + (int64_t)h * c.v_head * CS;
        const int64_t k_page = c.k_page * CS, k_token = c.k_token * CS, v_page = c.v_page * CS, v_token = c.v_token * CS;
        const uint32_t pages = (uint32_t)c.pages;
        const float by = a.scale * (c.k_scale ? scalar_load(c.k_scale + h) : 1.0f);
        const float v_scale = c.v_scale ? scalar_load(c.v_scale + h) : 1.0f;

        // Where a lane's loads lie within a key and a value.
        uint32_t k_at[NC], v_at[NP];
#pragma unroll
        for (int i = 0; i < NC; ++i)
            k_at[i] = (uint32_t)min(E * (4 * i + grp), c.dim - E) * CS + (TILED ? col * (uint32_t)k_token : 0);
#pragma unroll
        for (int i = 0; i < NP; ++i)
            v_at[i] = (uint32_t)min(VW * (16 * i + col), c.v_dim - VW) * CS + (TILED ? 4 * grp * (uint32_t)v_token : 0);

        const RowTokens row = row_tokens(p, mine.len, TILED);
        bool bad = row.bad;
        uint32_t begin = row.begin, end = row.end, done = 0;
        int64_t slot = -1;  // where the sums of this part go if the row has others
        if (p.shares.d) {
            const uint32_t x = mine.at - mine.row_at;
            done = min(row.units - x, mine.left);
            if (done < row.units)
                slot = ((int64_t)y * (p.units.d * beside) + unit) * 2 + (x == 0);
            if (unit == 0 && lane == 0 && turn == 0 && (p.by_row ? x == 0 : done == mine.left)) {
                const bool cut = x == 0 && done < row.units;  // it begins here, and does not end here
                p.cut[p.by_row ? b : y] = make_int3(cut ? (int)b : -1, (int)y, cut ? (int)((mine.at + row.units - 1) / mine.each) : 0);
            }
            end = x + done < row.units ? row.a0 + kUnit * (x + done) : end;
            begin = x ? row.a0 + kUnit * x : begin;
        } else if (p.parts.d > 1) {
            slot = (b * p.parts.d + part) * (p.units.d * beside) + unit;
            const int64_t x = begin + part * p.split;
            begin = (uint32_t)min(x, (int64_t)end), end = (uint32_t)min(x + p.split, (int64_t)end);
        }
        const uint32_t a0 = TILED ? begin & ~15u : begin, last = end > 0 ? end - 1 : 0;
        const uint32_t steps = end > begin ? (end - a0 + S::kStep - 1) / S::kStep : 0;

        // The queries as the operand of the score products, one lane's 16 bytes
        // after the other; a chunk that would pass the head's end starts earlier,
        // and what it repeats counts as zero.
        char *const queries = lds + in * S::kQ;
        constexpr int QS = QK == kF32 || QK == kSplit ? 4 : 2, PER = QK == kF32 ? 4 : 8, NQ = D / (4 * PER);
        const char *q = (const char *)a.q + (b * a.q_row + (int64_t)(head0 + min(col, live - 1)) * a.q_head) * QS;
        auto query_chunk = [&](int i) { return E * (4 * (i * PER / E) + grp); };
        Words<PER * QS> qw[NQ] = {};
#pragma unroll
        for (int i = 0; i < NQ; ++i)
            if ((i & (turns - 1)) == turn)
                __builtin_memcpy(&qw[i], q + (min(query_chunk(i), c.dim - E) + i * PER % E) * QS, PER * QS);

        const int32_t *table = a.table + b * a.table_row;
        // The pages of a step's tokens, looked up two steps ahead of the products:
        // where tiles lie within a page one scalar each, else one per lane and
        // token, handed to the lanes that load it when it is used.  Tokens past the
        // part are taken from its last ones, and masked.
        constexpr int IDS = TILED ? UT : 1;
        const uint32_t own = lane & (S::kStep - 1);
        struct Pages {
            int32_t id[IDS];
            uint32_t off[IDS];
        };
        auto look_up = [&](uint32_t s) {
            const uint32_t t0 = a0 + s * S::kStep;
            Pages g;
#pragma unroll
            for (int u = 0; u < IDS; ++u) {
                const uint32_t t = TILED ? min(t0 + 16 * u, last & ~15u) : min(t0 + own, last), n = divide(t, p.page);
                g.id[u] = TILED ? scalar_load(table + n) : table[n];
                g.off[u] = t - n * p.page.d;
            }
            return g;
        };
        auto valid = [&](int32_t id) {  // the page, 0 for one that is none
            const bool no = (uint32_t)id >= pages;
            bad |= no;
            return (int64_t)(no ? 0 : id);
        };

        Words<16> kw[UT][NC];
        Words<VW * CS> vw[NT][NP];
        auto load_keys = [&](const Pages &g) {
            int64_t at = 0;
            if (!TILED)
                at = valid(g.id[0]) * k_page + g.off[0] * k_token;
#pragma unroll
            for (int u = 0; u < UT; ++u) {
                const char *k = k0 + (TILED ? valid(g.id[u % IDS]) * k_page + g.off[u % IDS] * k_token : from_lane(at, 16 * u + col));
#pragma unroll
                for (int i = 0; i < NC; ++i)
                    kw[u][i] = load_words<16, KEEP == kNothing>(k + anew(k_at[i]));
            }
        };
        auto load_values = [&](const Pages &g) {
            int64_t at = 0;
            if (!TILED)
                at = valid(g.id[0]) * v_page + g.off[0] * v_token;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const char *v = v0 + (TILED ? valid(g.id[j / 4 % IDS]) * v_page + (g.off[j / 4 % IDS] + j % 4) * v_token
                                            : from_lane(at, 16 * (j / 4) + 4 * grp + j % 4));
#pragma unroll
                for (int i = 0; i < NP; ++i)
                    vw[j][i] = load_words<VW * CS, KEEP != kAll>(v + anew(v_at[i]));
            }
        };

        // Weights of 16-bit floats are held 2^15 times larger, so that small ones
        // keep their digits; the sum is too, and both are put right at the end.
        constexpr int kLift = PV == kF16 ? 15 : 0;
        float m = -INFINITY, l = 0.0f;
        f4 acc[NP][VW];
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
            for (int j = 0; j < VW; ++j)
                acc[i][j] = f4{0.0f, 0.0f, 0.0f, 0.0f};

        uint32_t s = turn;
        Pages now = {}, next = {};
        if (s < steps)
            now = look_up(s);
#pragma unroll
        for (int i = 0; i < NQ; ++i)
            if ((i & (turns - 1)) == turn) {
                const int drop = query_chunk(i) - min(query_chunk(i), c.dim - E) - i * PER % E;
#pragma unroll
                for (int j = 0; j < PER * QS / 4; ++j)
                    qw[i].w[j] = col < live ? qw[i].w[j] & keep_from(drop * QS, j) : 0u;
                if constexpr (QK == kSplit) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)  // a NaN whose bits all lie below the first part's would be an infinity there
                        qw[i].w[j] = __builtin_isnan(__builtin_bit_cast(float, qw[i].w[j])) ? 0x7fc00000u : qw[i].w[j];
#pragma unroll
                    for (int part = 0; part < 3; ++part) {  // the highest bits, of which two values' are stored together
                        u4 w;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            w[j] = __builtin_amdgcn_perm(qw[i].w[2 * j + 1], qw[i].w[2 * j], 0x07060302u);
                            qw[i].w[2 * j] = below(qw[i].w[2 * j]), qw[i].w[2 * j + 1] = below(qw[i].w[2 * j + 1]);
                        }
                        *(u4 *)(queries + (part * NQ + i) * 1024 + lane * 16) = w;
                    }
                } else {
                    *(u4 *)(queries + i * 1024 + lane * 16) = u4{qw[i].w[0], qw[i].w[1], qw[i].w[2], qw[i].w[3]};
                }
            }
        if (D == 256)  // else the queries' registers add to those of the loads below
            __builtin_amdgcn_sched_barrier(0);
        if (s < steps) {
            load_keys(now);
            load_values(now);
            now = look_up(min(s + turns, steps - 1));
        }
        __syncthreads();
        // One step; but for the last one it also issues the next one's loads, and
        // is compiled for that alone: with a branch instead, the wait for the values
        // would have to take the keys issued after them for values not yet there.
        auto step = [&](auto last_one) {
            constexpr bool more = !decltype(last_one)::value;
            const uint32_t t0 = a0 + s * S::kStep;
            const uint32_t q_at = anew(lane) * 16;
            // Scores: a row per token, a column per query head.
            f4 x[UT];
#pragma unroll
            for (int u = 0; u < UT; ++u)
                x[u] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                // Chunks past the head's end are not multiplied, and what the one at
                // its end repeats is cleared: there the queries are zero, but zero times
                // an infinite key would be NaN (an e4m3 key is never infinite).
                if (4 * E * i >= c.dim)
                    break;
                if (CS != 1 && 4 * E * (i + 1) > c.dim) {
                    const int at = E * (4 * i + anew(grp)), drop = at - min(at, c.dim - E);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t keep = keep_from(CS * drop, j);
#pragma unroll
                        for (int u = 0; u < UT; ++u)
                            kw[u][i].w[j] &= keep;
                    }
                }
#pragma unroll
                for (int u = 0; u < UT; ++u) {
                    if constexpr (QK == kF32) {
#pragma unroll
                        for (int e = 0; e < E; e += 4) {
                            const f4 q = *(const f4 *)(queries + (i * (E / 4) + e / 4) * 1024 + q_at);
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                x[u] = __builtin_amdgcn_mfma_f32_16x16x4f32(value32<C>(kw[u][i].w, e + j), q[j], x[u], 0, 0, 0);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < E; e += 8) {
                            const u4 k = {pair16<C, QK>(kw[u][i].w, e / 2), pair16<C, QK>(kw[u][i].w, e / 2 + 1),
                                          pair16<C, QK>(kw[u][i].w, e / 2 + 2), pair16<C, QK>(kw[u][i].w, e / 2 + 3)};
#pragma unroll
                            for (int part = 0; part < (QK == kSplit ? 3 : 1); ++part) {
                                const u4 q = *(const u4 *)(queries + (part * NQ + i * (E / 8) + e / 8) * 1024 + q_at);
                                x[u] = mfma16<QK>(k, q, x[u]);
                            }
                        }
                    }
                }
            }
            if constexpr (more) {
                next = look_up(min(s + 2 * turns, steps - 1));
                load_keys(now);
            }
            // Weights, relative to the largest score so far.
            float top = -INFINITY;
            const bool edge = t0 < begin || t0 + S::kStep > end;
            if (edge) {  // tokens of other parts, or none: their scores take no weight, and their values may be anything
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const uint32_t t = t0 + 16 * (j / 4) + 4 * grp + j % 4;
                    const bool out = t < begin || t >= end;
                    x[j / 4][j % 4] = out ? -INFINITY : x[j / 4][j % 4] * by;
#pragma unroll
                    for (int i = 0; i < NP; ++i)
#pragma unroll
                        for (int n = 0; n < VW * CS / 4; ++n)
                            vw[j][i].w[n] = out ? 0u : vw[j][i].w[n];
                }
            } else {
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    x[j / 4][j % 4] *= by;
            }
#pragma unroll
            for (int j = 0; j < NT; ++j)
                top = fmaxf(top, x[j / 4][j % 4]);
            top = fmaxf(m, over_groups(top, [](float y, float z) { return fmaxf(y, z); }));
            const float base = top == -INFINITY ? 0.0f : top;
            if (__any(top > m)) {
                const float turn = weight_of(m - base);
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
                    x[u][j] = weight_of<kLift>(x[u][j] - base);
                    l += x[u][j];
                }
            // Values: the output's rows are its dims, its columns the query heads.
            if constexpr (PV == kF32) {
#pragma unroll
                for (int j = 0; j < NT; ++j) {
#pragma unroll
                    for (int i = 0; i < NP; ++i)
#pragma unroll
                        for (int n = 0; n < VW; ++n)
                            acc[i][n] = __builtin_amdgcn_mfma_f32_16x16x4f32(value32<C>(vw[j][i].w, n), x[j / 4][j % 4], acc[i][n], 0, 0, 0);
                }
            } else {
#pragma unroll
                for (int u = 0; u < UT; u += 2) {
                    constexpr int TERMS = PV == kSplit ? 3 : 1;
                    u4 w[TERMS];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float y = x[u + j / 2][2 * (j % 2)], z = x[u + j / 2][2 * (j % 2) + 1];
                        if constexpr (PV == kF16) {
                            w[0][j] = __builtin_bit_cast(uint32_t, f16x2{(f16)y, (f16)z});
                        } else {
#pragma unroll
                            for (int n = 0; n < TERMS; ++n) {
                                const bf16x2 part = {(bf16)y, (bf16)z};
                                w[n][j] = __builtin_bit_cast(uint32_t, part);
                                y -= (float)part.x, z -= (float)part.y;
                            }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < NP; ++i)
#pragma unroll
                        for (int n = 0; n < VW; n += 2) {
                            u4 lo, hi;  // dims n and n + 1 of the lane's eight tokens
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint32_t y = pair16<C, PV>(vw[4 * u + 2 * j][i].w, n / 2), z = pair16<C, PV>(vw[4 * u + 2 * j + 1][i].w, n / 2);
                                lo[j] = __builtin_amdgcn_perm(z, y, 0x05040100u);
                                hi[j] = __builtin_amdgcn_perm(z, y, 0x07060302u);
                            }
#pragma unroll
                            for (int e = 0; e < TERMS; ++e) {
                                acc[i][n] = mfma16<PV>(lo, w[e], acc[i][n]);
                                acc[i][n + 1] = mfma16<PV>(hi, w[e], acc[i][n + 1]);
                            }
                        }
                }
            }
            if constexpr (more) {
                load_values(now);
                now = next;
            }
        };
        for (; s + turns < steps; s += turns)
            step(Last<false>{});
        if (s < steps)
            step(Last<true>{});

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

        // The waves' states, joined in order: each leaves its heads' sums in LDS,
        // over the queries, and a thread takes four dims of a head from every turn.
        const int heads = min(16, p.group);
        f2 *const state = (f2 *)lds;
        float *const sums = (float *)(lds + waves * 16 * sizeof(f2));
        __syncthreads();
        if (col < live) {
            float *mine = sums + (wave * heads + col) * S::kRow;
#pragma unroll
            for (int i = 0; i < NP; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int n = 0; n < VW; n += 4)
                        *(f4 *)(mine + VW * (16 * i + 4 * grp + j) + n) = f4{acc[i][n][j], acc[i][n + 1][j], acc[i][n + 2][j], acc[i][n + 3][j]};
            if (grp == 0)
                state[wave * 16 + col] = f2{m, l};
        }
        __syncthreads();
        const AttendArgs &pe = arguments();
        for (int i = 64 * turn + lane; i < live * (D / 4); i += 64 * turns) {
            const AttendArgs &p = pe;
            const detfold_attend &a = p.a;
            const int head = i / (D / 4), at = i % (D / 4) * 4, at0 = at / VW * VW;
            if (at0 >= p.c.v_dim)
                continue;
            float top = -INFINITY;
            for (int w = in; w < waves; w += beside)
                top = fmaxf(top, state[w * 16 + head].x);
            const float base = top == -INFINITY ? 0.0f : top;
            f4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
            float total = 0.0f;
            for (int w = in; w < waves; w += beside) {
                const f2 ml = state[w * 16 + head];
                const float by = weight_of(ml.x - base);
                total += ml.y * by;
                sum += *(const f4 *)(sums + (w * heads + head) * S::kRow + at) * by;
            }
            const int64_t g = b * a.q_heads + head0 + head, from = slot * heads + head;
            const int d = min(at0, p.c.v_dim - VW) + at - at0;
            if (slot >= 0) {
                __builtin_memcpy(p.acc + from * p.c.v_dim + d, &sum, sizeof(sum));
                if (at == 0)
                    p.ml[from] = make_float2(top, total);
            } else {
                const float by = out_scale(v_scale, total);
                const float o[4] = {sum.x * by, sum.y * by, sum.z * by, sum.w * by};
                put_out<4>(a, b * a.out_row + (int64_t)(head0 + head) * a.out_head + d, o);
                if (a.lse && at == 0)
                    a.lse[g] = log_sum(top, total);
            }
        }
        mine.left -= done;
        if (mine.left == 0)
            return;
        mine.at = mine.row_at = mine.at + done;
        ++b;
        mine.len = scalar_load(arguments().a.lens + b);
        __syncthreads();
    }
}

// The kernel of a call, of those that one can need: short steps read little and
// keep it, and only whole rows of 512 bytes or more keep nothing.
template <typename C, int QK, int PV, int D, int MOST, int KEEP> AttendKernel pick_tiled(const AttendArgs &a)
{
    typedef Attend<C, QK, PV, D, true, MOST, KEEP> S;
    const void *f = a.tiled ? (const void *)k_attend<C, QK, PV, D, true, MOST, KEEP>
                            : (const void *)k_attend<C, QK, PV, D, false, MOST, KEEP == kNothing ? kKeys : KEEP>;
    return {f, S::kQ, S::kRow * 4};
}
template <typename C, int QK, int PV, int D> AttendKernel pick_steps(const AttendArgs &a)
{
    if constexpr (Attend<C, QK, PV, D, true, 4, kAll>::kTiles > 2)
        if (a.brief)
            return pick_tiled<C, QK, PV, D, 2, kAll>(a);
    if constexpr (D * sizeof(C) >= 512)
        if (a.keep == kNothing)
            return pick_tiled<C, QK, PV, D, 4, kNothing>(a);
    return a.keep == kAll ? pick_tiled<C, QK, PV, D, 4, kAll>(a) : pick_tiled<C, QK, PV, D, 4, kKeys>(a);
}
template <typename C, int QK, int PV> AttendKernel pick_attend(const AttendArgs &a)
{
    const int dim = a.c.dim > a.c.v_dim ? a.c.dim : a.c.v_dim;
    return dim <= 64 ? pick_steps<C, QK, PV, 64>(a) : dim <= 128 ? pick_steps<C, QK, PV, 128>(a) : pick_steps<C, QK, PV, 256>(a);
}

}  // namespace detfold_impl

#endif  // DETFOLD_ATTEND_KERNEL_H
