// tree_kernel.h -- the kernel of the attention of drafted tokens: up to 64 new
// tokens per row over a paged key-value cache, each seeing the row's prefix and
// its own branch.  Included by the tree_*.hip files, each of which instantiates
// the kernels of one query type.
//
// Mathematics and layouts as in attend_kernel.h, with scores times log2 e.  The
// columns of both products are a key-value head's queries, drafted token by drafted
// token, 16 * QT of them to a wave, so that what is loaded of the cache serves QT
// products.  A capped score is cap * tanh(s / cap); a biased one gets slope *
// (position of the token - position of the query); what a query does not see scores
// -infinity.
//
// What bounds it.  Up to 32 queries of a key-value head: the cache's bytes, read once
// straight to registers (64 ragged rows of 8 drafted tokens over 8192 bfloat16 tokens
// of 8 heads of 128: 181 us, 5.5 TB/s; of one capped token each over their last 4096:
// 126 us, 5.8; 32 x 8192 e4m3: 93 us, 5.8).  Above: the instructions around the
// products, 8 cycles a score and lane, so that waves which take the same tokens share
// them through LDS (32 rows of 64 drafted tokens over 4096, capped: 281 us, 488
// TFLOP/s with the vector units busy three quarters of the time; 377 us straight to
// registers).  Small calls: the code, run once (1 x 8 over 1000: 17 us).  So:
// * Steps all of whose tokens all queries see hold no code for masks, or jump over it;
//   with masks in the loop their uniform values filled the scalar registers (1 x 8 over
//   1000 25 us, 32 x 64 over 4096 419).  A mask is looked at four tokens at a time.
// * Values that are infinite or no number are zeroed where some query may not see them
//   (zero times them is NaN), and added at the end, once, to the sums of those that do.
// * A capped score takes 9 instructions below half its cap, a polynomial, and 19 where a
//   wave has one above.
//
// Fewer bits.  As in attend_kernel.h the weights are rounded to the 16-bit type that the
// matrix units multiply where the output is of 16 bits too, and a float32 output takes
// them whole.  Against the definition the measured bfloat16 cases are off by 0.0017 to
// 0.0018 relative, where weights of 32 bits and the output's rounding alone give 0.0016
// to 0.0017; a model in 64 bits of flat scores over 8192 tokens, whose outputs are small
// beside the values, 0.0022 and 0.0016 (scores of a spread of 0.5: 0.0024 and 0.0017).
// The other choice, a second product for what the rounding leaves, would double the
// second products and their weights' conversions.
#ifndef DETFOLD_TREE_KERNEL_H
#define DETFOLD_TREE_KERNEL_H

#include "attend_kernel.h"
#include "draft.h"

namespace detfold_impl {

typedef const __attribute__((address_space(4))) TreeArgs *TreeArgsPtr;
__device__ __forceinline__ const TreeArgs &tree_arguments()
{
    uint64_t p = (uint64_t)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *(const TreeArgs *)(TreeArgsPtr)p;
}

// tanh, held to 24 units of 2^-24 relative.  Below 0.5 x + x^3 P(x^2), whose four
// coefficients were fitted to the smallest relative error (1.3 units there); above
// from exp(-2 |x|), of which the largest, e^-1, gives 4.  `line` is a score without its
// cap, y that over the cap.  A score's bits are its own: whether a wave takes near_cap
// for all of its scores or any_cap goes by the largest, and so by slots that no query
// sees, but below 0.5 both give the same to the last bit.
__device__ __forceinline__ float near_cap(float line, float y)
{
    const float z = y * y, p = __builtin_fmaf(__builtin_fmaf(__builtin_fmaf(z, 0.0172357764f, -0.0530423597f), z, 0.133258238f), z, -0.333331406f);
    return __builtin_fmaf(line * z, p, line);
}
__device__ __forceinline__ float any_cap(float line, float y, float cap)
{
    const float e = __builtin_amdgcn_exp2f(__builtin_fabsf(y) * (-2.0f * kLog2e));
    float near = near_cap(line, y), far = cap * __builtin_copysignf((1.0f - e) * __builtin_amdgcn_rcpf(1.0f + e), y);
    asm("" : "+v"(near), "+v"(far));  // both, without a branch for each
    return __builtin_fabsf(y) < 0.5f ? near : far;
}

// Scores are held times log2 e here, so that a weight is exp2 of a distance: a score
// of more than 2^127 / log2 e counts as infinite.
__device__ __forceinline__ float weight2_of(float s) { return __builtin_amdgcn_exp2f(s); }
__device__ __forceinline__ float log_sum2(float m, float l) { return (m == -INFINITY ? 0.0f : m * 0.693147181f) + logf(l); }

// What a query of a column goes by.
struct Column {
    uint64_t mask;
    int32_t at;  // its position
    float slope;  // times log2 e
};

// Whether words of the cache hold a value that is infinite or no number: what `seen`
// gathers from each, and what that says.
typedef uint16_t h2 __attribute__((ext_vector_type(2)));
template <typename C> __device__ __forceinline__ uint32_t gather_odd(uint32_t seen, uint32_t w)
{
    if constexpr (sizeof(C) == 4)
        return max(seen, w & 0x7fffffffu);
    else if constexpr (sizeof(C) == 1)
        return seen | ((w & 0x7f7f7f7fu) + 0x01010101u);
    else
        return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(h2, seen), __builtin_bit_cast(h2, w & 0x7fff7fffu)));
}
template <typename C> __device__ __forceinline__ bool is_odd(uint32_t seen)
{
    constexpr uint32_t top = __is_same(C, bf16) ? 0x7f80u : 0x7c00u;
    return sizeof(C) == 4 ? seen >= 0x7f800000u : sizeof(C) == 1 ? (seen & 0x80808080u) != 0 : (seen & 0xffffu) >= top || seen >> 16 >= top;
}

// A word of the cache with zeros in the place of such values.
template <typename C> __device__ __forceinline__ uint32_t finite_word(uint32_t w)
{
    if constexpr (sizeof(C) == 4) {
        return is_odd<C>(w & 0x7fffffffu) ? 0u : w;
    } else if constexpr (sizeof(C) == 2) {
        constexpr uint32_t top = __is_same(C, bf16) ? 0x7f80u : 0x7c00u;
        return ((w & top) == top ? 0u : w & 0xffffu) | ((w >> 16 & top) == top ? 0u : w & 0xffff0000u);
    } else {
        uint32_t r = 0;
#pragma unroll
        for (int i = 0; i < 32; i += 8)
            r |= (w >> i & 0x7f) == 0x7f ? 0u : w & 0xffu << i;
        return r;
    }
}

// A barrier for what the workgroup keeps in LDS: loads on their way stay on it.
__device__ __forceinline__ void meet_in_lds()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

template <bool FIRST, typename A, typename B> __device__ __forceinline__ auto &this_one(A &a, B &b)
{
    if constexpr (FIRST)
        return a;
    else
        return b;
}

// The lowest n of four bits.
__device__ __forceinline__ uint32_t low_bits(int n) { return (1u << min(max(n, 0), 4)) - 1; }

// What SHARE waves stage of a step's 32 tokens: keys and values in chunks of 16 bytes,
// kChunks of each thread, in two buffers of LDS, the next step's on their way in
// registers meanwhile.  Straight to registers, as for fewer queries, every wave would
// load all of it, and a load of keys, 16 tokens by 4 chunks, is 64 accesses of the
// compute unit's cache where one of neighbours is 16: 32 rows of 64 drafted tokens
// over 4096 kept it 81% busy and took 377 us, 281 so; 1 x 16 over 131072 128 us, 122
// so.  Keys lie so that the 16 tokens' same chunks are on different banks: a token's
// chunk c in the place of c ^ key(token).
template <typename C, int D, int SHARE> struct Staged {
    static constexpr int kRow = D * sizeof(C), kPerRow = kRow / 16, kTile = 32 * kRow;
    static constexpr int kChunks = SHARE ? kPerRow / SHARE : 1, kIds = kChunks > 1 ? kChunks / 2 : 1;
    static constexpr int kBytes = SHARE ? 2 * (8 / SHARE) * 2 * kTile : 0;  // of a workgroup
    static __device__ __forceinline__ int key(int token) { return kPerRow >= 16 ? token & 15 : token / (kPerRow < 16 ? 16 / kPerRow : 1) & (kPerRow - 1); }
};

template <bool B> struct Clean {
    static constexpr bool value = B;
};

// SHARE: 0, or the units of a workgroup that are one key-value head's and take its
// tokens from LDS together (see Staged).
template <typename C, int QK, int PV, int D, bool TILED, int QT, int MOST, int KEEP, int SHARE>
__global__ __launch_bounds__(tree_heavy(QT, D) ? 256 : 512) void k_tree(TreeArgs)
{
    typedef Attend<C, QK, PV, D, TILED, MOST, KEEP> S;
    constexpr int CS = S::kSize, E = S::kChunk, NC = S::kChunks, UT = S::kTiles, VW = S::kWide, NP = S::kParts, NT = S::kTokens;
    constexpr int COLS = 16 * QT;
    typedef Staged<C, D, SHARE> T;
    extern __shared__ __align__(16) char lds[];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const TreeArgs &p0 = tree_arguments();
    const uint32_t y = divide(blockIdx.x, p0.units);
    // A wave takes one of the workgroup's units, or one of several turns at it.
    const int beside = p0.beside, in = wave & (beside - 1), turn = wave / beside, turns = waves / beside;
    const uint32_t unit = (blockIdx.x - y * p0.units.d) * beside + in;

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
        const TreeArgs &p = tree_arguments();
        const detfold_attend &a = p.a;
        const detfold_paged_cache &c = p.c;
        const int lane = anew((int)threadIdx.x & 63), col = lane & 15, grp = lane >> 4;
        const uint32_t h = divide(unit, p.tiles), tile = unit - h * p.tiles.d;
        const int drafted = min(max(p.counts ? scalar_load(p.counts + b) : p.drafts, 0), p.drafts);
        const int col0 = (int)tile * COLS, live = min(max(drafted * p.group - col0, 0), COLS);
        const char *k0 = (const char *)c.k + (int64_t)h * c.k_head * CS, *v0 = (const char *)c.v + (int64_t)h * c.v_head * CS;
        const int64_t k_page = c.k_page * CS, k_token = c.k_token * CS, v_page = c.v_page * CS, v_token = c.v_token * CS;
        const uint32_t pages = (uint32_t)c.pages;
        const int c_dim = c.dim;
        const float cap = p.cap;
        const bool biased = p.slopes != nullptr, placed = biased || p.window > 0;  // whether positions matter
        // What products become scores by, times log2 e.  The host has looked at the scale
        // and the cap; a key scale that is no number, or takes the factor past binary32,
        // makes its head's scores no numbers.
        const float factor = a.scale * (c.k_scale ? scalar_load(c.k_scale + h) : 1.0f) * kLog2e;
        const float by = __builtin_fabsf(factor) < INFINITY ? factor : __builtin_nanf("");
        // What products become arguments of the tanh by: where that passes binary32 its
        // largest value, with which only products near the smallest are not past 4.
        const float bound = cap * kLog2e, ratio = by / bound;
        const float over = __builtin_fabsf(ratio) == INFINITY ? __builtin_copysignf(0x1.fffffep127f, ratio) : ratio;
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
        const int32_t base = max((int32_t)row.end - drafted, 0);  // tokens of the prefix
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
        const uint32_t steps = end > begin && (SHARE || live > 0) ? (end - a0 + S::kStep - 1) / S::kStep : 0;
        // Tokens below `low` are behind some query's window; a distance of `window` hides.
        const int32_t window = p.window > 0 ? (int32_t)min(p.window, (int64_t)INT32_MAX) : INT32_MAX;
        const int32_t low = p.window > 0 ? (int32_t)max((int64_t)base + (p.depths ? DETFOLD_MAX_DRAFTS : p.drafts) - window, (int64_t)0) : 0;

        // The columns, and the drafted tokens' depths, which all waves share.
        constexpr int kUnitQueries = SHARE ? 0 : QT * S::kQ;
        char *const queries = lds + in * kUnitQueries;
        Column *const columns = (Column *)(lds + T::kBytes + beside * kUnitQueries) + in * COLS;
        int32_t *const depths = (int32_t *)(lds + T::kBytes + beside * (kUnitQueries + COLS * (int)sizeof(Column)));
        auto depth = [&](int j) { return p.depths ? min(max(p.depths[b * p.drafts + j], 0), DETFOLD_MAX_DRAFTS - 1) : j; };
        if (turn == 0 && lane < live) {
            const int i = (int)divide((uint32_t)(col0 + lane), p.heads_of);
            Column x;
            x.mask = p.masks ? (uint64_t)p.masks[b * p.drafts + i] : ~0ull >> (63 - i);
            x.at = base + depth(i);
            x.slope = p.slopes ? p.slopes[h * p.group + (col0 + lane - i * p.group)] * kLog2e : 0.0f;
            columns[lane] = x;
        }
        if (wave == 0)
            depths[lane] = lane < drafted ? depth(lane) : 0;

        // The queries as the operand of the score products, one lane's 16 bytes
        // after the other; a chunk that would pass the head's end starts earlier,
        // and what it repeats counts as zero.
        constexpr int QS = QK == kF32 || QK == kSplit ? 4 : 2, PER = QK == kF32 ? 4 : 8, NQ = D / (4 * PER);
        auto query_chunk = [&](int i) { return E * (4 * (i * PER / E) + grp); };
        Words<PER * QS> qw[QT][NQ] = {};
#pragma unroll
        for (int n = 0; n < QT; ++n) {
            const int x = col0 + min(16 * n + col, max(live - 1, 0)), i = (int)divide((uint32_t)x, p.heads_of);
            const char *q = (const char *)a.q + (b * a.q_row + i * p.q_draft + ((int64_t)h * p.group + (x - i * p.group)) * a.q_head) * QS;
#pragma unroll
            for (int i = 0; i < NQ; ++i)
                if (live > 0 && (SHARE || ((n * NQ + i) & (turns - 1)) == turn))
                    __builtin_memcpy(&qw[n][i], q + (min(query_chunk(i), c.dim - E) + i * PER % E) * QS, PER * QS);
        }

        const int32_t *table = a.table + b * a.table_row;
        // The pages of a step's tokens, looked up two steps ahead of the products.
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
                    kw[u][i] = load_words<16, false>(k + anew(k_at[i]));
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

        // The staged chunks of this thread, of step s: the pages of their tokens, their
        // loads, and their stores to a buffer.
        struct Ids {
            int32_t id[T::kIds];
        };
        auto staged_place = [&]() { return anew(in * 64 + lane); };  // of this thread among those that stage together
        auto staged_token = [&](int place, int k) { return (place + k * 64 * SHARE) / T::kPerRow & 31; };
        auto staged_at = [&](int place, uint32_t s, int k) { return min(a0 + min(s, steps - 1) * 32 + staged_token(place, k), last); };
        auto staged_values = [&](int place, int k) { return T::kChunks > 1 ? k >= T::kChunks / 2 : place >= 32 * T::kPerRow; };
        auto stage_ids = [&](uint32_t s) {
            const int place = staged_place();
            Ids g;
#pragma unroll
            for (int k = 0; k < T::kIds; ++k)
                g.id[k] = table[divide(staged_at(place, s, k), p.page)];
            return g;
        };
        u4 staged[T::kChunks];
        auto stage_load = [&](uint32_t s, const Ids &g) {
            const int place = staged_place();
#pragma unroll
            for (int k = 0; k < T::kChunks; ++k) {
                const uint32_t t = staged_at(place, s, k % T::kIds), off = t - divide(t, p.page) * p.page.d, id = (uint32_t)valid(g.id[k % T::kIds]);
                const int c = (place + k * 64 * SHARE) % T::kPerRow;
                const bool values = staged_values(place, k);
                // Strides below 2^31 bytes, which the plan looks at.
                const char *from = (values ? v0 : k0) + min(16 * c, (values ? p.c.v_dim : c_dim) * CS - 16);
                from += (uint64_t)id * (uint32_t)(values ? v_page : k_page);
                from += (uint64_t)off * (uint32_t)(values ? v_token : k_token);
                const Words<16> w = load_words<16, false>(from);
                staged[k] = u4{w.w[0], w.w[1], w.w[2], w.w[3]};
            }
        };
        auto buffer = [&](uint32_t round) { return lds + ((round & 1) * turns + turn) * (2 * T::kTile); };
        auto stage_store = [&](uint32_t round) {
            const int place = staged_place();
#pragma unroll
            for (int k = 0; k < T::kChunks; ++k) {
                const int c = (place + k * 64 * SHARE) % T::kPerRow, t = staged_token(place, k);
                const bool values = staged_values(place, k);
                if (c_dim < D)  // past the head's end: zeros
                    staged[k] &= !values && 16 * c >= c_dim * CS ? 0u : ~0u;
                *(u4 *)(buffer(round) + (values ? T::kTile : 0) + t * T::kRow + 16 * (values ? c : c ^ T::key(t))) = staged[k];
            }
        };

        // Weights of 16-bit floats are held 2^15 times larger, so that small ones
        // keep their digits; the sum is too, and both are put right at the end.
        constexpr int kLift = PV == kF16 ? 15 : 0;
        float m[QT], l[QT];
        f4 acc[QT][NP][VW];
#pragma unroll
        for (int n = 0; n < QT; ++n) {
            m[n] = -INFINITY, l[n] = 0.0f;
#pragma unroll
            for (int i = 0; i < NP; ++i)
#pragma unroll
                for (int j = 0; j < VW; ++j)
                    acc[n][i][j] = f4{0.0f, 0.0f, 0.0f, 0.0f};
        }

        uint32_t s = turn;
        const uint32_t rounds = SHARE ? (steps + turns - 1) / turns : 0;  // steps of each of the workgroup's waves
        Pages now = {}, next = {};
        Ids ids = {};
        if constexpr (SHARE) {
            if (rounds) {
                ids = stage_ids(s);
                stage_load(s, ids);
                ids = stage_ids(s + turns);
            }
        } else if (s < steps) {
            now = look_up(s);
            load_keys(now);
            load_values(now);
            now = look_up(min(s + turns, steps - 1));
        }
        __builtin_amdgcn_sched_barrier(0);  // the first loads are on their way while the queries arrive
#pragma unroll
        for (int n = 0; n < QT; ++n)
#pragma unroll
            for (int i = 0; i < NQ; ++i)
                if (SHARE || ((n * NQ + i) & (turns - 1)) == turn) {
                    const int drop = query_chunk(i) - min(query_chunk(i), c.dim - E) - i * PER % E;
                    Words<PER * QS> &w = qw[n][i];
#pragma unroll
                    for (int j = 0; j < PER * QS / 4; ++j)
                        if (c_dim < D)
                            w.w[j] &= keep_from(drop * QS, j);
                    char *const to = queries + n * S::kQ + lane * 16;
                    if constexpr (SHARE) {
                    } else if constexpr (QK == kSplit) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)  // a NaN whose bits all lie below the first part's would be an infinity there
                            w.w[j] = __builtin_isnan(__builtin_bit_cast(float, w.w[j])) ? 0x7fc00000u : w.w[j];
#pragma unroll
                        for (int part = 0; part < 3; ++part) {  // the highest bits, of which two values' are stored together
                            u4 x;
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                x[j] = __builtin_amdgcn_perm(w.w[2 * j + 1], w.w[2 * j], 0x07060302u);
                                w.w[2 * j] = below(w.w[2 * j]), w.w[2 * j + 1] = below(w.w[2 * j + 1]);
                            }
                            *(u4 *)(to + (part * NQ + i) * 1024) = x;
                        }
                    } else {
                        *(u4 *)(to + i * 1024) = u4{w.w[0], w.w[1], w.w[2], w.w[3]};
                    }
                }
        if constexpr (SHARE) {
            if (rounds) {
                stage_store(0);
                stage_load(s + turns, ids);
                ids = stage_ids(s + 2 * turns);
            }
        }
        __syncthreads();
        // The queries are held in registers where those have room: 16 beside a step's
        // keys and values (32 are too many), and 32 where these come from LDS.
        constexpr bool kHeld = SHARE || QT * S::kQ <= 16 * 256;
        constexpr int QW = S::kQ / 1024;
        u4 held[kHeld ? QT : 1][kHeld ? QW : 1];
        if constexpr (kHeld)
#pragma unroll
            for (int n = 0; n < QT; ++n)
#pragma unroll
                for (int i = 0; i < QW; ++i) {
                    if constexpr (SHARE)
                        held[n][i] = u4{qw[n][i].w[0], qw[n][i].w[1], qw[n][i].w[2], qw[n][i].w[3]};
                    else
                        held[n][i] = *(const u4 *)(queries + n * S::kQ + i * 1024 + lane * 16);
                }
        auto query = [&](int n, int i, uint32_t at) {
            if constexpr (kHeld)
                return held[n][i];
            else
                return *(const u4 *)(queries + n * S::kQ + i * 1024 + at);
        };
        // Whether some query does not see some token of the step at t0, or sees it at
        // another position than its number.
        auto is_mixed = [&](uint32_t t0) { return (int32_t)(t0 + S::kStep) > base || (int32_t)t0 < low || t0 < begin || t0 + S::kStep > end; };
        bool odd = false;  // whether a mixed step had a value that is infinite or no number
        // One step, which also issues the next one's loads.  Steps of which all queries
        // see all, with another behind them, are compiled for that alone: a branch around
        // the next one's loads would make the wait for the values take the keys issued
        // after them for values not yet there, and what masks go by would fill the
        // scalar registers.
        auto step = [&](auto is_clean) {
            constexpr bool clean = decltype(is_clean)::value;
            const bool more = !SHARE && (clean || s + turns < steps);
            const uint32_t t0 = a0 + s * S::kStep;
            const char *const tile = buffer(s / turns);
            const int here = anew(lane), col = here & 15, grp = here >> 4;
            const uint32_t q_at = here * 16;
            // Staged tokens come to registers here; others are there, held across steps.
            Words<16> keys_here[SHARE ? UT : 1][SHARE ? NC : 1];
            Words<VW * CS> values_here[SHARE ? NT : 1][SHARE ? NP : 1];
            auto &kr = this_one<(SHARE > 0)>(keys_here, kw);
            auto &vr = this_one<(SHARE > 0)>(values_here, vw);
            if constexpr (SHARE) {
                const int at = (grp ^ T::key(col)) * 16;
#pragma unroll
                for (int u = 0; u < UT; ++u)
#pragma unroll
                    for (int i = 0; i < NC; ++i)
                        __builtin_memcpy(&kr[u][i], tile + (16 * u + col) * T::kRow + (at ^ 64 * i), 16);
            }
            // Scores: a row per token, a column per query.
            f4 x[QT][UT];
#pragma unroll
            for (int n = 0; n < QT; ++n)
#pragma unroll
                for (int u = 0; u < UT; ++u)
                    x[n][u] = f4{0.0f, 0.0f, 0.0f, 0.0f};
            // What a lane's loads repeat past the head's end is cleared: there the queries
            // are zero, but zero times an infinite key would be NaN (an e4m3 key is never
            // infinite).
            if (!SHARE && CS != 1 && c_dim < D) {
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    const int at = E * (4 * i + grp), drop = at - min(at, c_dim - E);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t keep = keep_from(CS * drop, j);
#pragma unroll
                        for (int u = 0; u < UT; ++u)
                            kr[u][i].w[j] &= keep;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                if (QK == kF32 && 4 * E * i >= c_dim)  // products that take long and add nothing
                    break;
                if constexpr (QK == kF32) {
#pragma unroll
                    for (int e = 0; e < E; e += 4)
#pragma unroll
                        for (int n = 0; n < QT; ++n) {
                            const f4 q = __builtin_bit_cast(f4, query(n, i * (E / 4) + e / 4, q_at));
#pragma unroll
                            for (int u = 0; u < UT; ++u)
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    x[n][u] = __builtin_amdgcn_mfma_f32_16x16x4f32(value32<C>(kr[u][i].w, e + j), q[j], x[n][u], 0, 0, 0);
                        }
                } else {
#pragma unroll
                    for (int e = 0; e < E; e += 8) {
                        u4 k[UT];
#pragma unroll
                        for (int u = 0; u < UT; ++u)
                            k[u] = u4{pair16<C, QK>(kr[u][i].w, e / 2), pair16<C, QK>(kr[u][i].w, e / 2 + 1),
                                      pair16<C, QK>(kr[u][i].w, e / 2 + 2), pair16<C, QK>(kr[u][i].w, e / 2 + 3)};
#pragma unroll
                        for (int n = 0; n < QT; ++n)
#pragma unroll
                            for (int part = 0; part < (QK == kSplit ? 3 : 1); ++part) {
                                const u4 q = query(n, part * NQ + i * (E / 8) + e / 8, q_at);
#pragma unroll
                                for (int u = 0; u < UT; ++u)
                                    x[n][u] = mfma16<QK>(k[u], q, x[n][u]);
                            }
                    }
                }
            }
            if (more) {
                next = look_up(min(s + 2 * turns, steps - 1));
                load_keys(now);
            }
            auto every = [&](auto f) {
#pragma unroll
                for (int n = 0; n < QT; ++n)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        x[n][j / 4][j % 4] = f(x[n][j / 4][j % 4]);
            };
            if (cap > 0.0f) {
                float most = 0.0f;
                every([&](float z) {
                    most = fmaxf(most, __builtin_fabsf(z));
                    return z;
                });
                if (__any(!(most * __builtin_fabsf(over) < 0.5f)))
                    every([&](float z) {
                        asm("" : "+v"(z));  // what both paths compute does not move before the branch, which would copy all scores
                        return any_cap(z * by, z * over, bound);
                    });
                else
                    every([&](float z) { return near_cap(z * by, z * over); });
            } else {
                every([&](float z) { return z * by; });
            }
            if constexpr (SHARE) {
                __builtin_amdgcn_sched_barrier(0);  // the values take the keys' registers
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int i = 0; i < NP; ++i)
                        __builtin_memcpy(&vr[j][i], tile + T::kTile + (16 * (j / 4) + 4 * grp + j % 4) * T::kRow + VW * (16 * i + col) * CS, VW * CS);
            }
            if (!clean && is_mixed(t0)) {
                // Of the lane's four tokens of each tile, bit by bit: which are this part's.
                // What others hold may be anything.
                const int first = (int)(grp * 4 + t0);  // the lane's first token
                uint32_t ours[UT];
#pragma unroll
                for (int u = 0; u < UT; ++u)
                    ours[u] = low_bits((int)(end - first - 16 * u)) & ~low_bits((int)(begin - first - 16 * u));
                if (t0 < begin || t0 + S::kStep > end) {
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const uint32_t keep = ours[j / 4] & 1u << j % 4 ? ~0u : 0u;
#pragma unroll
                        for (int i = 0; i < NP; ++i)
#pragma unroll
                            for (int n = 0; n < VW * CS / 4; ++n)
                                vr[j][i].w[n] &= keep;
                    }
                }
                // Zero times a value that a query does not see would be NaN where that is
                // infinite or no number: such values count as zero here, and are added
                // to the sums of those that see them at the end.
                uint32_t gathered = 0;
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int i = 0; i < NP; ++i)
#pragma unroll
                        for (int n = 0; n < VW * CS / 4; ++n)
                            gathered = gather_odd<C>(gathered, vr[j][i].w[n]);
                if (__builtin_expect(__any(is_odd<C>(gathered)), 0)) {
                    odd = true;
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int i = 0; i < NP; ++i)
#pragma unroll
                            for (int n = 0; n < VW * CS / 4; ++n)
                                vr[j][i].w[n] = finite_word<C>(vr[j][i].w[n]);
                }
#pragma unroll
                for (int u = 0; u < UT; ++u) {
                    const int rel = first + 16 * u - base;  // of the first token to the first drafted one
                    int32_t pos[4] = {};
                    if (placed) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            pos[j] = rel + j < 0 ? base + rel + j : base + depths[min(rel + j, DETFOLD_MAX_DRAFTS - 1)];
                    }
#pragma unroll
                    for (int n = 0; n < QT; ++n) {
                        const Column w = columns[16 * n + col];
                        uint32_t sees = rel >= 0 ? (uint32_t)(w.mask >> min(rel, 63)) : (uint32_t)(w.mask << min(-rel, 4)) | low_bits(-rel);
                        sees &= ours[u];
                        if (placed) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                sees &= w.at - pos[j] < window ? ~0u : ~(1u << j);
                                if (biased)
                                    x[n][u][j] += w.slope * (float)(pos[j] - w.at);
                            }
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            x[n][u][j] = sees & 1u << j ? x[n][u][j] : -INFINITY;
                    }
                }
            } else if (biased) {
#pragma unroll
                for (int n = 0; n < QT; ++n) {
                    const Column w = columns[16 * n + col];
                    const int32_t at = (int32_t)t0 + 4 * grp - w.at;
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        x[n][j / 4][j % 4] += w.slope * (float)(at + 16 * (j / 4) + j % 4);
                }
            }
            // Weights, relative to the largest score so far.
#pragma unroll
            for (int n = 0; n < QT; ++n) {
                float top = -INFINITY;
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    top = fmaxf(top, x[n][j / 4][j % 4]);
                top = fmaxf(m[n], over_groups(top, [](float y, float z) { return fmaxf(y, z); }));
                const float origin = top == -INFINITY ? 0.0f : top;
                if (__any(top > m[n])) {
                    const float turn = weight2_of(m[n] - origin);
                    l[n] *= turn;
#pragma unroll
                    for (int i = 0; i < NP; ++i)
#pragma unroll
                        for (int j = 0; j < VW; ++j)
                            acc[n][i][j] *= turn;
                    m[n] = top;
                }
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    x[n][j / 4][j % 4] = weight2_of(x[n][j / 4][j % 4] - origin + (float)kLift);
                    l[n] += x[n][j / 4][j % 4];
                }
            }
            // Values: the output's rows are its dims, its columns the queries.
            if constexpr (PV == kF32) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int i = 0; i < NP; ++i)
#pragma unroll
                        for (int e = 0; e < VW; ++e)
#pragma unroll
                            for (int n = 0; n < QT; ++n)
                                acc[n][i][e] = __builtin_amdgcn_mfma_f32_16x16x4f32(value32<C>(vr[j][i].w, e), x[n][j / 4][j % 4], acc[n][i][e], 0, 0, 0);
            } else {
                constexpr int TERMS = PV == kSplit ? 3 : 1;
#pragma unroll
                for (int u = 0; u < UT; u += 2) {
                    u4 w[QT][TERMS];
#pragma unroll
                    for (int n = 0; n < QT; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float y = x[n][u + j / 2][2 * (j % 2)], z = x[n][u + j / 2][2 * (j % 2) + 1];
                            if constexpr (PV == kF16) {
                                w[n][0][j] = __builtin_bit_cast(uint32_t, f16x2{(f16)y, (f16)z});
                            } else {
#pragma unroll
                                for (int e = 0; e < TERMS; ++e) {
                                    const bf16x2 part = {(bf16)y, (bf16)z};
                                    w[n][e][j] = __builtin_bit_cast(uint32_t, part);
                                    y -= (float)part.x, z -= (float)part.y;
                                }
                            }
                        }
#pragma unroll
                    for (int i = 0; i < NP; ++i)
#pragma unroll
                        for (int e = 0; e < VW; e += 2) {
                            u4 lo, hi;  // dims e and e + 1 of the lane's eight tokens
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint32_t y = pair16<C, PV>(vr[4 * u + 2 * j][i].w, e / 2), z = pair16<C, PV>(vr[4 * u + 2 * j + 1][i].w, e / 2);
                                lo[j] = __builtin_amdgcn_perm(z, y, 0x05040100u);
                                hi[j] = __builtin_amdgcn_perm(z, y, 0x07060302u);
                            }
#pragma unroll
                            for (int n = 0; n < QT; ++n)
#pragma unroll
                                for (int q = 0; q < TERMS; ++q) {
                                    acc[n][i][e] = mfma16<PV>(lo, w[n][q], acc[n][i][e]);
                                    acc[n][i][e + 1] = mfma16<PV>(hi, w[n][q], acc[n][i][e + 1]);
                                }
                        }
                }
            }
            if (more) {
                load_values(now);
                now = next;
            }
        };
        if constexpr (SHARE) {
            // A round: this one's tokens are there once all have stored theirs, and the
            // other buffer is free, of which the round before was computed.
            for (uint32_t round = 0; round < rounds; ++round, s += turns) {
                step(Clean<false>{});
                stage_store(round + 1);
                stage_load(s + 2 * turns, ids);  // past the last step: that one again
                ids = stage_ids(s + 3 * turns);
                meet_in_lds();
            }
        } else {
            for (; s < steps; s += turns) {
                for (; s + turns < steps && !is_mixed(a0 + s * S::kStep); s += turns)
                    step(Clean<true>{});
                step(Clean<false>{});
            }
        }

        // The waves' states, joined in order: each leaves its columns' sums in LDS, over
        // the queries, and a thread takes four dims of a column from every turn.
        f2 *const state = (f2 *)lds;
        int *const odds = (int *)(lds + waves * COLS * sizeof(f2));
        float *const sums = (float *)(odds + 4 * waves);
        const bool any_bad = __any(bad);
        __syncthreads();
        if (lane == 0)
            odds[wave] = odd | any_bad << 1;
#pragma unroll
        for (int n = 0; n < QT; ++n) {
            const float lift = PV == kF16 ? 0x1p-15f : 1.0f;
            float total = over_groups(l[n], [](float y, float z) { return y + z; }) * lift;
            if (16 * n + col < live) {
                float *mine = sums + (wave * COLS + 16 * n + col) * S::kRow;
#pragma unroll
                for (int i = 0; i < NP; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int e = 0; e < VW; e += 4)
                            *(f4 *)(mine + VW * (16 * i + 4 * grp + j) + e) =
                                f4{acc[n][i][e][j], acc[n][i][e + 1][j], acc[n][i][e + 2][j], acc[n][i][e + 3][j]} * lift;
                if (grp == 0)
                    state[wave * COLS + 16 * n + col] = f2{m[n], total};
            }
        }
        __syncthreads();
        const TreeArgs &pe = tree_arguments();
#pragma unroll 1
        for (int i = 64 * turn + lane; i < live * (D / 4); i += 64 * turns) {
            const TreeArgs &p = pe;
            const detfold_attend &a = p.a;
            const int head = i / (D / 4), at = i % (D / 4) * 4, at0 = at / VW * VW;
            if (at0 >= p.c.v_dim)
                continue;
            float top = -INFINITY;
            for (int w = in; w < waves; w += beside)
                top = fmaxf(top, state[w * COLS + head].x);
            const float origin = top == -INFINITY ? 0.0f : top;
            f4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
            float weights = 0.0f;
            int unfinished = 0;
            for (int w = in; w < waves; w += beside) {
                const f2 ml = state[w * COLS + head];
                const float by = weight2_of(ml.x - origin);
                weights += ml.y * by;
                sum += *(const f4 *)(sums + (w * COLS + head) * S::kRow + at) * by;
                unfinished |= odds[w];
            }
            if constexpr (SHARE)  // every wave looked up some of the pages
                for (int w = 0; w < waves; ++w)
                    unfinished |= odds[w] & 2;
            if (unfinished & 2)
                weights = __builtin_nanf("");
            const int d = min(at0, p.c.v_dim - VW) + at - at0, x = col0 + head, q = (int)divide((uint32_t)x, p.heads_of);
            if (unfinished & 1) {  // the values that the mixed steps left out
                const uint64_t mask = p.masks ? (uint64_t)p.masks[b * p.drafts + q] : ~0ull >> (63 - q);
                const int32_t own = base + depth(q);
#pragma unroll 1
                for (uint32_t t = begin; t < end; ++t) {
                    const uint32_t s = (t - a0) / S::kStep;
                    if (!is_mixed(a0 + s * S::kStep)) {
                        t = a0 + (s + 1) * S::kStep - 1;
                        continue;
                    }
                    const int rel = (int)t - base;
                    const uint32_t pg = divide(t, p.page), id = (uint32_t)table[pg];
                    if (id >= pages || (rel >= 0 && !(mask >> min(rel, 63) & 1)) || own - (rel < 0 ? (int)t : base + depth(rel)) >= window)
                        continue;
                    const C *v = (const C *)(v0 + id * v_page + (t - pg * p.page.d) * v_token) + d;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float z = to_f32(v[e]);
                        sum[e] += __builtin_fabsf(z) < INFINITY ? 0.0f : z;
                    }
                }
            }
            if (slot >= 0) {
                const int64_t from = slot * p.slot_cols + head;
                __builtin_memcpy(p.acc + from * p.c.v_dim + d, &sum, sizeof(sum));
                if (at == 0)
                    p.ml[from] = make_float2(top, weights);
            } else {
                const int g = (int)h * p.group + x - q * p.group;
                const float by = out_scale(v_scale, weights);
                const float o[4] = {sum.x * by, sum.y * by, sum.z * by, sum.w * by};
                put_out<4>(a, b * a.out_row + q * p.out_draft + (int64_t)g * a.out_head + d, o);
                if (a.lse && at == 0)
                    a.lse[(b * p.drafts + q) * a.q_heads + g] = log_sum2(top, weights);
            }
        }
        mine.left -= done;
        if (mine.left == 0)
            return;
        mine.at = mine.row_at = mine.at + done;
        ++b;
        mine.len = scalar_load(tree_arguments().a.lens + b);
        __syncthreads();
    }
}

// The kernel of a call and the LDS it takes: for a unit's queries and columns, and
// for the sums of a wave's tile.  Keys stay in the caches, also where attend_keep would
// rather have nothing kept: trees have no instance for that.
template <typename C, int QK, int PV, int D, int QT, int MOST, int KEEP> TreeKernel pick_tree_tiled(const TreeArgs &a)
{
    typedef Attend<C, QK, PV, D, true, MOST, KEEP> S;
    const void *f = a.tiled ? (const void *)k_tree<C, QK, PV, D, true, QT, MOST, KEEP, 0> : (const void *)k_tree<C, QK, PV, D, false, QT, MOST, KEEP, 0>;
    return {f, 0, QT * (S::kQ + 16 * (int)sizeof(Column)), 16 * QT * (8 + S::kRow * 4) + 16};
}
template <typename C, int QK, int PV, int D, int SHARE> TreeKernel pick_tree_shared()
{
    typedef Attend<C, QK, PV, D, false, 2, kAll> S;
    return {(const void *)k_tree<C, QK, PV, D, false, 2, 2, kAll, SHARE>, Staged<C, D, SHARE>::kBytes, 2 * 16 * (int)sizeof(Column), 32 * (8 + S::kRow * 4) + 16};
}
template <typename C, int QK, int PV, int D> TreeKernel pick_tree_columns(const TreeArgs &a)
{
    if constexpr (QK != kF32 && QK != kSplit && PV != kF32 && PV != kSplit) {
        if constexpr (D < 256) {
            if (a.shared == 2)
                return pick_tree_shared<C, QK, PV, D, 2>();
            if (a.shared == 4)
                return pick_tree_shared<C, QK, PV, D, 4>();
            if constexpr (D * sizeof(C) / 16 >= 8)
                if (a.shared == 8)
                    return pick_tree_shared<C, QK, PV, D, 8>();
        }
        if (a.tiles_of == 2)
            return a.keep == kAll ? pick_tree_tiled<C, QK, PV, D, 2, 2, kAll>(a) : pick_tree_tiled<C, QK, PV, D, 2, 2, kKeys>(a);
    }
    // A step of one tile is 16 KiB, or 32 of heads above 128.
    constexpr int MOST = D * sizeof(C) <= 128 ? 4 : 2;
    if constexpr (MOST > 2)
        if (a.brief)
            return pick_tree_tiled<C, QK, PV, D, 1, 2, kAll>(a);
    return a.keep == kAll ? pick_tree_tiled<C, QK, PV, D, 1, MOST, kAll>(a) : pick_tree_tiled<C, QK, PV, D, 1, MOST, kKeys>(a);
}
template <typename C, int QK, int PV> TreeKernel pick_tree(const TreeArgs &a)
{
    const int dim = a.c.dim > a.c.v_dim ? a.c.dim : a.c.v_dim;
    return dim <= 64 ? pick_tree_columns<C, QK, PV, 64>(a) : dim <= 128 ? pick_tree_columns<C, QK, PV, 128>(a) : pick_tree_columns<C, QK, PV, 256>(a);
}

}  // namespace detfold_impl

#endif  // DETFOLD_TREE_KERNEL_H
