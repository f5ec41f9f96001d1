// page_kernels.hip -- copies of whole pages of a paged cache, and the compaction
// of rows' kept tokens, for gfx950.

#include <hip/hip_runtime.h>

#include "decode_device.h"
#include "draft.h"

namespace detfold_impl {
namespace {

constexpr int kBlock = 256;
constexpr int64_t kOnceBytes = 8 << 20;  // that are not kept in the caches

// 16 bytes at any alignment, as one wide load or store; once: not kept in the caches.
typedef uint32_t u4 __attribute__((ext_vector_type(4), aligned(1)));
template <bool ONCE> __device__ __forceinline__ u4 load16(const char *p) { return ONCE ? __builtin_nontemporal_load((const u4 *)p) : *(const u4 *)p; }
template <bool ONCE> __device__ __forceinline__ void store16(char *p, u4 x)
{
    if (ONCE)
        __builtin_nontemporal_store(x, (u4 *)p);
    else
        *(u4 *)p = x;
}

// What a copy, or a compaction into other pages, moves: token by token, each token a
// number of runs of bytes, in the keys and in the values alike.  A wave takes `group`
// tokens: each lane looks one of them up, so that the lists' and the tables' latencies
// are paid once for all of them, and then the lanes take the tokens' chunks of 16
// bytes side by side, kDeep loads in flight each.  The last chunk of a run starts
// early enough to end with it, so runs of any length from 16 bytes on take wide
// accesses; what two chunks share is written twice, with the same bytes.
//
// Bytes bound it, as many written as read.  2048 pages of 64 tokens of 8 heads of 128
// bfloat16 (0.95 GB): 169 us, 5.6 TB/s, where torch copies whole tensors at 5.3; 2048
// of 8192 tokens of 32 rows (0.54 GB): 111 us, 4.8 TB/s, reads of 2 KiB here and
// there.  With a chunk's lists looked up by its own thread 196 and 280 us; with loads
// and stores through the caches 5 to 10% more; one to eight loads in flight 171, 171,
// 169 and 174 us.
constexpr int kDeep = 4;
template <bool ONCE, typename Look>
__device__ __forceinline__ void move_tokens(const Look &look, const TokenRuns &r, int64_t head_from, int64_t head_to, int64_t first, int64_t tokens)
{
    const int lane = threadIdx.x & 63;
    const char *from = nullptr;
    char *to = nullptr;
    if (lane < tokens)
        look(first + lane, from, to);
    if (!from)
        to = nullptr;
    const uint32_t items = (uint32_t)tokens * r.token.d;
    for (uint32_t x0 = lane; x0 - lane < items; x0 += 64 * kDeep) {
        u4 data[kDeep];
        char *put[kDeep];
#pragma unroll
        for (int j = 0; j < kDeep; ++j) {
            const uint32_t x = x0 + 64 * j, k = min(divide(x, r.token), 63u), in = x - k * r.token.d, head = divide(in, r.chunks), u = in - head * r.chunks.d;
            const int64_t at = min((int32_t)(16 * u), r.run - 16);
            const char *get = (const char *)from_lane((int64_t)from, k) + head * head_from + at;
            put[j] = (char *)from_lane((int64_t)to, k);
            if (x >= items)
                put[j] = nullptr;
            if (put[j]) {
                put[j] += head * head_to + at;
                data[j] = load16<ONCE>(get);
            }
        }
#pragma unroll
        for (int j = 0; j < kDeep; ++j)
            if (put[j])
                store16<ONCE>(put[j], data[j]);
    }
}

// Which tokens a wave of a launch takes: the keys' first, then the values'.
struct Portion {
    bool values;
    int64_t first, tokens;
};
__device__ __forceinline__ Portion portion(const MoveArgs &m)
{
    const uint32_t wave = __builtin_amdgcn_readfirstlane(blockIdx.x * (kBlock / 64) + (threadIdx.x >> 6));
    const bool values = wave >= m.waves;
    const int64_t first = (int64_t)(wave - (values ? m.waves : 0)) * m.group;
    return {values, first, max(min((int64_t)m.group, m.tokens - first), (int64_t)0)};
}

template <bool ONCE> __global__ __launch_bounds__(kBlock) void k_copy_pages(CopyArgs p)
{
    const Portion w = portion(p.m);
    const TokenRuns &r = w.values ? p.m.v : p.m.k;
    const CopySide &side = w.values ? p.v : p.k;
    auto look = [&](int64_t x, const char *&from, char *&to) {
        const uint32_t i = divide((uint32_t)x, p.page), token = (uint32_t)x - i * p.page.d;
        const int32_t s = p.src[p.first + i], d = p.dst[p.first + i];
        if (s < 0 || s >= p.pages || d < 0 || d >= p.into_pages || (p.tokens && (int32_t)token >= p.tokens[p.first + i]))
            return;
        from = side.from + s * side.from_page + token * side.from_token;
        to = side.to + d * side.to_page + token * side.to_token;
    };
    move_tokens<ONCE>(look, r, side.from_head, side.to_head, w.first, w.tokens);
}

// A row's tokens as the compaction reads and writes them: where token x of the row
// lies, or nothing.
struct Places {
    char *pool;
    int64_t page_bytes, token_bytes;
    int32_t pages;
    Divider page;
    __device__ __forceinline__ char *of(const int32_t *table, int64_t wide, int64_t x) const
    {
        if (x < 0 || x > INT32_MAX)
            return nullptr;
        const uint32_t pg = divide((uint32_t)x, page);
        if (pg >= wide)
            return nullptr;
        const int32_t id = table[pg];
        return id < 0 || id >= pages ? nullptr : pool + id * page_bytes + (x - (int64_t)pg * page.d) * token_bytes;
    }
};

template <bool ONCE> __global__ __launch_bounds__(kBlock) void k_gather(CompactArgs p)
{
    const detfold_compact &a = p.a;
    const Portion w = portion(p.m);
    const CompactSide &side = w.values ? p.v : p.k;
    const Places at = {side.pool, side.page_bytes, side.token_bytes, (int32_t)p.pages, p.page};
    auto look = [&](int64_t x, const char *&from, char *&to) {
        const uint32_t row = divide((uint32_t)x, p.most);
        const int64_t b = p.row0 + row, i = (uint32_t)x - row * p.most.d;
        if (i >= a.counts[b])
            return;
        const int32_t pick = a.picks[b * a.most + i];
        if (pick < 0)
            return;
        const int64_t start = a.starts ? a.starts[b] : 0;
        to = at.of(a.to + b * a.to_row, a.to_width, start + i);
        from = to ? at.of(a.table + b * a.table_row, a.table_width, start + pick) : nullptr;
    };
    move_tokens<ONCE>(look, w.values ? p.m.v : p.m.k, side.head_bytes, side.head_bytes, w.first, w.tokens);
}

// The compaction in place.  A workgroup takes one run, a head's keys or values, of one
// row, and of its tokens as many at a time as its threads hold, kTurns chunks each.  Nothing
// orders workgroups, so no two runs share memory (runs_in_place).  A move
// goes to a lower token: what is read with a tile of moves lies behind all that
// earlier tiles wrote, and what it writes before all that later tiles read.  So the
// one barrier between a tile's loads and its stores is enough, and the next tile's
// loads go out before this one's stores.
constexpr int kTurns = 4;
__global__ __launch_bounds__(kBlock) void k_compact(CompactArgs p)
{
    const detfold_compact &a = p.a;
    const uint32_t y = divide(blockIdx.x, p.runs), run = blockIdx.x - y * p.runs.d;
    const bool values = run >= (uint32_t)p.k_runs;
    const uint32_t head = run - (values ? p.k_runs : 0);
    const CompactSide &r = values ? p.v : p.k;
    const int64_t b = p.row0 + y;
    const int32_t *table = a.table + b * a.table_row;
    const int64_t start = a.starts ? a.starts[b] : 0, n = min((int64_t)a.counts[b], a.most);
    const uint32_t t = divide(threadIdx.x, r.chunks), u = threadIdx.x - t * r.chunks.d, beside = kBlock / r.chunks.d;
    const int at = min((int)(16 * u), r.run - 16);
    const Places places = {r.pool + head * r.head_bytes + at, r.page_bytes, r.token_bytes, (int32_t)p.pages, p.page};

    struct Tile {
        u4 data[kTurns];
        char *put[kTurns];
    };
    auto load = [&](int64_t i0) {
        Tile x;
#pragma unroll
        for (int j = 0; j < kTurns; ++j) {
            const int64_t i = i0 + j * beside + t;
            x.put[j] = nullptr;
            x.data[j] = u4{};
            if (t >= beside || i >= n)
                continue;
            const int32_t pick = a.picks[b * a.most + i];
            if (pick <= i)  // it stays, or is left out
                continue;
            const char *from = places.of(table, a.table_width, start + pick);
            char *to = places.of(table, a.table_width, start + i);
            if (from && to) {
                x.put[j] = to;
                x.data[j] = *(const u4 *)from;
            }
        }
        return x;
    };
    if (n <= 0)
        return;
    Tile now = load(0);
    for (int64_t i0 = 0; i0 < n; i0 += beside * kTurns) {
        Tile next = load(i0 + beside * kTurns);
#pragma unroll
        for (int j = 0; j < kTurns; ++j)  // what this tile read is there before any of it is written over
            asm volatile("" : "+v"(now.data[j]));
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kTurns; ++j)
            if (now.put[j])
                *(u4 *)now.put[j] = now.data[j];
        now = next;
    }
}

bool launch(const void *k, int64_t blocks, void *args, void *stream)
{
    void *list[] = {args};
    return hipLaunchKernel(k, dim3((unsigned)blocks), dim3(kBlock), list, 0, static_cast<hipStream_t>(stream)) == hipSuccess;
}

// How a launch's tokens are dealt out: a wave takes up to 64, but no more than leave
// waves four times over what the device holds at once, nor than 2048 chunks (110.7 us
// for the 2048 of 8192 tokens, 112.3 with waves once over).
MoveArgs deal(MoveArgs m, int64_t tokens)
{
    constexpr int64_t kWaves = 256 * 64;
    const int64_t each = m.k.token.d > m.v.token.d ? m.k.token.d : m.v.token.d;
    m.tokens = tokens;
    m.group = 64;
    while (m.group > 1 && (tokens * 2 < kWaves * m.group || each * m.group > 2048))
        m.group /= 2;
    const int64_t waves = (tokens + m.group - 1) / m.group, block = kBlock / 64;
    m.waves = (uint32_t)((waves + block - 1) / block * block);
    return m;
}

}  // namespace

int launch_copy_pages(const CopyArgs &a, int64_t count, void *stream)
{
    CopyArgs p = a;
    const int64_t some = kMaxMoved / a.page.d;  // pages of a launch
    const bool once = count * a.page.d * (int64_t)(a.m.k.token.d + a.m.v.token.d) * 16 >= kOnceBytes;
    for (p.first = 0; p.first < count; p.first += some) {
        p.m = deal(a.m, (count - p.first < some ? count - p.first : some) * a.page.d);
        if (!launch(once ? (const void *)k_copy_pages<true> : (const void *)k_copy_pages<false>, 2 * (int64_t)p.m.waves / (kBlock / 64), &p, stream))
            return DETFOLD_ELAUNCH;
    }
    return DETFOLD_OK;
}

int launch_compact(const CompactArgs &a, void *stream)
{
    CompactArgs p = a;
    if (!a.a.to) {
        const int64_t each = a.runs.d, some = kMaxBlocks / each;
        for (p.row0 = 0; p.row0 < a.a.batch; p.row0 += some)
            if (!launch((const void *)k_compact, (a.a.batch - p.row0 < some ? a.a.batch - p.row0 : some) * each, &p, stream))
                return DETFOLD_ELAUNCH;
        return DETFOLD_OK;
    }
    const int64_t some = a.a.most < kMaxMoved ? kMaxMoved / a.a.most : 1;  // rows of a launch
    const bool once = a.a.batch * a.a.most * (int64_t)(a.m.k.token.d + a.m.v.token.d) * 16 >= kOnceBytes;
    for (p.row0 = 0; p.row0 < a.a.batch; p.row0 += some) {
        p.m = deal(a.m, (a.a.batch - p.row0 < some ? a.a.batch - p.row0 : some) * a.a.most);
        if (!launch(once ? (const void *)k_gather<true> : (const void *)k_gather<false>, 2 * (int64_t)p.m.waves / (kBlock / 64), &p, stream))
            return DETFOLD_ELAUNCH;
    }
    return DETFOLD_OK;
}

}  // namespace detfold_impl
