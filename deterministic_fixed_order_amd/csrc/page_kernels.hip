// page_kernels.hip -- copies of whole pages of a paged cache, and the compaction
// of rows' kept tokens, for gfx950.

#include <hip/hip_runtime.h>

#include "decode_device.h"
#include "draft.h"

namespace detfold_impl {
namespace {

constexpr int kBlock = 256;
constexpr int64_t kMaxItems = (int64_t)1 << 30;  // chunks of a launch
constexpr int64_t kMaxBlocks = (int64_t)1 << 22; // workgroups of a launch

// 16 bytes at any alignment, as one wide load or store.
typedef uint32_t u4 __attribute__((ext_vector_type(4), aligned(1)));

// The copy.  A thread takes U chunks of 16 bytes, their loads in flight together.
// The last chunk of a run starts early enough to end with it, so runs of any
// length from 16 bytes on take wide accesses; what two chunks share is written
// twice, with the same bytes.
template <int U> __global__ __launch_bounds__(kBlock) void k_copy_pages(CopyArgs p)
{
    const bool values = blockIdx.x >= p.key_blocks;
    const CopyRuns &r = values ? p.v : p.k;
    const uint32_t x0 = (blockIdx.x - (values ? p.key_blocks : 0)) * (kBlock * U) + threadIdx.x;
    u4 data[U];
    char *to[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
        const uint32_t x = x0 + j * kBlock, i = divide(x, r.page);
        to[j] = nullptr;
        if (i >= p.count)
            continue;
        const int32_t s = p.src[p.first + i], d = p.dst[p.first + i];
        const uint32_t in = x - i * r.page.d, y = divide(in, r.chunks), u = in - y * r.chunks.d;
        const uint32_t token = divide(y, r.heads), head = y - token * r.heads.d;
        if (s < 0 || s >= p.pages || d < 0 || d >= p.into_pages || (p.tokens && (int32_t)token >= p.tokens[p.first + i]))
            continue;
        const int32_t at = min((int32_t)(16 * u), r.run - 16);
        to[j] = r.to + d * r.to_page + token * r.to_token + head * r.to_head + at;
        data[j] = *(const u4 *)(r.from + s * r.from_page + token * r.from_token + head * r.from_head + at);
    }
#pragma unroll
    for (int j = 0; j < U; ++j)
        if (to[j])
            *(u4 *)to[j] = data[j];
}

// The compaction.  A workgroup takes one head's keys or values of one row, and of
// these as many tokens at a time as its threads hold, U chunks each.  In place a
// move goes to a lower token: what is read with a tile of moves lies behind all
// that earlier tiles wrote, and what it writes before all that later tiles read,
// so that the one barrier between a tile's loads and its stores is enough.
template <int U> __global__ __launch_bounds__(kBlock) void k_compact(CompactArgs p)
{
    const detfold_paged_cache &c = p.c;
    const detfold_compact &a = p.a;
    const uint32_t y = divide(blockIdx.x >> 1, p.heads), head = (blockIdx.x >> 1) - y * p.heads.d;
    const bool values = blockIdx.x & 1;
    const int64_t b = p.row0 + y;
    const int size = elem_size(c.type);
    const Divider &per = values ? p.v_chunks : p.k_chunks;
    const int run = (values ? c.v_dim : c.dim) * size;
    char *const pool = (char *)(values ? c.v : c.k) + head * (values ? c.v_head : c.k_head) * size;
    const int64_t page_bytes = (values ? c.v_page : c.k_page) * size, token_bytes = (values ? c.v_token : c.k_token) * size;
    const int32_t *table = a.table + b * a.table_row, *to = a.to ? a.to + b * a.to_row : table;
    const int64_t width = a.table_width, to_width = a.to ? a.to_width : width;
    const int64_t start = a.starts ? a.starts[b] : 0;
    const int64_t n = min((int64_t)a.counts[b], a.most);
    const uint32_t t = divide(threadIdx.x, per), u = threadIdx.x - t * per.d, beside = kBlock / per.d;
    const int at = min((int)(16 * u), run - 16);

    // Where token x of the row lies, or nothing.
    auto place = [&](const int32_t *pages, int64_t wide, int64_t x) -> char * {
        if (x < 0 || x > INT32_MAX)
            return nullptr;
        const uint32_t pg = divide((uint32_t)x, p.page);
        if (pg >= wide)
            return nullptr;
        const int32_t id = pages[pg];
        return id < 0 || id >= c.pages ? nullptr : pool + id * page_bytes + (x - (int64_t)pg * c.page) * token_bytes + at;
    };
    for (int64_t i0 = 0; i0 < n; i0 += beside * U) {
        u4 data[U];
        char *put[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int64_t i = i0 + j * beside + t;
            put[j] = nullptr;
            if (t >= beside || i >= n)
                continue;
            const int64_t pick = a.picks[b * a.most + i];
            if (a.to ? pick < 0 : pick <= i)
                continue;
            const char *from = place(table, width, start + pick);
            char *x = place(to, to_width, start + i);
            if (from && x) {
                put[j] = x;
                data[j] = *(const u4 *)from;
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (put[j])
                *(u4 *)put[j] = data[j];
    }
}

bool launch(const void *k, int64_t blocks, void *args, void *stream)
{
    void *list[] = {args};
    return hipLaunchKernel(k, dim3((unsigned)blocks), dim3(kBlock), list, 0, static_cast<hipStream_t>(stream)) == hipSuccess;
}

}  // namespace

int launch_copy_pages(const CopyArgs &a, int64_t count, void *stream)
{
    constexpr int U = 4;
    CopyArgs p = a;
    const int64_t most = a.k.page.d > a.v.page.d ? a.k.page.d : a.v.page.d, some = kMaxItems / most;
    for (p.first = 0; p.first < count; p.first += some) {
        p.count = (uint32_t)(count - p.first < some ? count - p.first : some);
        auto blocks = [&](const CopyRuns &r) { return ((int64_t)p.count * r.page.d + kBlock * U - 1) / (kBlock * U); };
        p.key_blocks = (uint32_t)blocks(p.k);
        if (!launch((const void *)k_copy_pages<U>, p.key_blocks + blocks(p.v), &p, stream))
            return DETFOLD_ELAUNCH;
    }
    return DETFOLD_OK;
}

int launch_compact(const CompactArgs &a, void *stream)
{
    CompactArgs p = a;
    const int64_t each = 2 * (int64_t)a.c.heads, some = kMaxBlocks / each;
    for (p.row0 = 0; p.row0 < a.a.batch; p.row0 += some) {
        const int64_t rows = a.a.batch - p.row0 < some ? a.a.batch - p.row0 : some;
        if (!launch((const void *)k_compact<4>, rows * each, &p, stream))
            return DETFOLD_ELAUNCH;
    }
    return DETFOLD_OK;
}

}  // namespace detfold_impl
