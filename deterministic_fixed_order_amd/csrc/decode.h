// decode.h -- declarations shared by the decode-step operators: decode.cpp
// (host-only checks and planning, and their C ABI), cache_kernels.hip (the
// append and the softmax fold) and attend_kernels.hip (the paged attention).
// Not installed; the public interface is include/detfold.h.
#ifndef DETFOLD_DECODE_H
#define DETFOLD_DECODE_H

#include <hip/hip_vector_types.h>

#include <cstdint>

#include "detfold.h"

namespace detfold_impl {

constexpr int elem_size(int type)
{
    return type == DETFOLD_F32 ? 4 : type == DETFOLD_E4M3 ? 1 : 2;
}

constexpr float kE4m3Max = 448.0f;
constexpr int64_t kMaxBlocks = (int64_t)1 << 22;  // workgroups of a launch: a grid holds at most 2^32 threads

// x / d for 0 <= x < 2^31 and 1 <= d < 2^31 as a multiply and a shift: with
// s = ceil(log2 d) and m = ceil(2^(31+s) / d) (below 2^32), x * m >> (31 + s)
// is exact, since m * d exceeds 2^(31+s) by less than d <= 2^s.
struct Divider {
    uint32_t magic, shift, d;
};

inline Divider divider(uint32_t d)
{
    uint32_t s = 0;
    while (((uint64_t)1 << s) < d)
        ++s;
    const uint64_t m = (((uint64_t)1 << (31 + s)) + d - 1) / d;
    return {(uint32_t)m, 31 + s, d};
}

// Kernel arguments of the append: the two public structs, and what the host
// derives from them.
struct AppendArgs {
    detfold_paged_cache c;
    detfold_append a;
    Divider page;
    // Of the launch: chunks of a key or query head and of a value head, groups
    // of heads of a token (the queries' first) and of its values, the tokens,
    // and the workgroups that turn (the others copy values).
    Divider chunks, v_chunks, groups, v_groups;
    int64_t token0;
    uint32_t tokens, turn;
    int32_t q_groups;
    int32_t width;  // values of an access
};

struct AttendArgs {
    detfold_paged_cache c;
    detfold_attend a;
    Divider page;
    Divider units;  // workgroups per row and part: the units (key-value heads times
                    // tiles of 16 query heads) over those that lie beside each other in one
    Divider tiles;  // of a key-value head's query heads
    Divider parts;  // of every row's length, split tokens each, or
    Divider shares; // even shares of all rows' tokens (0: parts)
    int32_t brief;  // steps of 32 tokens at most
    int32_t keep;   // what the caches keep of the keys and values
    int32_t group;  // query heads of a key-value head
    int64_t split;
    int64_t row0;   // first row of the launch
    int32_t tiled;  // 16 tokens from a multiple of 16 on lie in one page
    int32_t waves;  // of a workgroup
    int32_t beside; // units of a workgroup, a power of two
    // What the parts of a row leave, in slots of min(16, group) query heads:
    // slot (row * parts + part) * units + unit, or slots (share * units + unit)
    // * 2 + 0 and 1 for the row that a share begins within and the one that it
    // ends within.
    float *acc;     // sums [slot][head][v_dim]
    float2 *ml;     // maxima and sums of weights [slot][head]
    // Of each row, or where there are more rows than shares, of each share: the
    // row that begins in it (-1: it also ends there), the first and the last
    // share of that row.
    int3 *cut;
    int32_t by_row;
};

enum Keep { kAll, kKeys, kNothing };
constexpr int kUnit = 64;  // tokens that shares are counted in

// A kernel of the attention and the LDS it takes: for the queries, and for the
// sums of a wave's query head.
struct AttendKernel {
    const void *f;
    int q_bytes, head_bytes;
};
AttendKernel attend_bf16(const AttendArgs &a);
AttendKernel attend_f16(const AttendArgs &a);
AttendKernel attend_f32(const AttendArgs &a);

struct SoftmaxArgs {
    void *out;
    const void *outs;
    const float *lses;
    float *lse;
    int64_t rows, dim, outs_pitch, lses_pitch;
    int32_t type, w;
    Divider chunks;  // of the launch: a row's, its first row and their count
    int64_t row0;
    uint32_t count;
};

// --- decode.cpp: host only, no device access ---------------------------------
bool types_pair(int32_t type, int32_t cache_type);
int check_cache(const detfold_paged_cache *c);
int check_append(const detfold_paged_cache *c, const detfold_append *a);
int access_width(int type, bool overlap, int64_t a, int64_t b, int64_t c);
int append_width(const detfold_paged_cache &c, const detfold_append &a);
int check_attend(const detfold_paged_cache *c, const detfold_attend *a);
int check_softmax(const SoftmaxArgs &s);
struct AttendPlan : detfold_attend_plan {
    int64_t shares, slots;
    int32_t waves, beside;
    bool brief;
};
int plan_attend(const detfold_paged_cache &c, int64_t batch, int32_t q_heads, int64_t max_len,
                int64_t window, int32_t split, bool wide, int32_t cu_count, AttendPlan *p);
bool attend_tiled(const detfold_paged_cache &c);
int attend_keep(const detfold_paged_cache &c, int tiles, bool brief);

// --- cache_kernels.hip, attend_kernels.hip: launches --------------------------
int launch_append(const AppendArgs &a, void *stream);
int launch_softmax(const SoftmaxArgs &s, void *stream);
int launch_attend(const AttendArgs &a, void *stream);

}  // namespace detfold_impl

#endif  // DETFOLD_DECODE_H
