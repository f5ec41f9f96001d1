// draft.h -- declarations shared by the drafted step's operators: draft.cpp
// (host-only checks and planning, and their C ABI), tree_kernels.hip with the
// tree_*.hip instances of tree_kernel.h (the attention of drafted tokens) and
// page_kernels.hip (copies and compaction of the cache).
#ifndef DETFOLD_DRAFT_H
#define DETFOLD_DRAFT_H

#include "decode.h"

namespace detfold_impl {

constexpr int64_t kMaxMoved = (int64_t)1 << 22;  // tokens of a page, or of a row, that one launch moves

// Kernel arguments of the attention of drafted tokens.  The base's window is
// widened by the drafted tokens, so that a row's first seen token is one that
// any of its queries may see; `window` is the caller's.
struct TreeArgs : AttendArgs {
    const int64_t *masks;
    const int32_t *counts, *depths;
    const float *slopes;
    int64_t q_draft, out_draft, window;
    float cap;
    int32_t drafts;
    int32_t tiles_of;    // tiles of 16 queries of a unit
    int32_t shared;      // units of a key-value head that take its tokens from LDS together, or 0
    int32_t slot_cols;   // queries of a slot, see AttendArgs
    Divider heads_of;    // query heads of a key-value head
    Divider join_blocks; // workgroups of the join for a row's queries
};

// Whether the sums and a step of so many tiles of queries and of heads of so many
// dims leave a compute unit's registers four waves, not eight.
constexpr bool tree_heavy(int tiles, int head) { return tiles * head > 256 || head > 128; }

// A kernel of the attention of drafted tokens and the LDS it takes: for staged tokens
// and a unit's queries, and for a wave's sums.
struct TreeKernel {
    const void *f;
    int staged_bytes, unit_bytes, wave_bytes;
};
TreeKernel tree_bf16(const TreeArgs &a);
TreeKernel tree_f16(const TreeArgs &a);
TreeKernel tree_f32(const TreeArgs &a);

struct TreePlan : detfold_attend_plan {
    int64_t shares, slots;
    int32_t waves, beside, tiles_of, slot_cols, shared;
    bool brief;
};

// What a token's keys, or values, are in bytes: runs, taken in chunks of 16.
struct TokenRuns {
    int32_t run;            // bytes
    Divider chunks, token;  // chunks of a run, and of a token
};
// Of a launch that moves tokens: what a wave takes, and the keys' waves.
struct MoveArgs {
    TokenRuns k, v;
    int64_t tokens;
    int32_t group;
    uint32_t waves;
};

// Kernel arguments of the page copy; strides in bytes.
struct CopySide {
    const char *from;
    char *to;
    int64_t from_page, from_token, from_head, to_page, to_token, to_head;
};
struct CopyArgs {
    MoveArgs m;
    CopySide k, v;
    const int32_t *src, *dst, *tokens;
    int64_t pages, into_pages;
    int64_t first;  // copy of the launch
    Divider page;
};

// Kernel arguments of the compaction; strides in bytes.
struct CompactSide {
    char *pool;
    int64_t page_bytes, token_bytes, head_bytes;
    int32_t run;     // of a head
    Divider chunks;
};
struct CompactArgs {
    MoveArgs m;
    detfold_compact a;
    CompactSide k, v;
    int64_t pages;
    Divider page, most;
    Divider runs;     // of a token, in place: its keys', k_runs of them, then its values'
    int32_t k_runs;
    int64_t row0;
};

// --- draft.cpp: host only, no device access ----------------------------------
int plan_tree(const detfold_paged_cache &c, int64_t batch, int32_t drafts, int32_t q_heads, int64_t max_len, int64_t window, int32_t split,
              int32_t type, int32_t out_type, int32_t cu_count, TreePlan *p);
int check_tree(const detfold_paged_cache *c, const detfold_tree *t);
int check_copy(const detfold_paged_cache *c, const detfold_paged_cache *into, const int32_t *src, const int32_t *dst,
               const int32_t *tokens, int64_t count);
int check_compact(const detfold_paged_cache *c, const detfold_compact *a);
int runs_in_place(const detfold_paged_cache &c, int32_t *keys, int32_t *values);

// --- tree_kernels.hip, page_kernels.hip: launches -----------------------------
int launch_tree(const TreeArgs &a, void *stream);
int launch_copy_pages(const CopyArgs &a, int64_t count, void *stream);
int launch_compact(const CompactArgs &a, void *stream);

}  // namespace detfold_impl

#endif  // DETFOLD_DRAFT_H
