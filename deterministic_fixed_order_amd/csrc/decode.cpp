// decode.cpp -- the host side of the decode-step operators: argument checks
// and planning (no device access), and their C ABI.  Every check comes before
// any HIP call, so an argument error never touches the device; nothing here
// allocates, synchronizes or keeps a pointer.

#include <cmath>
#include <cstdint>

#include "decode_check.h"
#include "internal.h"

namespace detfold_impl {
namespace {


// A view [tokens][heads][dim], in elements.
struct Heads {
    const void *p;
    int64_t token, head, heads, dim;
};

// Whether x + t * step lies within (-b, a) for some |t| < tokens.
bool reaches(int64_t x, int64_t step, int64_t tokens, int64_t a, int64_t b)
{
    if (tokens == 1 || step == 0)
        return x > -b && x < a;
    const int64_t y = -b - x;  // the first t with t * step > y
    const int64_t t = (y >= 0 ? y / step : -((-y + step - 1) / step)) + 1;
    return t < tokens && x + (t > -tokens ? t : 1 - tokens) * step < a;
}

// Whether two such views, whose spans meet, share an element.  Of tokens that are
// not equally far apart, and of more than 2^20 pairs of heads that interleave, it
// is taken as given.
bool share_elements(const Heads &q, const Heads &k, int64_t tokens, int size)
{
    if (tokens > 1 && q.token != k.token)
        return true;
    const int64_t apart = ((int64_t)(uintptr_t)k.p - (int64_t)(uintptr_t)q.p) / size;
    if (!reaches(apart, q.token, tokens, (q.heads - 1) * q.head + q.dim, (k.heads - 1) * k.head + k.dim))
        return false;
    if (q.heads * k.heads > (int64_t)1 << 20)
        return true;
    for (int64_t i = 0; i < q.heads; ++i)
        for (int64_t j = 0; j < k.heads; ++j)
            if (reaches(apart + j * k.head - i * q.head, q.token, tokens, q.dim, k.dim))
                return true;
    return false;
}

}  // namespace

bool types_pair(int32_t type, int32_t cache_type)
{
    if (type != DETFOLD_F32 && type != DETFOLD_BF16 && type != DETFOLD_F16)
        return false;
    return cache_type == type || cache_type == DETFOLD_E4M3 ||
           (type == DETFOLD_F32 && cache_type == DETFOLD_BF16);
}

int check_cache(const detfold_paged_cache *c)
{
    if (!c || !c->k || !c->v || c->reserved != 0 || c->type < DETFOLD_F32 || c->type > DETFOLD_E4M3)
        return DETFOLD_EINVAL;
    if (c->pages < 1 || c->page < 1 || c->pages >= kMaxCount / c->page || c->heads < 1 || c->heads > kMaxHeads)
        return DETFOLD_EINVAL;
    for (int32_t d : {c->dim, c->v_dim})
        if (d < DETFOLD_MIN_HEAD || d > DETFOLD_MAX_HEAD)
            return DETFOLD_EINVAL;
    if (cache_span(*c, false) < 0 || cache_span(*c, true) < 0)
        return DETFOLD_EINVAL;
    const uintptr_t size = (uintptr_t)elem_size(c->type);
    if (!aligned(c->k, size) || !aligned(c->v, size) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
        return DETFOLD_EINVAL;
    if (c->type != DETFOLD_E4M3 && (c->k_scale || c->v_scale))
        return DETFOLD_EINVAL;
    return DETFOLD_OK;
}

int check_append(const detfold_paged_cache *c, const detfold_append *a)
{
    int rc = check_cache(c);
    if (rc != DETFOLD_OK)
        return rc;
    if (!a || a->tokens < 0 || a->tokens >= kMaxCount || a->q_heads < 0 || a->q_heads > kMaxHeads ||
        a->rot < 0 || a->rot > c->dim || (a->rot & 1) || (a->pairs != 0 && a->pairs != 1) || a->angles < 0 ||
        !types_pair(a->type, c->type))
        return DETFOLD_EINVAL;
    if (a->tokens == 0)
        return DETFOLD_OK;
    if (!a->k || !a->v || !a->slots || (a->q_heads > 0) != (a->q != nullptr) || (a->q != nullptr) != (a->q_out != nullptr))
        return DETFOLD_EINVAL;
    if (a->rot > 0 && (!a->positions || !a->cos || !a->sin || a->angles < 1 || a->angles > kMaxElems / 128))
        return DETFOLD_EINVAL;
    const int size = elem_size(a->type);
    const int64_t nq = a->q_heads > 0 ? a->q_heads : 1;
    const int64_t ks = span2(a->tokens, a->k_token, c->heads, a->k_head, c->dim);
    const int64_t vs = span2(a->tokens, a->v_token, c->heads, a->v_head, c->v_dim);
    const int64_t qs = a->q ? span2(a->tokens, a->q_token, nq, a->q_head, c->dim) : 0;
    const int64_t os = a->q ? span2(a->tokens, a->out_token, nq, a->out_head, c->dim) : 0;
    if (ks < 0 || vs < 0 || qs < 0 || os < 0)
        return DETFOLD_EINVAL;
    for (const void *p : {a->k, a->v, a->q, (const void *)a->q_out})
        if (!aligned(p, (uintptr_t)size))
            return DETFOLD_EINVAL;
    if (!aligned(a->slots, 8) || !aligned(a->positions, 8) || !aligned(a->cos, 4) || !aligned(a->sin, 4))
        return DETFOLD_EINVAL;
    if (a->q_out && !distinct(a->tokens, a->out_token, nq, a->out_head, c->dim))
        return DETFOLD_EOVERLAP;
    // What is written (q_out, the cache) against what is read and against each other.
    const Range k = cache_range(*c, false), v = cache_range(*c, true);
    const Range in[] = {range(a->k, ks, size), range(a->v, vs, size), range(a->q, qs, size),
                        range(a->slots, a->tokens, 8),
                        range(a->rot ? a->positions : nullptr, a->tokens, 8),
                        range(a->rot ? a->cos : nullptr, a->angles * (a->rot / 2), 4),
                        range(a->rot ? a->sin : nullptr, a->angles * (a->rot / 2), 4),
                        range(c->k_scale, c->heads, 4), range(c->v_scale, c->heads, 4)};
    const Range out = range(a->q_out, os, size);
    // In place, a query view among its neighbours of one projection: the
    // spans of k and v interleave with it, its elements must not.
    const bool in_place = a->q_out && a->q_out == a->q && a->out_token == a->q_token && a->out_head == a->q_head;
    const Heads turned = {a->q, a->q_token, a->q_head, nq, c->dim};
    const Heads beside[] = {{a->k, a->k_token, a->k_head, c->heads, c->dim}, {a->v, a->v_token, a->v_head, c->heads, c->v_dim}};
    for (int i = 0; i < (int)(sizeof(in) / sizeof(in[0])); ++i) {
        if (meet(k, in[i]) || meet(v, in[i]))
            return DETFOLD_EOVERLAP;
        if (meet(out, in[i]) && !(in_place && (i == 2 || (i < 2 && !share_elements(turned, beside[i], a->tokens, size)))))
            return DETFOLD_EOVERLAP;
    }
    if (meet(out, k) || meet(out, v))
        return DETFOLD_EOVERLAP;
    return DETFOLD_OK;
}

// The widest access of at most 16 bytes that each of these runs of values holds
// at least once (the last one of a run may then overlap another, which writes
// the same), or, where a write must not come before another's read, divides.
int access_width(int type, bool overlap, int64_t a, int64_t b, int64_t c)
{
    int v = 16 / elem_size(type);
    for (int64_t n : {a, b, c})
        while (overlap ? n > 0 && n < v : n % v != 0)
            v /= 2;
    return v;
}

int append_width(const detfold_paged_cache &c, const detfold_append &a)
{
    const bool in_place = a.q_heads > 0 && a.q == a.q_out;
    return access_width(a.type, !in_place, a.rot / 2, c.dim - a.rot, c.v_dim);
}

int plan_attend(const detfold_paged_cache &c, int64_t batch, int32_t q_heads, int64_t max_len,
                int64_t window, int32_t split, bool wide, int32_t cu_count, AttendPlan *p)
{
    if (batch < 0 || batch >= kMaxCount || max_len < 0 || max_len >= kMaxCount || window < 0 || q_heads < 1 ||
        q_heads > kMaxHeads || q_heads % c.heads != 0 || split < 0 || split % DETFOLD_ATTEND_STEP != 0 || cu_count < 1)
        return DETFOLD_EINVAL;
    const int64_t group = q_heads / c.heads, tiles = (group + 15) / 16, units = c.heads * tiles;
    const int64_t seen = window > 0 && window < max_len ? window : max_len;
    const int64_t full = cu_count, waves = (int64_t)cu_count * kWavesPerCu;
    p->units = batch * units;
    p->shares = 0;
    p->waves = wide || 64 * (c.dim + c.v_dim) * elem_size(c.type) < kStepBytes ? 8 : 4;
    p->beside = units % 4 == 0 ? 4 : units % 2 == 0 ? 2 : 1;
    p->brief = seen <= 32;
    const int64_t groups = units / p->beside;
    // Three steps of a wave take less than a join (1 token 6.6 us, each step of 64
    // bfloat16 tokens 1.2 more, one of 1000 in parts 11.5).
    const int head = c.dim > c.v_dim ? c.dim : c.v_dim, wide_head = head <= 64 ? 64 : head <= 128 ? 128 : 256;
    const int tiles_fit = 1024 / (wide_head * elem_size(c.type)), tiles_most = wide_head == 256 ? 2 : 4;
    const int64_t few = 3 * 16 * (tiles_fit < tiles_most ? tiles_fit : tiles_most) * (4 / p->beside);
    int64_t part = split > 0 ? split : kLongPart;
    if (split == 0) {
        if (seen <= few || (batch * groups >= full && seen <= kShortRow)) {
            part = seen;
        } else if (batch > 0 && batch * ((seen + 31) / 32) <= waves / units) {
            // One step for every wave that the device holds is enough: the
            // least steps, and no more waves to a workgroup than heads.
            part = DETFOLD_ATTEND_STEP;
            p->brief = true;
            p->waves = p->beside;
        } else if (batch > 0 && groups <= full / 2 && batch <= kMaxEven && batch * (seen / 32 + 2) < kMaxCount / 2) {
            p->shares = full / groups;
            const int64_t even = (batch * seen + p->shares - 1) / p->shares, half = (seen + 1) / 2;
            part = even < half ? even : half;
        } else if (batch > 0 && seen > kMaxBlocks / p->units * part) {
            part = (seen - 1) / (kMaxBlocks / p->units + 1) + 1;
        }
        part = (part + DETFOLD_ATTEND_STEP - 1) / DETFOLD_ATTEND_STEP * DETFOLD_ATTEND_STEP + (part == 0) * DETFOLD_ATTEND_STEP;
    }
    p->splits = seen > part ? (seen + part - 1) / part : 1;
    p->split = p->splits > 1 ? part : seen;
    // A part leaves v_dim sums, its maximum and its sum of weights per query
    // head.  Smaller calls take no more parts of their own, and the number of
    // shares does not depend on them.
    const int64_t each = (group < 16 ? group : 16) * ((int64_t)c.v_dim + 2) * 4;
    const int64_t least = split > 0 ? split : kLongPart, most = (max_len + least - 1) / least;
    const int64_t shared = split > 0 ? 0 : groups <= full / 2 && 2 * (full / groups) * units > waves ? 2 * (full / groups) * units : waves;
    if (p->units > kMaxElems / 16 || (split > 0 && p->units > 0 && most > kMaxElems / p->units))
        return DETFOLD_EINVAL;
    int64_t upto = most == 1 ? 0 : split > 0 || p->units < kMaxBlocks ? p->units * most : kMaxBlocks + 2 * p->units;
    if (split == 0 && upto > kMaxBlocks + 2 * p->units)
        upto = kMaxBlocks + 2 * p->units;
    upto = upto > shared ? upto : shared;
    p->slots = p->shares ? 2 * p->shares * units : p->splits > 1 ? p->units * p->splits : 0;
    p->workspace_bytes = batch > 0 ? p->slots * each + p->shares * 12 : 0;
    p->workspace_upto = batch > 0 && max_len > (split > 0 ? split : few) ? upto * each + full * 12 : 0;
    return DETFOLD_OK;
}

// 16 tokens from a multiple of 16 on lie in one page, and within 2^31 bytes of it.
bool attend_tiled(const detfold_paged_cache &c)
{
    const int64_t far = ((int64_t)1 << 31) / 16 / elem_size(c.type) - DETFOLD_MAX_HEAD;
    return c.page % 16 == 0 && c.k_token < far && c.v_token < far;
}

// What is worth keeping in the caches.  A line that a head's end shares with its
// neighbour, or that another tile of query heads reads too, is read again soon:
// kept, heads of 80 bfloat16 run at 4.9 TB/s instead of 3.8 and 24 queries a
// head at 65 us instead of 84.  Of whole lines the values are not, since one load
// takes all of a row (128 bfloat16: 90 us instead of 98), and the keys, of which
// a load takes 64 bytes a row, are, but where a row is 512 bytes or more (128
// float32: 316 us instead of 329).
int attend_keep(const detfold_paged_cache &c, int tiles, bool brief)
{
    const int size = elem_size(c.type), k = c.dim * size, v = c.v_dim * size;
    if (brief || tiles > 1 || k % 128 || v % 128)
        return kAll;
    return c.dim == c.v_dim && k >= 512 && (c.dim == 128 || c.dim == 256) && attend_tiled(c) ? kNothing : kKeys;
}

int check_attend(const detfold_paged_cache *c, const detfold_attend *a)
{
    int rc = check_cache(c);
    if (rc != DETFOLD_OK)
        return rc;
    if (!a || a->reserved != 0 || !types_pair(a->type, c->type) || (a->out_type != a->type && a->out_type != DETFOLD_F32))
        return DETFOLD_EINVAL;
    AttendPlan p;  // checks the counts; the device's own plan follows
    if ((rc = plan_attend(*c, a->batch, a->q_heads, a->max_len, a->window, a->split, false, 1, &p)) != DETFOLD_OK)
        return rc;
    if (!std::isfinite(a->scale) || a->table_width < 0 || a->table_row < 0 || a->workspace_bytes < 0)
        return DETFOLD_EINVAL;
    if (a->batch == 0)
        return DETFOLD_OK;
    if (!a->out || !a->q || !a->lens || (a->table_width > 0 && !a->table))
        return DETFOLD_EINVAL;
    const int size = elem_size(a->type), out_size = elem_size(a->out_type);
    const int64_t qs = span2(a->batch, a->q_row, a->q_heads, a->q_head, c->dim);
    const int64_t os = span2(a->batch, a->out_row, a->q_heads, a->out_head, c->v_dim);
    const int64_t ts = a->table_width > 0 ? span2(a->batch, a->table_row, 1, 0, a->table_width) : 0;
    if (qs < 0 || os < 0 || ts < 0)
        return DETFOLD_EINVAL;
    if (!aligned(a->q, (uintptr_t)size) || !aligned(a->out, (uintptr_t)out_size) || !aligned(a->lse, 4) ||
        !aligned(a->table, 4) || !aligned(a->lens, 4) || !aligned(a->workspace, 16))
        return DETFOLD_EINVAL;
    if (!distinct(a->batch, a->out_row, a->q_heads, a->out_head, c->v_dim))
        return DETFOLD_EOVERLAP;
    const Range out = range(a->out, os, out_size), lse = range(a->lse, a->batch * a->q_heads, 4);
    const Range work = range(a->workspace, a->workspace_bytes, 1);
    const Range in[] = {range(a->q, qs, size), range(a->table, ts, 4), range(a->lens, a->batch, 4),
                        cache_range(*c, false), cache_range(*c, true),
                        range(c->k_scale, c->heads, 4), range(c->v_scale, c->heads, 4)};
    for (const Range &r : in)
        if (meet(out, r) || meet(lse, r) || meet(work, r))
            return DETFOLD_EOVERLAP;
    if (meet(out, lse) || meet(out, work) || meet(lse, work))
        return DETFOLD_EOVERLAP;
    return DETFOLD_OK;
}

int check_softmax(const SoftmaxArgs &s)
{
    if (s.w < 1 || s.rows < 0 || s.dim < 1 || s.dim >= kMaxCount / 2 || s.type < DETFOLD_F32 || s.type > DETFOLD_F16)
        return DETFOLD_EINVAL;
    if (s.rows == 0)
        return DETFOLD_OK;
    if (s.dim > kMaxElems / s.rows || s.outs_pitch < s.rows * s.dim || s.lses_pitch < s.rows)
        return DETFOLD_EINVAL;
    const int64_t os = span2(s.w, s.outs_pitch, 1, 0, s.rows * s.dim);
    const int64_t ls = span2(s.w, s.lses_pitch, 1, 0, s.rows);
    const int size = elem_size(s.type);
    if (os < 0 || ls < 0 || !s.out || !s.outs || !s.lses)
        return DETFOLD_EINVAL;
    if (!aligned(s.out, (uintptr_t)size) || !aligned(s.outs, (uintptr_t)size) || !aligned(s.lses, 4) || !aligned(s.lse, 4))
        return DETFOLD_EINVAL;
    const Range out = range(s.out, s.rows * s.dim, size), lse = range(s.lse, s.rows, 4);
    const Range outs = range(s.outs, os, size), lses = range(s.lses, ls, 4);
    if (meet(out, outs) || meet(out, lses) || meet(lse, outs) || meet(lse, lses) || meet(out, lse))
        return DETFOLD_EOVERLAP;
    return DETFOLD_OK;
}

}  // namespace detfold_impl

using namespace detfold_impl;

// ---------------------------------------------------------------------------
// C ABI

extern "C" {

int detfold_cache_append(const detfold_paged_cache *cache, const detfold_append *args, void *stream)
{
    int rc = check_append(cache, args);
    if (rc != DETFOLD_OK || args->tokens == 0)
        return rc;
    AppendArgs k = {};
    k.c = *cache;
    k.a = *args;
    k.page = divider((uint32_t)cache->page);
    k.width = append_width(*cache, *args);
    return launch_append(k, stream);
}

int detfold_plan_attend(const detfold_paged_cache *cache, int64_t batch, int32_t q_heads, int64_t max_len,
                        int64_t window, int32_t split, int32_t cu_count, detfold_attend_plan *plan)
{
    if (!plan)
        return DETFOLD_EINVAL;
    AttendPlan p;
    int rc = check_cache(cache);
    if (rc == DETFOLD_OK)
        rc = plan_attend(*cache, batch, q_heads, max_len, window, split, false, cu_count, &p);
    if (rc == DETFOLD_OK)
        *plan = p;
    return rc;
}

int detfold_attend_workspace(const detfold_paged_cache *cache, int64_t batch, int32_t q_heads, int64_t max_len,
                             int32_t split, int64_t *bytes)
{
    if (!bytes)
        return DETFOLD_EINVAL;
    detfold_attend_plan p;
    int rc = detfold_plan_attend(cache, batch, q_heads, max_len, 0, split, 1, &p);
    if (rc != DETFOLD_OK)
        return rc;
    int32_t cu = 0;
    if ((rc = current_cu_count(&cu)) != DETFOLD_OK)
        return rc;
    rc = detfold_plan_attend(cache, batch, q_heads, max_len, 0, split, cu, &p);
    *bytes = p.workspace_upto;
    return rc;
}

int detfold_attend_paged(const detfold_paged_cache *cache, const detfold_attend *args, void *stream)
{
    int rc = check_attend(cache, args);
    if (rc != DETFOLD_OK || args->batch == 0)
        return rc;
    int32_t cu = 0;
    if ((rc = current_cu_count(&cu)) != DETFOLD_OK)
        return rc;
    AttendPlan p;
    if ((rc = plan_attend(*cache, args->batch, args->q_heads, args->max_len, args->window, args->split, args->out_type == DETFOLD_F32 && cache->type != DETFOLD_F32, cu,
                          &p)) != DETFOLD_OK)
        return rc;
    const int64_t groups = p.units / args->batch / p.beside;
    if (groups * p.splits > kMaxBlocks)
        return DETFOLD_EINVAL;
    if (p.workspace_bytes > 0 && (!args->workspace || args->workspace_bytes < p.workspace_bytes))
        return DETFOLD_ESIZE;
    AttendArgs k = {};
    k.c = *cache;
    k.a = *args;
    k.group = args->q_heads / cache->heads;
    k.page = divider((uint32_t)cache->page);
    k.tiles = divider((uint32_t)(k.group + 15) / 16);
    k.beside = p.beside;
    k.units = divider((uint32_t)cache->heads * k.tiles.d / p.beside);
    k.parts = divider((uint32_t)(p.shares ? 1 : p.splits));
    k.shares = p.shares ? divider((uint32_t)p.shares) : Divider{0, 0, 0};
    k.brief = p.brief;
    k.split = p.split;
    k.tiled = attend_tiled(*cache);
    k.keep = attend_keep(*cache, k.tiles.d, k.brief);
    k.waves = p.waves;
    const int64_t heads = p.slots * (k.group < 16 ? k.group : 16);
    k.ml = (float2 *)args->workspace;
    k.acc = (float *)(k.ml + heads);
    k.cut = (int3 *)(k.acc + heads * cache->v_dim);
    k.by_row = args->batch <= p.shares;
    return launch_attend(k, stream);
}

int detfold_fold_softmax(void *out, const void *outs, const float *lses, float *lse, int32_t type, int32_t W,
                         int64_t rows, int64_t dim, int64_t outs_pitch, int64_t lses_pitch, void *stream)
{
    const SoftmaxArgs s = {out, outs, lses, lse, rows, dim, outs_pitch, lses_pitch, type, W, {}, 0, 0};
    const int rc = check_softmax(s);
    if (rc != DETFOLD_OK || rows == 0)
        return rc;
    return launch_softmax(s, stream);
}

}  // extern "C"
