// draft.cpp -- the host side of the drafted step's operators: argument checks
// and planning (no device access), and their C ABI.  Every check comes before
// any HIP call, so an argument error never touches the device; nothing here
// allocates, synchronizes or keeps a pointer.

#include <cmath>
#include <cstdint>

#include "decode_check.h"
#include "draft.h"
#include "internal.h"

namespace detfold_impl {
namespace {

constexpr int64_t kFewSteps = 4;

// Whether a written [n0][n1][n2][last] buffer has no element twice: in the order
// of the strides, each passes what lies within it.
bool distinct3(int64_t (&d)[3][2], int64_t last)
{
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2 - i; ++j)
            if (d[j][1] > d[j + 1][1]) {
                const int64_t n = d[j][0], s = d[j][1];
                d[j][0] = d[j + 1][0], d[j][1] = d[j + 1][1];
                d[j + 1][0] = n, d[j + 1][1] = s;
            }
    int64_t inner = last;
    for (const auto &x : d)
        if (x[0] > 1) {
            if (x[1] < inner)
                return false;
            inner += (x[0] - 1) * x[1];
        }
    return true;
}

int64_t span3(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t last)
{
    const int64_t d[3][2] = {{n0, s0}, {n1, s1}, {n2, s2}};
    return span(d, 3, last);
}

bool same_cache(const detfold_paged_cache &a, const detfold_paged_cache &b)
{
    return a.k == b.k && a.v == b.v && a.pages == b.pages && a.k_page == b.k_page && a.k_token == b.k_token && a.k_head == b.k_head &&
           a.v_page == b.v_page && a.v_token == b.v_token && a.v_head == b.v_head;
}

// Whether heads are whole chunks of 16 bytes, at such addresses, and pages and tokens
// less than 2^31 bytes apart.
bool tree_staged(const detfold_paged_cache &c)
{
    const int64_t of = 16 / elem_size(c.type);
    for (int64_t x : {c.k_page, c.k_token, c.v_page, c.v_token})
        if (x >= kMaxCount / elem_size(c.type))
            return false;
    for (int64_t x : {c.k_page, c.k_token, c.k_head, c.v_page, c.v_token, c.v_head, (int64_t)c.dim, (int64_t)c.v_dim})
        if (x % of != 0)
            return false;
    return aligned(c.k, 16) && aligned(c.v, 16) && c.dim <= 128 && c.v_dim <= 128;
}

}  // namespace

// What plan_attend does, with up to 32 queries of a key-value head to a unit.
int plan_tree(const detfold_paged_cache &c, int64_t batch, int32_t drafts, int32_t q_heads, int64_t max_len, int64_t window, int32_t split,
              int32_t type, int32_t out_type, int32_t cu_count, TreePlan *p)
{
    AttendPlan checked;
    const int rc = plan_attend(c, batch, q_heads, max_len, window, split, false, cu_count, &checked);
    if (rc != DETFOLD_OK)
        return rc;
    if (drafts < 1 || drafts > DETFOLD_MAX_DRAFTS || max_len > kMaxCount - 1 - DETFOLD_MAX_DRAFTS || !types_pair(type, c.type) ||
        (out_type != type && out_type != DETFOLD_F32))
        return DETFOLD_EINVAL;
    const int64_t cols = (int64_t)drafts * (q_heads / c.heads), pairs = (cols + 31) / 32;
    // At least the units times a slot's queries, however they are dealt out below.
    const int64_t queries = c.heads * (cols <= 16 ? cols : 32 * (pairs <= 2 ? pairs : pairs <= 4 ? 4 : (pairs + 7) / 8 * 8));
    if (batch > 0 && queries > kMaxElems / 16 / batch)
        return DETFOLD_EINVAL;
    const int head = c.dim > c.v_dim ? c.dim : c.v_dim, wide_head = head <= 64 ? 64 : head <= 128 ? 128 : 256;
    const int64_t seen = window > 0 && window < max_len - (drafts - 1) ? window + drafts - 1 : max_len, full = cu_count;
    // Two tiles of 16 queries to a wave share what is loaded, where the products are
    // of 16 bits and there are as many queries.  Four do not fit the registers with
    // eight waves to a compute unit (1 x 16 tokens over 131072 took 163 us with four,
    // 139 with two).  Products in float32, and in parts, are what bounds one tile
    // already.  Where one step for every wave that the device holds is enough, its
    // time is the code's, which one tile has less of (1 x 8 over 1000: 17 us, 20 with
    // two).  One token a row is split as attend_paged splits it, in the same
    // workspace.
    const bool narrow = type != DETFOLD_F32 && out_type != DETFOLD_F32;
    const bool once = split == 0 && batch * ((seen + 31) / 32) <= full * kWavesPerCu / (c.heads * ((cols + 15) / 16));
    const int tiles = narrow && drafts > 1 && cols > 16 && !once ? 2 : 1;
    int64_t of_head = (cols + 16 * tiles - 1) / (16 * tiles);  // units of a key-value head
    // More units than one of a key-value head take its tokens from LDS together: 2, 4 or
    // 8 to a workgroup (1 x 16 tokens over 131072, two units: 122 us, 128 straight to
    // registers; 32 x 64 over 4096, eight: 281 and 377).
    const int most_shared = wide_head * elem_size(c.type) >= 128 ? 8 : 4;
    p->shared = tiles < 2 || of_head < 2 || !tree_staged(c) ? 0 : of_head <= 2 ? 2 : of_head <= 4 || most_shared == 4 ? 4 : 8;
    if (p->shared)
        of_head = (of_head + p->shared - 1) / p->shared * p->shared;
    const int64_t units = c.heads * of_head;
    // Heads above 128 leave a compute unit's registers four waves.
    const int64_t per_cu = tree_heavy(tiles, wide_head) ? kWavesPerCu / 2 : kWavesPerCu, waves = full * per_cu;
    p->tiles_of = tiles;
    p->slot_cols = (int32_t)(cols < 16 * tiles ? cols : 16 * tiles);
    p->units = batch * units;
    p->shares = 0;
    p->waves = (int32_t)per_cu;
    p->beside = p->shared ? p->shared : units % 4 == 0 ? 4 : units % 2 == 0 ? 2 : 1;
    p->brief = seen <= 32;
    const int64_t groups = units / p->beside;
    const int fit = 1024 / (wide_head * elem_size(c.type)), most_tiles = tiles > 1 || wide_head == 256 ? 2 : 4;
    // Three steps of each of four waves take less than a join, as for one token.  Straight
    // to registers trees have eight waves to a workgroup, for which it is half of that.
    const int64_t few = p->shared ? 3 * 32 * (p->waves / p->shared) : 3 * 16 * (fit < most_tiles ? fit : most_tiles) * (4 / p->beside);
    int64_t part = split > 0 ? split : kLongPart;
    if (split == 0) {
        if (seen <= few || (batch * groups >= full && seen <= kShortRow)) {
            part = seen;
        } else if (batch > 0 && !p->shared && batch * ((seen + 31) / 32) <= waves / units) {
            part = DETFOLD_ATTEND_STEP;
            p->brief = true;
            p->waves = p->beside;
        } else if (batch > 0 && groups <= full / 2 && batch <= kMaxEven && batch * (seen / 32 + 2) < kMaxCount / 2) {
            p->shares = full / groups;
            const int64_t even = (batch * seen + p->shares - 1) / p->shares, half = (seen + 1) / 2;
            part = even < half ? even : half;
            // Shares of a few steps for every wave would pay for two rows' ends where a
            // part of one row pays for one (7 x 13 float32 tokens over 1500: 31.5 us in
            // parts, 35 in shares).
            if (even <= kFewSteps * 32 * (p->waves / p->beside) && batch * groups <= full) {
                p->shares = 0;
                part = (seen + full / (batch * groups) - 1) / (full / (batch * groups));
            }
        } else if (batch > 0 && seen > kMaxBlocks / p->units * part) {
            part = (seen - 1) / (kMaxBlocks / p->units + 1) + 1;
        }
        part = (part + DETFOLD_ATTEND_STEP - 1) / DETFOLD_ATTEND_STEP * DETFOLD_ATTEND_STEP + (part == 0) * DETFOLD_ATTEND_STEP;
    }
    p->splits = seen > part ? (seen + part - 1) / part : 1;
    p->split = p->splits > 1 ? part : seen;
    // A part leaves v_dim sums, its maximum and its sum of weights per query.
    // Shares and short parts leave no more than the device holds queries of at once,
    // twice, whatever the rows; parts of a fixed length as many as the rows have.
    const int64_t each = ((int64_t)c.v_dim + 2) * 4, least = split > 0 ? split : kLongPart, most = (max_len + least - 1) / least;
    p->slots = p->shares ? 2 * p->shares * units : p->splits > 1 ? p->units * p->splits : 0;
    p->workspace_bytes = batch > 0 ? p->slots * p->slot_cols * each + p->shares * 12 : 0;
    if (split > 0 && most > 0 && batch > 0 && queries * batch > kMaxElems / most)
        return DETFOLD_EINVAL;
    int64_t upto = most > 1 ? (most < kMaxBlocks ? most : kMaxBlocks) * queries * batch : 0;
    if (split == 0) {
        const int64_t capped = kMaxBlocks * 32 + 2 * queries * batch, even = kWavesPerCu * 2 * cu_count * (cols < 32 ? cols : 32);
        upto = upto > capped ? capped : upto;
        upto = upto > even ? upto : even;
    }
    p->workspace_upto = batch > 0 && max_len > (split > 0 ? split : DETFOLD_ATTEND_STEP) ? upto * each + full * 12 : 0;
    return DETFOLD_OK;
}

int check_tree(const detfold_paged_cache *c, const detfold_tree *t)
{
    int rc = check_cache(c);
    if (rc != DETFOLD_OK)
        return rc;
    if (!t)
        return DETFOLD_EINVAL;
    const detfold_attend &a = t->attend;
    if (a.reserved != 0 || !types_pair(a.type, c->type) || (a.out_type != a.type && a.out_type != DETFOLD_F32) || t->drafts < 1 ||
        t->drafts > DETFOLD_MAX_DRAFTS || !(t->cap == 0.0f || std::isnormal(t->cap)) || t->cap < 0.0f)
        return DETFOLD_EINVAL;
    TreePlan p;  // checks the counts; the device's own plan follows
    if ((rc = plan_tree(*c, a.batch, t->drafts, a.q_heads, a.max_len, a.window, a.split, a.type, a.out_type, 1, &p)) != DETFOLD_OK)
        return rc;
    // Times log2 e, as the kernel holds them, both are finite.
    if (!(std::fabs(a.scale) <= 0x1p127f) || !(t->cap <= 0x1p127f) || a.table_width < 0 || a.table_row < 0 || a.workspace_bytes < 0)
        return DETFOLD_EINVAL;
    if (t->masks && !t->depths && (a.window > 0 || t->slopes))
        return DETFOLD_EINVAL;
    if (a.batch == 0)
        return DETFOLD_OK;
    if (!a.out || !a.q || !a.lens || (a.table_width > 0 && !a.table))
        return DETFOLD_EINVAL;
    const int size = elem_size(a.type), out_size = elem_size(a.out_type);
    const int64_t qs = span3(a.batch, a.q_row, t->drafts, t->q_draft, a.q_heads, a.q_head, c->dim);
    const int64_t os = span3(a.batch, a.out_row, t->drafts, t->out_draft, a.q_heads, a.out_head, c->v_dim);
    const int64_t ts = a.table_width > 0 ? span2(a.batch, a.table_row, 1, 0, a.table_width) : 0;
    if (qs < 0 || os < 0 || ts < 0)
        return DETFOLD_EINVAL;
    if (!aligned(a.q, (uintptr_t)size) || !aligned(a.out, (uintptr_t)out_size) || !aligned(a.lse, 4) || !aligned(a.table, 4) ||
        !aligned(a.lens, 4) || !aligned(a.workspace, 16) || !aligned(t->masks, 8) || !aligned(t->counts, 4) || !aligned(t->depths, 4) ||
        !aligned(t->slopes, 4))
        return DETFOLD_EINVAL;
    int64_t dims[3][2] = {{a.batch, a.out_row}, {t->drafts, t->out_draft}, {a.q_heads, a.out_head}};
    if (!distinct3(dims, c->v_dim))
        return DETFOLD_EOVERLAP;
    const int64_t queries = a.batch * t->drafts;
    const Range out = range(a.out, os, out_size), lse = range(a.lse, queries * a.q_heads, 4);
    const Range work = range(a.workspace, a.workspace_bytes, 1);
    const Range in[] = {range(a.q, qs, size), range(a.table, ts, 4), range(a.lens, a.batch, 4), range(t->masks, queries, 8),
                        range(t->counts, a.batch, 4), range(t->depths, queries, 4), range(t->slopes, a.q_heads, 4),
                        cache_range(*c, false), cache_range(*c, true), range(c->k_scale, c->heads, 4), range(c->v_scale, c->heads, 4)};
    for (const Range &r : in)
        if (meet(out, r) || meet(lse, r) || meet(work, r))
            return DETFOLD_EOVERLAP;
    if (meet(out, lse) || meet(out, work) || meet(lse, work))
        return DETFOLD_EOVERLAP;
    return DETFOLD_OK;
}

namespace {

// The runs of a cache's keys or values, [pages][page][heads] of `last` elements each.
struct Runs {
    int64_t n[3], s[3], last;
    int64_t span(int from) const
    {
        int64_t e = last;
        for (int i = from; i < 3; ++i)
            e += (n[i] - 1) * s[i];
        return e;
    }
};
Runs all_runs(const detfold_paged_cache &c, bool values)
{
    const int64_t head = values ? c.v_head : c.k_head;  // 0: all heads are one
    return {{c.pages, c.page, head == 0 ? 1 : c.heads}, {values ? c.v_page : c.k_page, values ? c.v_token : c.k_token, head},
            values ? c.v_dim : c.dim};
}

// Which elements two sets of runs share, of which neither has one twice: none, some of
// runs of the same indexes, or others.  `apart` is from the first run of the one to that
// of the other.  Dims come in the order of their strides, so what lies within one index
// spans no more than its stride, and of all differences of an index two can meet.
// Runs that are not equally far apart, or in another order, count as sharing others
// where their spans meet.
enum { kNone, kSame, kOthers };
int shared_runs(const Runs &a, const Runs &b, int64_t apart, int i = 0, bool moved = false)
{
    if (apart >= a.span(i) || apart <= -b.span(i))
        return kNone;
    if (i == 3)
        return moved ? kOthers : kSame;
    if (a.n[i] == 1 && b.n[i] == 1)
        return shared_runs(a, b, apart, i + 1, moved);
    if (a.n[i] != b.n[i] || a.s[i] != b.s[i] || a.span(i + 1) > a.s[i] || b.span(i + 1) > b.s[i])
        return kOthers;
    const int64_t n = a.n[i], s = a.s[i], down = (apart >= 0 ? apart : apart - (s - 1)) / s;
    int most = kNone;
    for (int64_t j : {down, down + 1})
        if (j > -n && j < n) {
            const int got = shared_runs(a, b, apart - j * s, i + 1, moved || j != 0);
            most = got > most ? got : most;
        }
    return most;
}

}  // namespace

// The runs of a token that a compaction in place moves, each in a workgroup of its own:
// heads that are one move once, and so do values that lie within the keys, or keys
// within the values.  Runs that share memory otherwise are refused.
int runs_in_place(const detfold_paged_cache &c, int32_t *keys, int32_t *values)
{
    Runs k = all_runs(c, false), v = all_runs(c, true);
    for (const Runs *r : {&k, &v}) {
        int64_t dims[3][2] = {{r->n[0], r->s[0]}, {r->n[1], r->s[1]}, {r->n[2], r->s[2]}};
        if (!distinct3(dims, r->last))
            return DETFOLD_EOVERLAP;
    }
    *keys = (int32_t)k.n[2], *values = (int32_t)v.n[2];
    for (int i = 0; i < 2; ++i)  // the largest strides first
        for (int j = 0; j < 2 - i; ++j) {
            auto stride = [&](int d) { return k.n[d] > 1 ? k.s[d] : v.n[d] > 1 ? v.s[d] : 0; };
            if (stride(j) < stride(j + 1))
                for (Runs *r : {&k, &v}) {
                    const int64_t n = r->n[j], s = r->s[j];
                    r->n[j] = r->n[j + 1], r->s[j] = r->s[j + 1];
                    r->n[j + 1] = n, r->s[j + 1] = s;
                }
        }
    const int64_t apart = ((int64_t)(uintptr_t)c.v - (int64_t)(uintptr_t)c.k) / elem_size(c.type);
    const int shared = shared_runs(k, v, apart);
    if (shared == kNone)
        return DETFOLD_OK;
    if (shared == kSame && apart >= 0 && apart + c.v_dim <= c.dim)
        *values = 0;
    else if (shared == kSame && apart <= 0 && c.dim - apart <= c.v_dim)
        *keys = 0;
    else
        return DETFOLD_EOVERLAP;
    return DETFOLD_OK;
}

namespace {

// Whether a token copied from c to w writes no element of w with two values: what is one
// memory in w, heads or keys and values, is so in c.
bool takes_copies(const detfold_paged_cache &c, const detfold_paged_cache &w)
{
    int32_t ck, cv, wk, wv;
    const intptr_t c_apart = (intptr_t)c.v - (intptr_t)c.k, w_apart = (intptr_t)w.v - (intptr_t)w.k;
    if (runs_in_place(w, &wk, &wv) != DETFOLD_OK)  // as it is in c, if that lies the same
        return c_apart == w_apart && c.k_page == w.k_page && c.k_token == w.k_token && c.k_head == w.k_head && c.v_page == w.v_page &&
               c.v_token == w.v_token && c.v_head == w.v_head;
    if (wk == w.heads && wv == w.heads)
        return true;
    return runs_in_place(c, &ck, &cv) == DETFOLD_OK && ck == wk && cv == wv && (wk * wv != 0 || c_apart == w_apart);
}

}  // namespace

int check_copy(const detfold_paged_cache *c, const detfold_paged_cache *into, const int32_t *src, const int32_t *dst,
               const int32_t *tokens, int64_t count)
{
    int rc = check_cache(c);
    if (rc != DETFOLD_OK || (into && (rc = check_cache(into)) != DETFOLD_OK))
        return rc;
    if (into && (into->page != c->page || into->heads != c->heads || into->dim != c->dim || into->v_dim != c->v_dim || into->type != c->type))
        return DETFOLD_EINVAL;
    if (count < 0 || count >= kMaxCount || c->page > kMaxMoved)
        return DETFOLD_EINVAL;
    if (count == 0)
        return DETFOLD_OK;
    if (!src || !dst || !aligned(src, 4) || !aligned(dst, 4) || !aligned(tokens, 4))
        return DETFOLD_EINVAL;
    const Range from[] = {cache_range(*c, false), cache_range(*c, true)};
    const detfold_paged_cache &w = into ? *into : *c;
    const Range to[] = {cache_range(w, false), cache_range(w, true)};
    const Range lists[] = {range(src, count, 4), range(dst, count, 4), range(tokens, count, 4)};
    for (const Range &t : to) {
        for (const Range &r : lists)
            if (meet(t, r))
                return DETFOLD_EOVERLAP;
        if (into && !same_cache(*c, *into))
            for (const Range &r : from)
                if (meet(t, r))
                    return DETFOLD_EOVERLAP;
    }
    return into && !takes_copies(*c, *into) ? DETFOLD_EOVERLAP : DETFOLD_OK;
}

int check_compact(const detfold_paged_cache *c, const detfold_compact *a)
{
    int rc = check_cache(c);
    if (rc != DETFOLD_OK)
        return rc;
    if (!a || a->batch < 0 || a->batch >= kMaxCount || a->most < 0 || a->most >= kMaxCount || a->table_row < 0 || a->table_width < 0 ||
        (a->to && (a->to_row < 0 || a->to_width < 0)))
        return DETFOLD_EINVAL;
    if (a->batch == 0 || a->most == 0)
        return DETFOLD_OK;
    if (!a->picks || !a->counts || (a->table_width > 0 && !a->table))
        return DETFOLD_EINVAL;
    for (const void *p : {a->table, a->to, a->picks, a->counts, a->starts})
        if (!aligned(p, 4))
            return DETFOLD_EINVAL;
    if (a->to && a->most > kMaxMoved)
        return DETFOLD_EINVAL;
    const int64_t ts = a->table_width > 0 ? span2(a->batch, a->table_row, 1, 0, a->table_width) : 0;
    const int64_t os = a->to && a->to_width > 0 ? span2(a->batch, a->to_row, 1, 0, a->to_width) : 0;
    if (ts < 0 || os < 0 || a->most > kMaxElems / a->batch)
        return DETFOLD_EINVAL;
    const Range in[] = {range(a->table, ts, 4), range(a->to, os, 4), range(a->picks, a->batch * a->most, 4), range(a->counts, a->batch, 4),
                        range(a->starts, a->batch, 4)};
    const Range k = cache_range(*c, false), v = cache_range(*c, true);
    for (const Range &r : in)
        if (meet(k, r) || meet(v, r))
            return DETFOLD_EOVERLAP;
    return DETFOLD_OK;
}

namespace {

int chunks_of(int64_t bytes) { return (int)((bytes + 15) / 16); }

// A token's runs: heads that lie beside each other, on both sides, are one.
TokenRuns runs_of(const detfold_paged_cache &c, const detfold_paged_cache &w, bool values)
{
    const int64_t size = elem_size(c.type), dim = values ? c.v_dim : c.dim;
    const bool joined = values ? c.v_head == dim && w.v_head == dim : c.k_head == dim && w.k_head == dim;
    TokenRuns r;
    r.run = (int32_t)(size * dim * (joined ? c.heads : 1));
    r.chunks = divider((uint32_t)chunks_of(r.run));
    r.token = divider(r.chunks.d * (uint32_t)(joined ? 1 : c.heads));
    return r;
}

CopySide copy_side(const detfold_paged_cache &c, const detfold_paged_cache &w, bool values)
{
    const int64_t size = elem_size(c.type);
    return {(const char *)(values ? c.v : c.k), (char *)(values ? w.v : w.k),
            size * (values ? c.v_page : c.k_page), size * (values ? c.v_token : c.k_token), size * (values ? c.v_head : c.k_head),
            size * (values ? w.v_page : w.k_page), size * (values ? w.v_token : w.k_token), size * (values ? w.v_head : w.k_head)};
}

CompactSide compact_side(const detfold_paged_cache &c, bool values)
{
    const int64_t size = elem_size(c.type), run = size * (values ? c.v_dim : c.dim);
    return {(char *)(values ? c.v : c.k), size * (values ? c.v_page : c.k_page), size * (values ? c.v_token : c.k_token),
            size * (values ? c.v_head : c.k_head), (int32_t)run, divider((uint32_t)chunks_of(run))};
}

}  // namespace

}  // namespace detfold_impl

using namespace detfold_impl;

// ---------------------------------------------------------------------------
// C ABI

extern "C" {

int detfold_plan_tree(const detfold_paged_cache *cache, int64_t batch, int32_t drafts, int32_t q_heads, int64_t max_len,
                      int64_t window, int32_t split, int32_t type, int32_t out_type, int32_t cu_count, detfold_attend_plan *plan)
{
    if (!plan || drafts < 1 || drafts > DETFOLD_MAX_DRAFTS)
        return DETFOLD_EINVAL;
    TreePlan p;
    int rc = check_cache(cache);
    if (rc == DETFOLD_OK)
        rc = plan_tree(*cache, batch, drafts, q_heads, max_len, window, split, type, out_type, cu_count, &p);
    if (rc == DETFOLD_OK)
        *plan = p;
    return rc;
}

int detfold_tree_workspace(const detfold_paged_cache *cache, int64_t batch, int32_t drafts, int32_t q_heads, int64_t max_len,
                           int32_t split, int64_t *bytes)
{
    if (!bytes)
        return DETFOLD_EINVAL;
    detfold_attend_plan p;
    // What any type of query needs: float32 goes with every cache but of float16.
    const int32_t type = cache && cache->type == DETFOLD_F16 ? DETFOLD_F16 : DETFOLD_F32;
    int rc = detfold_plan_tree(cache, batch, drafts, q_heads, max_len, 0, split, type, type, 1, &p);
    if (rc != DETFOLD_OK)
        return rc;
    int32_t cu = 0;
    if ((rc = current_cu_count(&cu)) != DETFOLD_OK)
        return rc;
    rc = detfold_plan_tree(cache, batch, drafts, q_heads, max_len, 0, split, type, type, cu, &p);
    *bytes = p.workspace_upto;
    return rc;
}

int detfold_attend_tree(const detfold_paged_cache *cache, const detfold_tree *args, void *stream)
{
    int rc = check_tree(cache, args);
    if (rc != DETFOLD_OK || args->attend.batch == 0)
        return rc;
    int32_t cu = 0;
    if ((rc = current_cu_count(&cu)) != DETFOLD_OK)
        return rc;
    const detfold_attend &a = args->attend;
    TreePlan p;
    if ((rc = plan_tree(*cache, a.batch, args->drafts, a.q_heads, a.max_len, a.window, a.split, a.type, a.out_type, cu, &p)) != DETFOLD_OK)
        return rc;
    const int64_t units = p.units / a.batch;
    if (units / p.beside * p.splits > kMaxBlocks)
        return DETFOLD_EINVAL;
    if (p.workspace_bytes > 0 && (!a.workspace || a.workspace_bytes < p.workspace_bytes))
        return DETFOLD_ESIZE;
    TreeArgs k = {};
    k.c = *cache;
    k.a = a;
    k.masks = args->masks, k.counts = args->counts, k.depths = args->depths, k.slopes = args->slopes;
    k.q_draft = args->q_draft, k.out_draft = args->out_draft;
    k.window = a.window;
    if (a.window > 0)
        k.a.window = (a.window < kMaxCount ? a.window : kMaxCount) + args->drafts - 1;
    k.cap = args->cap;
    k.drafts = args->drafts;
    k.group = a.q_heads / cache->heads;
    k.heads_of = divider((uint32_t)k.group);
    k.page = divider((uint32_t)cache->page);
    k.tiles_of = p.tiles_of;
    k.slot_cols = p.slot_cols;
    k.shared = p.shared;
    k.tiles = divider((uint32_t)(units / cache->heads));
    k.beside = p.beside;
    k.units = divider((uint32_t)(units / p.beside));
    k.parts = divider((uint32_t)(p.shares ? 1 : p.splits));
    k.shares = p.shares ? divider((uint32_t)p.shares) : Divider{0, 0, 0};
    k.brief = p.brief;
    k.split = p.split;
    k.tiled = attend_tiled(*cache) && !p.shared;
    k.keep = attend_keep(*cache, k.tiles.d, k.brief);
    k.waves = p.waves;
    const int64_t queries = p.slots * p.slot_cols;
    k.ml = (float2 *)a.workspace;
    k.acc = (float *)(k.ml + queries);
    k.cut = (int3 *)(k.acc + queries * cache->v_dim);
    k.by_row = a.batch <= p.shares;
    return launch_tree(k, stream);
}

int detfold_cache_copy(const detfold_paged_cache *cache, const detfold_paged_cache *into, const int32_t *src, const int32_t *dst,
                       const int32_t *tokens, int64_t count, void *stream)
{
    const int rc = check_copy(cache, into, src, dst, tokens, count);
    if (rc != DETFOLD_OK || count == 0)
        return rc;
    const detfold_paged_cache &w = into ? *into : *cache;
    CopyArgs k = {};
    k.m.k = runs_of(*cache, w, false), k.m.v = runs_of(*cache, w, true);
    k.k = copy_side(*cache, w, false), k.v = copy_side(*cache, w, true);
    k.page = divider((uint32_t)cache->page);
    k.src = src, k.dst = dst, k.tokens = tokens;
    k.pages = cache->pages, k.into_pages = w.pages;
    return launch_copy_pages(k, count, stream);
}

int detfold_cache_compact(const detfold_paged_cache *cache, const detfold_compact *args, void *stream)
{
    int rc = check_compact(cache, args);
    if (rc != DETFOLD_OK || args->batch == 0 || args->most == 0)
        return rc;
    CompactArgs k = {};
    if (!args->to) {
        int32_t keys = 0, values = 0;
        if ((rc = runs_in_place(*cache, &keys, &values)) != DETFOLD_OK)
            return rc;
        k.k_runs = keys;
        k.runs = divider((uint32_t)(keys + values));
    }
    k.a = *args;
    k.m.k = runs_of(*cache, *cache, false), k.m.v = runs_of(*cache, *cache, true);
    k.k = compact_side(*cache, false), k.v = compact_side(*cache, true);
    k.pages = cache->pages;
    k.page = divider((uint32_t)cache->page);
    k.most = divider((uint32_t)args->most);
    return launch_compact(k, stream);
}

}  // extern "C"
