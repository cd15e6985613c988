// Host-side argument checks of a serving step's entry points (the 4-bit cache,
// rotary positions, page tables), and how attention over the 4-bit cache is
// laid out over the device.
//
// Pure C++: no HIP header and no device call, like args.cpp.
#include <cstddef>
#include <cstdint>

#include "args_util.hpp"
#include "sgemm.h"
#include "step_plan.hpp"

using namespace sgemm_impl;

namespace {

int check_kv4(const sgemm_kv4_cache *c, const sgemm_kv8_batch *b)
{
    const int rc = check_cache_batch(c, b);
    if (rc != SGEMM_OK) return rc;
    // Four scales are read at once.
    return aligned16(c->Ks) && aligned16(c->Vs) ? SGEMM_OK : SGEMM_ERR_CACHE;
}

struct CacheSpans {
    Span s[4];
};

CacheSpans spans_of(const sgemm_kv4_cache *c)
{
    const i64 ph = i64(c->pages) * c->heads, codes = i64(c->block) * (c->dim / 2);
    return {{span_of(c->K, ph, codes, codes, 1), span_of(c->V, ph, codes, codes, 1), span_of(c->Ks, ph, c->block, c->block, 2),
             span_of(c->Vs, ph, c->block, c->block, 2)}};
}

bool overlaps_kv4(Span x, const sgemm_kv4_cache *c)
{
    for (const Span &s : spans_of(c).s)
        if (overlap(x, s)) return true;
    return false;
}

// A rows x heads x dim operand (strides_ok), in bytes.
struct RowsOperand {
    const void *p;
    int rows, heads, dim, ld, hs, elem;
    Span span() const { return rows_span(p, rows, heads, dim, ld, hs, elem); }
    i64 bytes() const { return i64(dim) * elem; }  // of a row of one head
    i64 width() const { return heads > 1 ? i64(heads - 1) * hs * elem + bytes() : bytes(); }  // of a row
};

i64 floor_div(i64 a, i64 b) { return a / b - (a % b < 0 ? 1 : 0); }  // b > 0

// Whether pieces of `a` bytes at every multiple of pitch lie apart from pieces
// of `b` bytes at `at` and every multiple of pitch from there.
bool apart_in(i64 pitch, i64 a, i64 b, i64 at)
{
    at -= floor_div(at, pitch) * pitch;
    return at >= a && at + b <= pitch;
}

// Whether two operands of the same rows share a byte. Where the ranges that
// they span meet and their strides are the same (of one row or one head there
// is none), this is exact: rows and heads of the two may then be interleaved in
// any way (queries, keys and values of each row, or of each head, in one
// buffer). With other strides operands whose ranges meet count as sharing.
bool share(const RowsOperand &a, const RowsOperand &b)
{
    if (!overlap(a.span(), b.span())) return false;
    if (a.rows > 1 && i64(a.ld) * a.elem != i64(b.ld) * b.elem) return true;
    if (a.heads > 1 && b.heads > 1 && i64(a.hs) * a.elem != i64(b.hs) * b.elem) return true;
    const std::uintptr_t pa = reinterpret_cast<std::uintptr_t>(a.p), pb = reinterpret_cast<std::uintptr_t>(b.p);
    if ((pa <= pb ? pb - pa : pa - pb) >> 60) return true;
    const i64 pitch = a.rows > 1 ? i64(a.ld) * a.elem : 1, head = a.heads > 1 ? i64(a.hs) * a.elem : i64(b.hs) * b.elem;
    const i64 apart = pa <= pb ? i64(pb - pa) : -i64(pa - pb);
    // Side by side in each row, or in each head of each row: told without a walk over the heads.
    if (a.rows > 1 && apart_in(pitch, a.width(), b.width(), apart)) return false;
    if ((a.heads > 1 || b.heads > 1) && (a.rows == 1 || pitch % head == 0) && apart_in(head, a.bytes(), b.bytes(), apart)) return false;
    // A row of b's head h + dh begins at x + dr pitch, dr rows on, where one of a's head h begins at 0.
    for (i64 dh = 1 - a.heads; dh < b.heads; ++dh) {
        const i64 x = apart + dh * head;
        i64 first = -floor_div(x + b.bytes() - 1, pitch), last = floor_div(a.bytes() - 1 - x, pitch);  // of the rows that meet
        if (first < 1 - a.rows) first = 1 - a.rows;
        if (last > b.rows - 1) last = b.rows - 1;
        if (first <= last) return true;
    }
    return false;
}

}  // namespace

extern "C" int sgemm_kv4_check_args(const sgemm_kv4_cache *c, const sgemm_kv8_batch *b, int dtype, const void *K,
                                    int ldk, int hsk, const void *V, int ldv, int hsv)
{
    if (!known_type(dtype)) return SGEMM_ERR_DTYPE;
    const int rc = check_kv4(c, b);
    if (rc != SGEMM_OK) return rc;
    if (!strides_ok(b->rows, c->heads, c->dim, ldk, hsk) || !strides_ok(b->rows, c->heads, c->dim, ldv, hsv)) return SGEMM_ERR_LD;
    if (b->seqs == 0 || b->rows == 0) return SGEMM_OK;
    if (missing_arrays(c, b) || K == nullptr || V == nullptr) return SGEMM_ERR_NULL;
    const Span k = rows_span(K, b->rows, c->heads, c->dim, ldk, hsk, size_of(dtype));
    const Span v = rows_span(V, b->rows, c->heads, c->dim, ldv, hsv, size_of(dtype));
    if (overlaps_kv4(k, c) || overlaps_kv4(v, c)) return SGEMM_ERR_ALIAS;
    return SGEMM_OK;
}

extern "C" int sgemm_kv4_attend_check_args(const sgemm_kv4_cache *c, const sgemm_kv8_batch *b, int dtype, int heads_q,
                                           const void *Q, int ldq, int hsq, float scale, int causal, int window,
                                           const float *O, int ldo, int hso, const void *workspace,
                                           std::size_t workspace_bytes)
{
    (void)scale;
    if (!known_type(dtype)) return SGEMM_ERR_DTYPE;
    const int rc = check_kv4(c, b);
    if (rc != SGEMM_OK) return rc;
    if (heads_q < 1 || heads_q % c->heads != 0) return SGEMM_ERR_HEADS;
    if ((causal != 0 && causal != 1) || window < 0 || (window > 0 && causal == 0)) return SGEMM_ERR_MASK;
    if (!strides_ok(b->rows, heads_q, c->dim, ldq, hsq) || !strides_ok(b->rows, heads_q, c->dim, ldo, hso)) return SGEMM_ERR_LD;
    if (b->seqs == 0 || b->rows == 0) return SGEMM_OK;
    if (missing_arrays(c, b) || Q == nullptr || O == nullptr) return SGEMM_ERR_NULL;
    const Span o = rows_span(O, b->rows, heads_q, c->dim, ldo, hso, 4);
    const Span q = rows_span(Q, b->rows, heads_q, c->dim, ldq, hsq, size_of(dtype));
    if (overlap(o, q) || overlaps_kv4(o, c) || overlaps_batch(o, b)) return SGEMM_ERR_ALIAS;
    if (workspace != nullptr && workspace_bytes > 0) {
        const std::uintptr_t base = reinterpret_cast<std::uintptr_t>(workspace);
        const Span w{base, workspace_bytes > UINTPTR_MAX - base ? UINTPTR_MAX : base + workspace_bytes};
        if (overlap(w, o) || overlap(w, q) || overlaps_kv4(w, c) || overlaps_batch(w, b)) return SGEMM_ERR_ALIAS;
    }
    return SGEMM_OK;
}

extern "C" int sgemm_rope_check_args(int dtype, int otype, int rows, int dim, int rot, int interleaved, int inverse,
                                     float amplitude, const int *positions, const double *freqs,
                                     const sgemm_rope_rows *first, const sgemm_rope_rows *second)
{
    (void)amplitude;
    if (!known_type(dtype) || !known_type(otype)) return SGEMM_ERR_DTYPE;
    if (first == nullptr) return SGEMM_ERR_NULL;
    if (rows < 0 || dim < 1 || dim > kMostRopeDim || rot < 0 || rot > dim || rot % 2 != 0) return SGEMM_ERR_DIM;
    const sgemm_rope_rows *const all[] = {first, second};
    for (const sgemm_rope_rows *o : all)
        if (o != nullptr && (o->heads < 1 || o->heads > kMostHeads)) return SGEMM_ERR_DIM;
    if ((interleaved != 0 && interleaved != 1) || (inverse != 0 && inverse != 1)) return SGEMM_ERR_MASK;
    for (const sgemm_rope_rows *o : all)
        if (o != nullptr && (!strides_ok(rows, o->heads, dim, o->ldx, o->hsx) || !strides_ok(rows, o->heads, dim, o->ldy, o->hsy)))
            return SGEMM_ERR_LD;
    if (rows == 0) return SGEMM_OK;
    if (positions == nullptr || (freqs == nullptr && rot > 0)) return SGEMM_ERR_NULL;
    for (const sgemm_rope_rows *o : all)
        if (o != nullptr && (o->X == nullptr || o->Y == nullptr)) return SGEMM_ERR_NULL;
    for (int i = 0; i < 2; ++i) {
        const sgemm_rope_rows *const o = all[i];
        if (o == nullptr) continue;
        const RowsOperand y{o->Y, rows, o->heads, dim, o->ldy, o->hsy, size_of(otype)};
        if (overlap(y.span(), span_of(positions, 1, rows, rows, 4)) || overlap(y.span(), span_of(freqs, 1, rot / 2, rot / 2, 8)))
            return SGEMM_ERR_ALIAS;
        for (int j = 0; j < 2; ++j) {
            const sgemm_rope_rows *const a = all[j];
            if (a == nullptr) continue;
            const RowsOperand x{a->X, rows, a->heads, dim, a->ldx, a->hsx, size_of(dtype)};
            const bool in_place = i == j && o->Y == a->X && otype == dtype && (rows == 1 || o->ldy == a->ldx) &&
                                  (o->heads == 1 || o->hsy == a->hsx);
            if (!in_place && share(y, x)) return SGEMM_ERR_ALIAS;
            if (i < j && share(y, RowsOperand{a->Y, rows, a->heads, dim, a->ldy, a->hsy, size_of(otype)})) return SGEMM_ERR_ALIAS;
        }
    }
    return SGEMM_OK;
}

extern "C" int sgemm_kv_tables_check_args(const sgemm_kv_step *t)
{
    if (t == nullptr) return SGEMM_ERR_NULL;
    if (t->seqs < 0 || t->table_ld < 0 || t->pool_size < 0 || t->rows < 0) return SGEMM_ERR_DIM;
    if (t->block < 16 || t->block > 1024 || (t->block & (t->block - 1)) != 0) return SGEMM_ERR_CACHE;
    if (t->starts == nullptr || t->taken == nullptr || t->taken_after == nullptr ||
        (t->seqs > 0 && (t->lens == nullptr || t->news == nullptr || (t->table == nullptr && t->table_ld > 0))) ||
        (t->pool == nullptr && t->pool_size > 0) || (t->rows > 0 && (t->positions == nullptr || t->slots == nullptr)))
        return SGEMM_ERR_NULL;
    const Span out[] = {span_of(t->table, t->seqs, t->table_ld, t->table_ld, 4), span_of(t->starts, 1, i64(t->seqs) + 1, i64(t->seqs) + 1, 4),
                        span_of(t->positions, 1, t->rows, t->rows, 4), span_of(t->slots, 1, t->rows, t->rows, 8),
                        span_of(t->taken_after, 1, 1, 1, 4)};
    const Span in[] = {span_of(t->lens, 1, t->seqs, t->seqs, 4), span_of(t->news, 1, t->seqs, t->seqs, 4),
                       span_of(t->pool, 1, t->pool_size, t->pool_size, 4), span_of(t->taken, 1, 1, 1, 4)};
    for (int i = 0; i < 5; ++i) {
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return SGEMM_ERR_ALIAS;
        for (int j = 0; j < 4; ++j)
            if (overlap(out[i], in[j]) && !(i == 4 && j == 3 && t->taken == t->taken_after)) return SGEMM_ERR_ALIAS;
    }
    return SGEMM_OK;
}

namespace sgemm_impl {

bool kv4_write_overlaps(const sgemm_kv4_cache &c, const sgemm_kv8_batch &b)
{
    const CacheSpans own = spans_of(&c);
    for (int i = 0; i < 4; ++i) {
        if (overlaps_batch(own.s[i], &b)) return true;
        for (int j = 0; j < i; ++j)
            if (overlap(own.s[i], own.s[j])) return true;
    }
    return false;
}

bool kv4_read_overlaps(const sgemm_kv4_cache &c, const sgemm_kv8_batch &b, int dtype, const void *K, int ldk, int hsk,
                       const void *V, int ldv, int hsv)
{
    const RowsOperand k{K, b.rows, c.heads, c.dim, ldk, hsk, size_of(dtype)}, v{V, b.rows, c.heads, c.dim, ldv, hsv, size_of(dtype)};
    return share(k, v) || overlaps_batch(k.span(), &b) || overlaps_batch(v.span(), &b);
}

Kv4Plan plan_kv4_attend(const sgemm_kv4_cache &c, const sgemm_kv8_batch &b, int heads_q, int window, int cus)
{
    cus = cus <= 0 ? 256 : cus < 4096 ? cus : 4096;
    const i64 new_rows = b.max_new < b.rows ? b.max_new : b.rows, rows = at_least_1(new_rows * (heads_q / c.heads));
    const i64 heads = i64(b.seqs) * c.heads;  // of all sequences
    const auto tiles_of = [&](i64 tile) { return (rows + tile - 1) / tile; };
    // A launch covers at most 2^22 work-groups at once; kernels walk the rest.
    const i64 most = at_least_1((i64(1) << 22) / c.heads);
    const auto cut = [&](i64 tiles) { return int(tiles < most ? tiles : most); };

    Kv4Plan plan = {};
    plan.cus = cus;
    // Waves take row tiles of their own once that gives every compute unit a work-group.
    const int groups = c.dim > 128 ? 1 : 2;  // longer heads have no registers for two
    plan.rows = rows >= 64 * groups && (heads >= cus || tiles_of(64 * groups) * heads >= cus);
    if (plan.rows) {
        plan.copies = 1;
        plan.mt = groups;
        plan.tiles = cut(tiles_of(64 * groups));
        return plan;
    }
    // Else they share one group of 16. Two would halve the work on codes a row, but
    // leave registers for fewer waves: 32 sequences of 2000 tokens and 20 rows 45
    // us, with two 39, but in float32 47 and 52, and 64 of 200 and 100 rows 51 and 54.
    plan.mt = 1;
    plan.copies = rows <= 4 ? 4 : rows <= 8 ? 2 : 1;
    plan.tiles = cut(tiles_of(plan.tile_rows()));
    // As many work-groups as the compute units hold at once share the tokens of
    // all sequences, each with at least 256 of those that the longest sequences
    // can have, unless there are many times as many sequences and heads in any case.
    // (Three of them, or two with more than 8 rows of more than 64 components: 8
    // sequences of 4096 tokens and 16 rows 28 us, with three a unit 35.)
    const int resident = c.dim > 128 || (plan.copies == 1 && c.dim > 64) ? 2 : 3;
    const i64 units = i64(plan.tiles) * c.heads;
    if (b.seqs > kMostShared || units * b.seqs >= 4 * resident * i64(cus)) return plan;
    i64 tokens = i64(b.table_ld) * c.block;
    if (window > 0 && tokens > window + new_rows) tokens = window + new_rows;
    i64 slots = resident * i64(cus) / units, room = i64(b.seqs) * (tokens / (32 * kKv4LeastTurns));
    if (slots > room) slots = room;
    // 64 for each sequence at most, on average, as the join has to add what they leave:
    // 1 sequence of 131072 tokens and 1, 2, 4 and 8 cache heads 31, 32, 33 and 39 us,
    // with 192 at most 34, 37, 41 and 42, with all that fit 57, 51, 40 and 42.
    if (slots > kMostParts * i64(b.seqs)) slots = kMostParts * i64(b.seqs);
    if (slots <= b.seqs && room <= b.seqs) return plan;  // no sequence long enough to be shared
    if (slots < 1) return plan;
    // A whole number for each sequence, if that leaves out few: sequences of one
    // length then end where parts do (13 of 1023 tokens seen 23.5 us against 27.9).
    if (slots % b.seqs <= slots / 8) slots -= slots % b.seqs;
    plan.slots = int(slots);
    plan.parts = plan.slots + b.seqs;
    return plan;
}

}  // namespace sgemm_impl

extern "C" size_t sgemm_kv4_attend_workspace_size(const sgemm_kv4_cache *c, const sgemm_kv8_batch *b, int heads_q,
                                                  int window, int cus)
{
    if (check_kv4(c, b) != SGEMM_OK || heads_q < 1 || heads_q % c->heads != 0 || window < 0) return 0;
    if (b->seqs == 0 || b->rows == 0) return 0;
    const Kv4Plan plan = plan_kv4_attend(*c, *b, heads_q, window, cus);
    // For each row of each part: the sums of its components, and what the softmax
    // has of it. For each sequence: how it was shared out.
    const std::size_t units = std::size_t(c->heads) * std::size_t(plan.tiles);
    return units * (std::size_t(plan.parts) * std::size_t(plan.tile_rows()) * std::size_t(c->dim + 4) * 4 + std::size_t(plan.slots ? b->seqs : 0) * kKv4SplitBytes);
}

extern "C" int sgemm_kv4_attend_shape(const sgemm_kv4_cache *c, const sgemm_kv8_batch *b, int heads_q, int window, int cus,
                                      int *shape)
{
    const int rc = check_kv4(c, b);
    if (rc != SGEMM_OK) return rc;
    if (heads_q < 1 || heads_q % c->heads != 0) return SGEMM_ERR_HEADS;
    if (window < 0) return SGEMM_ERR_MASK;
    if (shape == nullptr) return SGEMM_ERR_NULL;
    const Kv4Plan plan = plan_kv4_attend(*c, *b, heads_q, window, cus);
    shape[0] = plan.tile_rows();
    shape[1] = plan.rows ? 4 : 1;
    shape[2] = plan.tiles;
    shape[3] = plan.slots;
    return SGEMM_OK;
}
