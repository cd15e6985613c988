// Host-side argument checks of the products whose stored operand is held in
// few bits, and how products and attention are laid out over the device.
//
// Pure C++: no HIP header and no device call, like args.cpp.
#include <cstddef>
#include <cstdint>

#include "args_util.hpp"
#include "lowbit_plan.hpp"
#include "sgemm.h"

using namespace sgemm_impl;

namespace {

i64 groups_of(int K, int group) { return (i64(K) + group - 1) / group; }

// A limit that keeps the kernels' indexes (k + a few hundred) in 32 bits.
constexpr int kMostK = 1 << 30;

int check_group(int group) { return group <= 0 || group % 32 != 0 ? SGEMM_ERR_GROUP : SGEMM_OK; }

// Leading dimensions of the W4 form itself.
bool w4_ld_ok(int K, int group, int ldw, int lds, const void *Z, int ldz)
{
    const i64 g = at_least_1(groups_of(K, group));
    return ldw >= at_least_1((i64(K) + 1) / 2) && lds >= g && (Z == nullptr || ldz >= g);
}

bool overlaps_cache(Span x, const sgemm_kv8_cache *c)
{
    const i64 ph = i64(c->pages) * c->heads, codes = i64(c->block) * c->dim;
    return overlap(x, span_of(c->K, ph, codes, codes, 1)) || overlap(x, span_of(c->V, ph, codes, codes, 1)) ||
           overlap(x, span_of(c->Ks, 1, ph, ph, 4)) || overlap(x, span_of(c->Vs, 1, ph, ph, 4));
}

}  // namespace

extern "C" int sgemm_w4_check_args(int dtype, int stype, int M, int N, int K, int group, float alpha, const void *A,
                                   int lda, const unsigned char *W, int ldw, const void *S, int lds,
                                   const unsigned char *Z, int ldz, float beta, const float *C, int ldc)
{
    (void)beta;
    if (!known_type(dtype) || !known_type(stype)) return SGEMM_ERR_DTYPE;
    if (M < 0 || N < 0 || K < 0 || K > kMostK) return SGEMM_ERR_DIM;
    if (check_group(group) != SGEMM_OK) return SGEMM_ERR_GROUP;
    if (lda < at_least_1(K) || !w4_ld_ok(K, group, ldw, lds, Z, ldz) || ldc < at_least_1(N)) return SGEMM_ERR_LD;
    if (M == 0 || N == 0) return SGEMM_OK;
    if (C == nullptr) return SGEMM_ERR_NULL;
    if (K > 0 && alpha != 0.0f) {
        if (A == nullptr || W == nullptr || S == nullptr) return SGEMM_ERR_NULL;
        const Span c = span_of(C, M, N, ldc, 4);
        const i64 g = groups_of(K, group);
        if (overlap(c, span_of(A, M, K, lda, size_of(dtype))) || overlap(c, span_of(W, N, (i64(K) + 1) / 2, ldw, 1)) ||
            overlap(c, span_of(S, N, g, lds, size_of(stype))) || overlap(c, span_of(Z, N, g, ldz, 1)))
            return SGEMM_ERR_ALIAS;
    }
    return SGEMM_OK;
}

extern "C" int sgemm_w4_pack_check_args(int dtype, int stype, int N, int K, int group, const void *B, int ldb,
                                        const unsigned char *W, int ldw, const void *S, int lds,
                                        const unsigned char *Z, int ldz)
{
    if (!known_type(dtype) || !known_type(stype)) return SGEMM_ERR_DTYPE;
    if (N < 0 || K < 0 || K > kMostK) return SGEMM_ERR_DIM;
    if (check_group(group) != SGEMM_OK) return SGEMM_ERR_GROUP;
    if (ldb < at_least_1(K) || !w4_ld_ok(K, group, ldw, lds, Z, ldz)) return SGEMM_ERR_LD;
    if (N == 0 || K == 0) return SGEMM_OK;
    if (B == nullptr || W == nullptr || S == nullptr) return SGEMM_ERR_NULL;
    const i64 g = groups_of(K, group);
    const Span spans[] = {span_of(B, N, K, ldb, size_of(dtype)), span_of(W, N, (i64(K) + 1) / 2, ldw, 1),
                          span_of(S, N, g, lds, size_of(stype)), span_of(Z, N, g, ldz, 1)};
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < i; ++j)
            if (overlap(spans[i], spans[j])) return SGEMM_ERR_ALIAS;
    return SGEMM_OK;
}

extern "C" int sgemm_kv8_check_args(const sgemm_kv8_cache *c, const sgemm_kv8_batch *b, int dtype, const void *K,
                                    int ldk, int hsk, const void *V, int ldv, int hsv)
{
    if (!known_type(dtype)) return SGEMM_ERR_DTYPE;
    const int rc = check_cache_batch(c, b);
    if (rc != SGEMM_OK) return rc;
    if (!strides_ok(b->rows, c->heads, c->dim, ldk, hsk) || !strides_ok(b->rows, c->heads, c->dim, ldv, hsv)) return SGEMM_ERR_LD;
    if (b->seqs == 0 || b->rows == 0) return SGEMM_OK;
    if (missing_arrays(c, b) || K == nullptr || V == nullptr) return SGEMM_ERR_NULL;
    const Span k = rows_span(K, b->rows, c->heads, c->dim, ldk, hsk, size_of(dtype));
    const Span v = rows_span(V, b->rows, c->heads, c->dim, ldv, hsv, size_of(dtype));
    if (overlaps_cache(k, c) || overlaps_cache(v, c)) return SGEMM_ERR_ALIAS;
    return SGEMM_OK;
}

extern "C" int sgemm_kv8_attend_check_args(const sgemm_kv8_cache *c, const sgemm_kv8_batch *b, int dtype, int heads_q,
                                           const void *Q, int ldq, int hsq, float scale, int causal, int window,
                                           const float *O, int ldo, int hso, const void *workspace,
                                           std::size_t workspace_bytes)
{
    (void)scale;
    if (!known_type(dtype)) return SGEMM_ERR_DTYPE;
    const int rc = check_cache_batch(c, b);
    if (rc != SGEMM_OK) return rc;
    if (heads_q < 1 || heads_q % c->heads != 0) return SGEMM_ERR_HEADS;
    if ((causal != 0 && causal != 1) || window < 0 || (window > 0 && causal == 0)) return SGEMM_ERR_MASK;
    if (!strides_ok(b->rows, heads_q, c->dim, ldq, hsq) || !strides_ok(b->rows, heads_q, c->dim, ldo, hso)) return SGEMM_ERR_LD;
    if (b->seqs == 0 || b->rows == 0) return SGEMM_OK;
    if (missing_arrays(c, b) || Q == nullptr || O == nullptr) return SGEMM_ERR_NULL;
    const Span o = rows_span(O, b->rows, heads_q, c->dim, ldo, hso, 4);
    const Span q = rows_span(Q, b->rows, heads_q, c->dim, ldq, hsq, size_of(dtype));
    if (overlap(o, q) || overlaps_cache(o, c) || overlaps_batch(o, b)) return SGEMM_ERR_ALIAS;
    if (workspace != nullptr && workspace_bytes > 0) {
        const std::uintptr_t base = reinterpret_cast<std::uintptr_t>(workspace);
        const Span w{base, workspace_bytes > UINTPTR_MAX - base ? UINTPTR_MAX : base + workspace_bytes};
        if (overlap(w, o) || overlap(w, q) || overlaps_cache(w, c) || overlaps_batch(w, b)) return SGEMM_ERR_ALIAS;
    }
    return SGEMM_OK;
}

namespace sgemm_impl {

bool kv8_read_overlaps(const sgemm_kv8_cache &c, const sgemm_kv8_batch &b, int dtype, const void *K, int ldk, int hsk,
                       const void *V, int ldv, int hsv)
{
    const Span k = rows_span(K, b.rows, c.heads, c.dim, ldk, hsk, size_of(dtype));
    const Span v = rows_span(V, b.rows, c.heads, c.dim, ldv, hsv, size_of(dtype));
    return overlap(k, v) || overlaps_batch(k, &b) || overlaps_batch(v, &b);
}

bool kv8_write_overlaps(const sgemm_kv8_cache &c, const sgemm_kv8_batch &b)
{
    const i64 ph = i64(c.pages) * c.heads, codes = i64(c.block) * c.dim;
    const Span own[] = {span_of(c.K, ph, codes, codes, 1), span_of(c.V, ph, codes, codes, 1), span_of(c.Ks, 1, ph, ph, 4),
                        span_of(c.Vs, 1, ph, ph, 4)};
    for (int i = 0; i < 4; ++i) {
        if (overlaps_batch(own[i], &b)) return true;
        for (int j = 0; j < i; ++j)
            if (overlap(own[i], own[j])) return true;
    }
    return false;
}

W4Plan plan_w4(int dtype, int M, int N, int K, int cus)
{
    cus = cus <= 0 ? 256 : cus;
    const bool f32 = dtype == SGEMM_F32;
    W4Plan plan = {};
    // Up to 8 rows (16 in float32, whose parts fill the tile kernel's LDS) the
    // rows kernel is faster: bf16, 8 rows by 8192 x 8192 16.2 us against 17.2,
    // 4096 x 4096 8.0 against 9.0, 16384 x 4096 14.1 against 18.4; float32, 16
    // rows 32.1 against 40.5, 13.2 against 21.0, 24.0 against 40.6. From 9 to
    // 16 bf16 rows it depends on the width: 16 rows by 8192 x 8192 21.2 against
    // 18.3, 4096 x 4096 9.9 against 9.2, but 16384 x 4096 16.8 against 18.8.
    if (M > (f32 ? 16 : 8)) {
        // The largest tile that still gives every compute unit one; with fewer
        // tiles the waves divide K. float32 rows take three times the LDS.
        const auto tiles = [&](int bm, int bn) { return (i64(M) + bm - 1) / bm * ((i64(N) + bn - 1) / bn); };
        if (tiles(64, 256) >= cus) {
            plan.mt = 2, plan.nt = 2, plan.wn = 4, plan.wk = 1;
        } else if (f32) {
            plan.mt = 1, plan.nt = 1, plan.wn = 1, plan.wk = 4;
        } else if (tiles(64, 64) >= 2 * i64(cus)) {
            plan.mt = 2, plan.nt = 2, plan.wn = 1, plan.wk = 4;
        } else {
            plan.mt = M > 32 ? 2 : 1, plan.nt = 1, plan.wn = 1, plan.wk = 8;
        }
        return plan;
    }
    plan.few = 1;
    constexpr i64 kLds = 160 * 1024;
    // Waves along K while there are too few columns to fill the device.
    const i64 tiles_n = (i64(N) + 15) / 16;
    plan.wn = 1;
    while (plan.wn < 4 && tiles_n >= 2 * plan.wn * i64(cus)) plan.wn *= 2;
    // K in as few slabs as the LDS holds, of even length, each with a whole
    // step for every wave. (A slab of one step and the rest always fits: 16
    // float32 rows take 25 KB of it.)
    const int step = w4_step(f32), steps = K / step, rest = K % step;
    const auto pitch = [&](i64 slab_steps) { return (2 * (slab_steps * step + (rest + 31) / 32 * 32) + 127) / 128 * 128 + 16; };
    const auto held = [&](i64 slab_steps) { return (f32 ? 3 : 1) * M * pitch(slab_steps); };  // bytes
    // A that does not fit at once goes straight to registers while there is at
    // most one column tile for each compute unit: 16 rows of float32 by 4096
    // columns, K = 4096, 13.5 us against 17.8, by 1024, K = 16384, 38.8 against
    // 54.9, but by 8192, K = 8192, 41.8 against 32.8.
    if (held(steps) > kLds && tiles_n <= cus) {
        plan.slabs = 0;
    } else {
        plan.slabs = 1;
        const auto longest = [&] { return (i64(steps) + plan.slabs - 1) / plan.slabs; };
        while (plan.slabs < steps && held(longest()) > kLds) ++plan.slabs;
        plan.pitch = int(pitch(longest()));
        plan.held = int(held(longest()));
    }
    plan.wk = 1;
    while (2 * plan.wk * plan.wn <= kRowsWaves && 2 * plan.wk <= steps / (plan.slabs ? plan.slabs : 1)) plan.wk *= 2;
    return plan;
}

Kv8Plan plan_kv8_attend(const sgemm_kv8_cache &c, const sgemm_kv8_batch &b, int heads_q, int window, int cus)
{
    cus = cus <= 0 ? 256 : cus < 4096 ? cus : 4096;
    const i64 new_rows = b.max_new < b.rows ? b.max_new : b.rows, rows = at_least_1(new_rows * (heads_q / c.heads));
    const i64 heads = i64(b.seqs) * c.heads;  // of all sequences
    const auto tiles_of = [&](i64 tile) { return (rows + tile - 1) / tile; };
    // A launch covers at most 2^22 work-groups at once; kernels walk the rest.
    const i64 most = at_least_1((i64(1) << 22) / c.heads);
    const auto cut = [&](i64 tiles) { return int(tiles < most ? tiles : most); };

    Kv8Plan plan;
    plan.splits = 1;
    // Waves take row tiles of their own once that gives every compute unit a work-group
    // (8 sequences of 64 rows behind 2048 tokens, at half of that: 118 us against 66).
    const int most_mt = c.dim > 128 ? 1 : 2;  // longer heads have no registers for two
    plan.rows = rows >= 64 * most_mt && (heads >= cus || tiles_of(64 * most_mt) * heads >= cus);
    plan.mt = plan.rows || rows > 16 ? most_mt : 1;
    if (plan.rows) {
        plan.tiles = cut(tiles_of(64 * most_mt));
        return plan;
    }
    plan.tiles = cut(tiles_of(16 * plan.mt));
    // Else as many work-groups as the compute units hold at once (their
    // registers allow 4, 3 or 1 by the head's length: 32 sequences of 8192
    // tokens and 128 components in 3 splits 92 us, in 4 104), each with at
    // least 256 of the tokens that the longest sequence can have.
    const int resident = c.dim <= 64 ? 4 : c.dim <= 128 ? 3 : 1;
    const i64 units = heads < 8 * i64(cus) ? heads * plan.tiles : heads;
    i64 tokens = i64(b.table_ld) * c.block;
    if (window > 0 && tokens > window + new_rows) tokens = window + new_rows;
    i64 splits = units > 0 ? (resident * i64(cus) + units - 1) / units : 1;
    if (splits > tokens / 256) splits = tokens / 256;
    if (splits > 64) splits = 64;
    plan.splits = int(splits < 1 ? 1 : splits);
    return plan;
}

}  // namespace sgemm_impl

extern "C" size_t sgemm_kv8_attend_workspace_size(const sgemm_kv8_cache *c, const sgemm_kv8_batch *b, int heads_q,
                                                  int window, int cus)
{
    if (check_cache_batch(c, b) != SGEMM_OK || heads_q < 1 || heads_q % c->heads != 0 || window < 0) return 0;
    if (b->seqs == 0 || b->rows == 0) return 0;
    const sgemm_impl::Kv8Plan plan = sgemm_impl::plan_kv8_attend(*c, *b, heads_q, window, cus);
    if (plan.splits == 1) return 0;
    // For each row of each split: the sums of its components, maximum and sum of the softmax.
    return std::size_t(b->seqs) * std::size_t(c->heads) * std::size_t(plan.tiles) * std::size_t(plan.splits) * std::size_t(16 * plan.mt) *
           std::size_t(c->dim + 4) * 4;
}

extern "C" int sgemm_w4_shape(int dtype, int M, int N, int K, int cus, int *shape)
{
    if (!known_type(dtype)) return SGEMM_ERR_DTYPE;
    if (M < 0 || N < 0 || K < 0 || K > kMostK) return SGEMM_ERR_DIM;
    if (shape == nullptr) return SGEMM_ERR_NULL;
    const sgemm_impl::W4Plan plan = sgemm_impl::plan_w4(dtype, M, N, K, cus);
    shape[0] = plan.few ? 16 : 32 * plan.mt;
    shape[1] = plan.few ? 16 * plan.wn : 32 * plan.nt * plan.wn;
    shape[2] = plan.wn;
    shape[3] = plan.wk;
    shape[4] = plan.few ? plan.slabs : 1;
    return SGEMM_OK;
}

extern "C" int sgemm_kv8_attend_shape(const sgemm_kv8_cache *c, const sgemm_kv8_batch *b, int heads_q, int window, int cus,
                                      int *shape)
{
    const int rc = check_cache_batch(c, b);
    if (rc != SGEMM_OK) return rc;
    if (heads_q < 1 || heads_q % c->heads != 0) return SGEMM_ERR_HEADS;
    if (window < 0) return SGEMM_ERR_MASK;
    if (shape == nullptr) return SGEMM_ERR_NULL;
    const sgemm_impl::Kv8Plan plan = sgemm_impl::plan_kv8_attend(*c, *b, heads_q, window, cus);
    shape[0] = 16 * plan.mt;
    shape[1] = plan.rows ? 4 : 1;
    shape[2] = plan.tiles;
    shape[3] = plan.splits;
    return SGEMM_OK;
}
