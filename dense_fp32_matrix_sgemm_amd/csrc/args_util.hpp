// What the host-side argument checks share (args_lowbit.cpp, args_step.cpp).
// Pure C++ (no HIP header).
#pragma once

#include <cstddef>
#include <cstdint>

#include "sgemm.h"

namespace sgemm_impl {

typedef std::int64_t i64;

inline bool known_type(int t) { return t == SGEMM_F32 || t == SGEMM_LP_BF16 || t == SGEMM_LP_F16; }

inline int size_of(int t) { return t == SGEMM_F32 ? 4 : 2; }

inline i64 at_least_1(i64 x) { return x > 1 ? x : 1; }

// Byte range of a rows x cols row-major extent with row stride ld (elements).
struct Span {
    std::uintptr_t lo, hi;
};

inline Span span_of(const void *p, i64 rows, i64 cols, i64 ld, i64 elem)
{
    const std::uintptr_t base = reinterpret_cast<std::uintptr_t>(p);
    if (p == nullptr || rows <= 0 || cols <= 0) return {base, base};
    const unsigned __int128 bytes =
        (static_cast<unsigned __int128>(rows - 1) * static_cast<unsigned __int128>(ld) + static_cast<unsigned __int128>(cols)) *
        static_cast<unsigned __int128>(elem);
    const std::uintptr_t room = UINTPTR_MAX - base;
    return {base, bytes > room ? UINTPTR_MAX : base + static_cast<std::uintptr_t>(bytes)};
}

inline bool overlap(Span a, Span b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }

// Heads of a cache at most: a limit that keeps the work-items of a launch in
// 32 bits.
constexpr int kMostHeads = 1 << 16;

inline bool aligned16(const void *p) { return reinterpret_cast<std::uintptr_t>(p) % 16 == 0; }

// A cache of keys and values (sgemm_kv8_cache, sgemm_kv4_cache) and the
// sequences of a call.
template <class Cache> int check_cache_batch(const Cache *c, const sgemm_kv8_batch *b)
{
    if (c == nullptr || b == nullptr) return SGEMM_ERR_NULL;
    if (c->pages < 1 || c->heads < 1 || c->heads > kMostHeads || b->seqs < 0 || b->table_ld < 0 || b->rows < 0 || b->max_new < 0) return SGEMM_ERR_DIM;
    const bool power = c->block >= 16 && c->block <= 1024 && (c->block & (c->block - 1)) == 0;
    if (!power || c->dim < 16 || c->dim > 256 || c->dim % 16 != 0) return SGEMM_ERR_CACHE;
    if (!aligned16(c->K) || !aligned16(c->V)) return SGEMM_ERR_CACHE;
    return SGEMM_OK;
}

// A rows x heads x dim operand whose rows lie apart (heads inside a row) or
// whose heads do (rows inside a head); one row or one head needs no stride.
inline bool strides_ok(int rows, int heads, int dim, int ld, int hs)
{
    if (rows == 0) return true;
    if (rows == 1) return heads == 1 || hs >= dim;
    if (heads == 1) return ld >= dim;
    return (hs >= dim && ld >= i64(heads - 1) * hs + dim) || (ld >= dim && hs >= i64(rows - 1) * ld + dim);
}

inline Span rows_span(const void *p, int rows, int heads, int dim, int ld, int hs, int elem)
{
    const i64 last = (rows > 1 ? i64(rows - 1) * ld : 0) + (heads > 1 ? i64(heads - 1) * hs : 0) + dim;
    return span_of(p, 1, last, last, elem);
}

template <class Cache> bool missing_arrays(const Cache *c, const sgemm_kv8_batch *b)
{
    return c->K == nullptr || c->V == nullptr || c->Ks == nullptr || c->Vs == nullptr || b->lens == nullptr ||
           b->starts == nullptr || (b->table == nullptr && b->table_ld > 0);
}

inline bool overlaps_batch(Span x, const sgemm_kv8_batch *b)
{
    return overlap(x, span_of(b->table, b->seqs, b->table_ld, b->table_ld, 4)) || overlap(x, span_of(b->lens, 1, b->seqs, b->seqs, 4)) ||
           overlap(x, span_of(b->starts, 1, i64(b->seqs) + 1, i64(b->seqs) + 1, 4));
}

}  // namespace sgemm_impl
