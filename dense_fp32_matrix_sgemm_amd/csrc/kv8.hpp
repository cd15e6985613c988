// What the 8-bit cache's kernels read of the device's arrays, made safe: the
// host has seen none of it.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "sgemm.h"

namespace sgemm_impl {

// Sequence `seq` of a batch: its tokens, its rows of the operand and where
// they start. Row i stands at position len - n + i.
struct Kv8Sequence {
    int seq;
    std::int64_t len, n, row0;
};

__device__ inline Kv8Sequence kv8_sequence(const sgemm_kv8_batch &b, int seq)
{
    auto cut = [&](int row) { return std::int64_t(row < 0 ? 0 : row < b.rows ? row : b.rows); };
    const std::int64_t row0 = cut(b.starts[seq]), end = cut(b.starts[seq + 1]);
    const int len = b.lens[seq];
    return {seq, len > 0 ? len : 0, end > row0 ? end - row0 : 0, row0};
}

// The cache's page that holds page `page` of a sequence, or -1 where the
// table has no such column or names no page of the cache.
__device__ inline std::int64_t kv8_page(const sgemm_kv8_cache &c, const sgemm_kv8_batch &b, int seq, std::int64_t page)
{
    if (page >= b.table_ld) return -1;
    const int id = b.table[std::int64_t(seq) * b.table_ld + page];
    return id >= 0 && id < c.pages ? id : -1;
}

}  // namespace sgemm_impl
