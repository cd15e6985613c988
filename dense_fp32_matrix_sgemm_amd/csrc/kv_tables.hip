// The tables of a step over a paged cache (sgemm_kv_tables): where each
// sequence's rows start, the pages that its new tokens take from the pool, and
// each row's position and place.
//
// All of it follows from two running sums over the sequences, of their new
// rows and of the pages that they take. One work-group walks the sequences
// 1024 at a time, a thread each, forms both sums side by side, and then turns
// its threads over to what the sums count: each page taken, and each row, finds
// its sequence in them by bisection, so that long and short sequences cost
// alike. A batch with one new token each is done with that one launch: 4.7 us for
// 64 sequences, three round trips (lengths, pool, stores) and four barriers. Over
// kTablesAlone rows, a second kernel over the whole device places the rows from
// the starts and the table: 8 prompts of up to 16384 tokens 4.9 us and 3.2, where
// the one work-group alone would take 60.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "gemm.hpp"
#include "step.hpp"

namespace sgemm_impl {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
typedef std::int64_t i64;

struct Sequence {
    int len, n, first, behind;  // tokens, new ones, first column to fill, first one behind
};

__device__ inline Sequence sequence_of(const sgemm_kv_step &t, int shift, int seq)
{
    const int len = t.lens[seq] < 0 ? 0 : t.lens[seq], fresh = t.news[seq];
    const int n = fresh < 0 ? 0 : fresh < len ? fresh : len, up = (1 << shift) - 1;
    auto pages = [&](int tokens) { return int((unsigned(tokens) + unsigned(up)) >> shift); };
    const int last = pages(len) < t.table_ld ? pages(len) : t.table_ld, first = pages(len - n);
    return {len, n, first, last > first ? last : first};
}

__device__ inline int capped(i64 x) { return x < INT32_MAX ? int(x) : INT32_MAX; }

__device__ inline i64 slot_of(i64 page, int position, int shift)
{
    return page < 0 ? -1 : (page << shift) + (position & ((1 << shift) - 1));
}

__global__ __launch_bounds__(kThreads) void kv_tables_kernel(sgemm_kv_step t, int place_rows)
{
    __shared__ i64 rows_to[kThreads], pages_to[kThreads], wave_rows[kWaves], wave_pages[kWaves];
    __shared__ Sequence held[kThreads];
    const int shift = 31 - __builtin_clz(unsigned(t.block)), lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const i64 taken = *t.taken;
    i64 rows = 0, pages = 0;  // of the sequences before
    auto page_at = [&](i64 k) {
        const i64 at = taken + k;
        return at >= 0 && at < t.pool_size ? t.pool[at] : -1;
    };
    if (threadIdx.x == 0) t.starts[0] = 0;
    for (i64 seq0 = 0; seq0 < t.seqs; seq0 += kThreads) {
        const int count = t.seqs - seq0 < kThreads ? int(t.seqs - seq0) : kThreads;
        Sequence s = {0, 0, 0, 0};
        if (int(threadIdx.x) < count) s = sequence_of(t, shift, int(seq0) + int(threadIdx.x));
        i64 a = s.n, b = s.behind - s.first;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const i64 x = __shfl_up(a, d), y = __shfl_up(b, d);
            if (lane >= d) a += x, b += y;
        }
        if (lane == 63) wave_rows[wave] = a, wave_pages[wave] = b;
        __syncthreads();
        for (int w = 0; w < wave; ++w) a += wave_rows[w], b += wave_pages[w];
        rows_to[threadIdx.x] = a;
        pages_to[threadIdx.x] = b;
        held[threadIdx.x] = s;
        if (int(threadIdx.x) < count) t.starts[seq0 + threadIdx.x + 1] = capped(rows + a);
        __syncthreads();
        const i64 more_rows = rows_to[kThreads - 1], more_pages = pages_to[kThreads - 1];
        for (i64 k = threadIdx.x; k < more_pages; k += kThreads) {
            const int b0 = above(pages_to, count, k);
            const i64 column = held[b0].behind - (pages_to[b0] - k);
            t.table[(seq0 + b0) * t.table_ld + column] = page_at(pages + k);
        }
        if (place_rows) {
            for (i64 r = threadIdx.x; r < more_rows && rows + r < t.rows; r += kThreads) {
                const int b0 = above(rows_to, count, r);
                const Sequence &q = held[b0];
                const int position = q.len - int(rows_to[b0] - r), column = position >> shift;
                // A column that this call fills is not read back: its page comes from the pool.
                i64 page = -1;
                if (column < q.first) page = column < t.table_ld ? t.table[(seq0 + b0) * t.table_ld + column] : -1;
                else if (column < q.behind) page = page_at(pages + pages_to[b0] - (q.behind - column));
                t.positions[rows + r] = position;
                t.slots[rows + r] = slot_of(page, position, shift);
            }
        }
        rows += more_rows;
        pages += more_pages;
        __syncthreads();  // the sums are no longer read
    }
    if (threadIdx.x == 0) *t.taken_after = capped(taken + pages);
}

// Positions and places of the rows, from the starts and the table that the
// first kernel left.
__global__ __launch_bounds__(256) void kv_rows_kernel(sgemm_kv_step t)
{
    const int shift = 31 - __builtin_clz(unsigned(t.block));
    for (i64 r = i64(blockIdx.x) * 256 + threadIdx.x; r < t.rows; r += i64(gridDim.x) * 256) {
        const int seq = above(t.starts + 1, t.seqs, r);
        if (seq >= t.seqs) return;  // behind the last row, and so are the rows to come
        const Sequence s = sequence_of(t, shift, seq);
        const int position = s.len - s.n + int(r - t.starts[seq]), column = position >> shift;
        const i64 page = column < t.table_ld ? t.table[i64(seq) * t.table_ld + column] : -1;
        t.positions[r] = position;
        t.slots[r] = slot_of(page, position, shift);
    }
}

}  // namespace

hipError_t launch_kv_tables(const sgemm_kv_step &t, hipStream_t stream)
{
    sgemm_kv_step q = t;
    int place_rows = t.rows <= kTablesAlone ? 1 : 0;
    void *args[] = {&q, &place_rows};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void *>(&kv_tables_kernel), dim3(1), dim3(kThreads), args, 0, stream);
    if (e != hipSuccess || place_rows || t.seqs == 0) return e;
    const i64 groups = (i64(t.rows) + 255) / 256;
    void *more[] = {&q};
    return hipLaunchKernel(reinterpret_cast<const void *>(&kv_rows_kernel), dim3(unsigned(groups < 8192 ? groups : 8192)), dim3(256), more, 0, stream);
}

}  // namespace sgemm_impl
