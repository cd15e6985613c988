// Host logic of the entry points of a serving step: the 4-bit cache, rotary
// positions, page tables (args_step.cpp). Pure C++ (no HIP header).
#pragma once

#include <cstdint>

#include "lowbit_plan.hpp"
#include "sgemm.h"

namespace sgemm_impl {

// How attention over the 4-bit cache is laid out over the device; from sizes
// the host knows, so that the workspace's size needs no device.
struct Kv4Plan {
    int rows;    // 1: a work-group's waves take row tiles of their own; 0: the tokens of one row tile
    int mt;      // groups of 16 rows a wave holds (one but for row tiles of its own)
    int copies;  // how often the 16 columns of a group hold each row (4, 2 or 1)
    int tiles;   // row tiles (of one wave, or four when rows) per sequence and head the grid covers at once
    int slots;   // work-groups that share the tokens that a row tile of all sequences sees; 0: one for each sequence
    int parts;   // parts of sequences that they may leave in the workspace
    int cus;     // compute units
    int tile_rows() const { return 16 * mt / copies; }
};

// Turns of 32 tokens that a work-group which shares a tile's tokens has at
// least, on average.
constexpr int kKv4LeastTurns = 8;

// What the workspace holds of each sequence and row tile besides parts (Kv4Split).
constexpr int kKv4SplitBytes = 8;

// Sequences whose turns are shared out together at most: each work-group adds
// them all up.
constexpr int kMostShared = 1024;

// Work-groups that share the tokens of a tile's sequences at most, for each sequence.
constexpr int kMostParts = 64;

Kv4Plan plan_kv4_attend(const sgemm_kv4_cache &c, const sgemm_kv8_batch &b, int heads_q, int window, int cus);

// Whether sgemm_kv4_write's arrays overlap one another or the batch's.
bool kv4_write_overlaps(const sgemm_kv4_cache &c, const sgemm_kv8_batch &b);

// Whether the two outputs of sgemm_kv4_read share elements, or overlap the
// batch's arrays.
bool kv4_read_overlaps(const sgemm_kv4_cache &c, const sgemm_kv8_batch &b, int dtype, const void *K, int ldk, int hsk,
                       const void *V, int ldv, int hsv);

constexpr int kMostRopeDim = 1024;

// Bytes of an output (what the L2 of a die holds) from which on it is kept out
// of the caches, which else are still writing it when the next kernel starts. K
// and V of 6 MB each read back in bf16 with the write before: 18.4 us instead of
// 19.1, 24 MB 34.5 instead of 40.9; 100 MB of rows turned 48.9 instead of 53.0;
// under 4 MB no difference.
constexpr std::int64_t kStreamBytes = std::int64_t(4) << 20;

// Rows of sgemm_kv_tables that its first kernel, one work-group, places itself:
// 8 prompts of up to 512, 1024 and 2048 tokens 5.4, 7.0 and 10.4 us, where the
// second kernel makes it 7.2, 7.0 and 7.1 and a launch.
constexpr int kTablesAlone = 8192;

// The first of n ascending sums that is above x, or n.
template <class A> constexpr int above(const A &sums, int n, std::int64_t x)
{
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = lo + ((hi - lo) >> 1);
        if (std::int64_t(sums[mid]) > x) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// The sequence `step` behind seq (< seqs), or seqs where there is none.
constexpr int next_sequence(int seq, int step, int seqs) { return seq < seqs - step ? seq + step : seqs; }

}  // namespace sgemm_impl
