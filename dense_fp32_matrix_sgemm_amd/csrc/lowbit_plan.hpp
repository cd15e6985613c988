// Host logic of the 8-bit cache's entry points. Pure C++ (no HIP header).
#pragma once

#include "sgemm.h"

namespace sgemm_impl {

// How attention is laid out over the device; from sizes the host knows
// (args_lowbit.cpp), so that the workspace's size needs no device.
struct Kv8Plan {
    int mt;        // groups of 16 rows a wave holds
    int rows;      // 1: a work-group's waves take row tiles of their own; 0: the tokens of one row tile
    int tiles;     // row tiles (of one wave, or four when rows) per sequence and head the grid covers at once
    int splits;    // work-groups that share a row tile's tokens
};
Kv8Plan plan_kv8_attend(const sgemm_kv8_cache &c, const sgemm_kv8_batch &b, int heads_q, int window, int cus);

// Whether the two outputs of sgemm_kv8_read overlap each other or the batch's
// arrays.
bool kv8_read_overlaps(const sgemm_kv8_cache &c, const sgemm_kv8_batch &b, int dtype, const void *K, int ldk, int hsk,
                       const void *V, int ldv, int hsv);

}  // namespace sgemm_impl
