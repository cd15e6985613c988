// Host logic of the entry points of a serving step: the 4-bit cache, rotary
// positions, page tables (args_step.cpp). Pure C++ (no HIP header).
#pragma once

#include "lowbit_plan.hpp"
#include "sgemm.h"

namespace sgemm_impl {

// How attention over the 4-bit cache is laid out, as for the 8-bit one.
Kv8Plan plan_kv4_attend(const sgemm_kv4_cache &c, const sgemm_kv8_batch &b, int heads_q, int window, int cus);

// Whether sgemm_kv4_write's arrays overlap one another or the batch's.
bool kv4_write_overlaps(const sgemm_kv4_cache &c, const sgemm_kv8_batch &b);

// Whether the two outputs of sgemm_kv4_read share elements, or overlap the
// batch's arrays.
bool kv4_read_overlaps(const sgemm_kv4_cache &c, const sgemm_kv8_batch &b, int dtype, const void *K, int ldk, int hsk,
                       const void *V, int ldv, int hsv);

constexpr int kMostRopeDim = 1024;

// Rows of sgemm_kv_tables that its first kernel, one work-group, places
// itself.
constexpr int kTablesAlone = 16384;

}  // namespace sgemm_impl
