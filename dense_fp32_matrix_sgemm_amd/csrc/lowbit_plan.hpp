// Host logic of the 8-bit cache's entry points. Pure C++ (no HIP header).
#pragma once

#include "sgemm.h"

namespace sgemm_impl {

// How sgemm_w4 is laid out over the device (args_lowbit.cpp).
struct W4Plan {
    int few;     // 1: the kernel for few rows (16 rows by 16 wn columns a work-group); 0: the tile kernel
    int mt, nt;  // tile kernel: a wave's tile is 32 mt rows by 32 nt columns
    int wn, wk;  // waves of a work-group along N and along K
    int slabs;   // few rows: runs of K whose A is held in LDS one after the other; 0: A goes straight to registers
    int pitch;   // few rows: bytes from one held row to the next
    int held;    // few rows: bytes of LDS for them
};
W4Plan plan_w4(int dtype, int M, int N, int K, int cus);

// k that a wave of the kernel for few rows takes at a time, and its waves at most.
constexpr int w4_step(bool f32) { return f32 ? 128 : 256; }
constexpr int kRowsWaves = 16;

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

// Whether the cache's arrays overlap one another or the batch's: two writers,
// or a table that changes while it is read.
bool kv8_write_overlaps(const sgemm_kv8_cache &c, const sgemm_kv8_batch &b);

}  // namespace sgemm_impl
