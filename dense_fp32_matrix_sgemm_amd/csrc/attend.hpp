// What attention over the 8-bit and the 4-bit cache share: exchanges between
// the lanes of a column, which tokens a row sees, and the join of split
// sequences.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "kv8.hpp"
#include "lowbit.hpp"

namespace sgemm_impl {
namespace {

constexpr int kAttendWaves = 4;
constexpr float kLog2e = 1.4426950408889634f;

// The larger (sum) of a value over the four lanes that hold one column.
__device__ inline float column_max(float x)
{
    const auto a = __builtin_amdgcn_permlane16_swap(f32_bits(x), f32_bits(x), false, false);
    const float y = __builtin_fmaxf(bits_f32(a[0]), bits_f32(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(f32_bits(y), f32_bits(y), false, false);
    return __builtin_fmaxf(bits_f32(b[0]), bits_f32(b[1]));
}
__device__ inline float column_sum(float x)
{
    const auto a = __builtin_amdgcn_permlane16_swap(f32_bits(x), f32_bits(x), false, false);
    const float y = bits_f32(a[0]) + bits_f32(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(f32_bits(y), f32_bits(y), false, false);
    return bits_f32(b[0]) + bits_f32(b[1]);
}

// An element that all lanes read, of an array that no kernel writes meanwhile:
// through the constant address space it becomes a scalar load, which no wait
// for a vector load holds up.
template <class V> __device__ inline V uniform_load(const V *p, std::int64_t i)
{
    return reinterpret_cast<const __attribute__((address_space(4))) V *>(reinterpret_cast<std::uintptr_t>(p))[i];
}

// Eight weights p * scale, p >= 0, as three bf16 parts that add up to them
// exactly (split3 without its care for infinities: a weight that is not
// finite makes its whole row NaN in any case).
__device__ inline void split_weights(const float *w, Frag &hi, Frag &mid, Frag &lo)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float h[2], m[2], l[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float x = w[2 * i + j];
            h[j] = bits_f32(f32_bits(x) & 0xffff0000u);
            const float r = x - h[j];
            m[j] = bits_f32(f32_bits(r) & 0xffff0000u);
            l[j] = r - m[j];
        }
        hi.v[i] = pack_hi(h[0], h[1]);
        mid.v[i] = pack_hi(m[0], m[1]);
        lo.v[i] = pack_hi(l[0], l[1]);
    }
}

// The factor that brings a sum with maximum m to maximum top.
__device__ inline float rescale(float m, float top) { return m == top ? 1.0f : __builtin_amdgcn_exp2f(m - top); }

// What the rows of one tile see: row `row` of a sequence (row / R th new row,
// query head row % R of the group) sees `count` tokens from `from` on, of
// those that the table can name (from + count <= nameable).
struct KvSeen {
    std::int64_t first, len, nameable;  // position of new row 0, tokens, tokens that the table can name
    int R, causal, window;
    // By the new row itself: where what it sees ends, what it sees, and whether
    // the last token seen lies behind the table's last column (the row is NaN).
    __device__ std::int64_t end_of(std::int64_t fresh) const { return causal ? first + fresh + 1 : len; }
    __device__ void by_new(std::int64_t fresh, int &from, int &count) const
    {
        const std::int64_t end = end_of(fresh), begin = window > 0 ? end - window : 0;
        const std::int64_t hi = end < 0 ? 0 : end < nameable ? end : nameable, lo = begin < 0 ? 0 : begin < hi ? begin : hi;
        from = int(lo);
        count = int(hi - lo);
    }
    __device__ bool beyond_new(std::int64_t fresh) const { return end_of(fresh) > nameable; }
    __device__ void operator()(std::int64_t row, int &from, int &count) const { by_new(row / R, from, count); }
    __device__ bool beyond(std::int64_t row) const { return beyond_new(row / R); }
};

// Adds the sums that the splits of a row tile left in the workspace, in their
// order: one wave for each row (32 sequences of 8192 tokens in 3 splits: 5 us,
// most of it the launch).
template <class Problem, int MT> __global__ __launch_bounds__(256) void kv_join_kernel(Problem p)
{
    constexpr int kRows = 16 * MT;
    const int lane = threadIdx.x & 63, R = p.heads_q / p.c.heads, dim = p.c.dim, splits = p.plan.splits;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const unsigned unit = blockIdx.x / (kRows / 4), i = blockIdx.x % (kRows / 4) * 4 + unsigned(wave);
    const int tile = int(unit % unsigned(p.plan.tiles)), head = int(unit / unsigned(p.plan.tiles) % unsigned(p.c.heads));
    const int seq = int(unit / unsigned(p.plan.tiles) / unsigned(p.c.heads));
    const Kv8Sequence s = kv8_sequence(p.b, seq);
    const std::int64_t row = std::int64_t(tile) * kRows + i;
    if (row >= s.n * R) return;
    const float *const part = p.ws + (std::int64_t(unit) * splits * kRows + i) * (dim + 4);
    const std::int64_t pitch = std::int64_t(kRows) * (dim + 4);
    // Lane x: split x's maximum and sum (at most 64 splits).
    float m = -__builtin_inff(), l = 0.0f;
    if (lane < splits) m = part[lane * pitch + dim], l = part[lane * pitch + dim + 1];
    float top = m;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, d));
    // A split that saw nothing of its row weighs nothing, and its components were left as sums of nothing: zeros.
    const float a = l == 0.0f ? 0.0f : rescale(m, top);
    float sum = l * a;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
    f32x4 y = {0, 0, 0, 0};
    const float *const at = part + (4 * lane < dim ? 4 * lane : 0);
    int x = 0;
    for (; x + 4 <= splits; x += 4) {
        f32x4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const f32x4 *>(at + (x + i) * pitch);
#pragma unroll
        for (int i = 0; i < 4; ++i) y += v[i] * __shfl(a, x + i);
    }
    for (; x < splits; ++x) y += *reinterpret_cast<const f32x4 *>(at + x * pitch) * __shfl(a, x);
    if (4 * lane >= dim) return;
    y = y / sum;
    const KvSeen seen{s.len - s.n, s.len, std::int64_t(p.b.table_ld) * p.c.block, R, p.causal, p.window};
    if (seen.beyond(row)) y = y * __builtin_nanf("");
    __builtin_memcpy(p.O + (s.row0 + row / R) * p.ldo + (head * R + row % R) * p.hso + 4 * lane, &y, sizeof(y));
}

}  // namespace
}  // namespace sgemm_impl
