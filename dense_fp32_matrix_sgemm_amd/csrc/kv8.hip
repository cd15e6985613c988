// The 8-bit cache of keys and values: quantising new rows into its pages
// (sgemm_kv8_write) and reading rows back (sgemm_kv8_read).
//
// A page and head share one scale, a power of two: e4m3 is a floating format,
// so the choice of power costs no precision but at its subnormal end, dividing
// by it is exact, and a page whose scale rises while it fills keeps its older
// codes' values exactly (again but for subnormals), however often it rises.
//
// Work is laid out by what shares a scale: one work-group for each sequence,
// page that the sequence's rows reach, head, and K or V. It alone reads and
// writes that scale and those codes, so nothing is atomic and the result does
// not depend on timing. Rows come in once (what does not stay in registers
// until the maximum is known is read again, from the caches). 4 prompts of up
// to 4096 rows in bf16 (11674 rows, 72 MB): reading back 15.3 us, 4.7 TB/s,
// bound by memory; writing 18.9 us, 3.8 TB/s: a work-group's loads and stores
// lie on either side of a barrier and its vector instructions take over half
// of the time. 64 sequences of one new token each: 6.5, round trips, and their
// last tokens read back in float32 17.5 to 18.8.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "gemm.hpp"
#include "kv8.hpp"
#include "lowbit.hpp"

namespace sgemm_impl {
namespace {

constexpr int kThreads = 256;

// Pages that n rows reach at most.
std::int64_t pages_reached(std::int64_t n, int block) { return n < 1 ? 1 : (n + block - 2) / block + 1; }

struct Grid {
    unsigned pieces, seqs;  // pages of a sequence, and sequences, that the launch covers at once
};

// Work-groups: sequences x pieces (pages) x heads x {K, V}; kernels walk the
// pages and sequences beyond.
Grid grid_of(const Kv8Problem &p)
{
    const std::int64_t n = p.b.max_new < p.b.rows ? p.b.max_new : p.b.rows, most = std::int64_t(1) << 23;
    const std::int64_t heads = 2 * std::int64_t(p.c.heads);
    std::int64_t pieces = pages_reached(n, p.c.block), room = most / heads;
    room = room < 1 ? 1 : room;
    if (pieces > room) pieces = room;
    std::int64_t seqs = most / (pieces * heads);
    seqs = seqs < 1 ? 1 : seqs < p.b.seqs ? seqs : p.b.seqs;
    return {unsigned(pieces), unsigned(seqs)};
}

// One work-group's share: rows of one sequence in one page, for one head of K
// or V.
struct Piece {
    int head, kv;
    Kv8Sequence s;
    std::int64_t page;  // within the sequence
};

// Calls body(piece) for every piece that falls to this work-group.
template <class Body> __device__ inline void for_each_piece(const Kv8Problem &p, const Grid &g, Body &&body)
{
    unsigned id = blockIdx.x;
    Piece w;
    w.kv = int(id & 1);
    id >>= 1;
    w.head = int(id % unsigned(p.c.heads));
    id /= unsigned(p.c.heads);
    const unsigned first = id % g.pieces;
    const int shift = 31 - __builtin_clz(unsigned(p.c.block));
    for (unsigned seq = id / g.pieces; seq < unsigned(p.b.seqs); seq += g.seqs) {
        w.s = kv8_sequence(p.b, int(seq));
        if (w.s.n == 0) continue;
        const std::int64_t from = w.s.len - w.s.n > 0 ? w.s.len - w.s.n : 0;
        for (w.page = (from >> shift) + first; w.page << shift < w.s.len; w.page += g.pieces) body(w);
    }
}

// A work-group's threads over rows of dim / 8 pieces of 8 elements: each keeps
// its piece and goes from row to row.
struct Lanes {
    int row, step, at;  // first row, rows between, first element
    __device__ explicit Lanes(int dim)
    {
        const int per_row = dim / 8;
        step = kThreads / per_row;
        row = int(threadIdx.x) / per_row;
        at = int(threadIdx.x) % per_row * 8;
        if (row >= step) row = 1 << 30;  // threads left over
    }
};

constexpr int kHeld = 4;  // pieces a thread has in flight

// The largest |x| among the finite of eight elements, as bits.
template <class T> __device__ inline std::uint32_t largest(const typename T::elem *x, std::uint32_t m)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const std::uint32_t a = f32_bits(to_f32<T>(x[i])) & 0x7fffffffu;
        m = a < 0x7f800000u && a > m ? a : m;
    }
    return m;
}

// The smallest power of two s >= 2^-126 with amax / s <= 448 = 1.75 * 2^8; 0
// for 0.
__device__ inline float scale_for(std::uint32_t amax)
{
    if (amax == 0) return 0.0f;
    int field = int(amax >> 23) - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
    return bits_f32(std::uint32_t(field < 1 ? 1 : field) << 23);
}

// Whether s > 0 is a power of two with a normal inverse.
__device__ inline bool exact_inverse(float s)
{
    const std::uint32_t u = f32_bits(s), e = u >> 23;
    return (u & 0x7fffffu) == 0 && e >= 1 && e <= 253;
}

__device__ inline std::uint32_t to_codes(float a, float b, float c, float d)
{
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return std::uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true));
}

template <class T> struct Eight {
    typename T::elem x[8];
};

template <class T> __global__ __launch_bounds__(kThreads) void kv8_write_kernel(Kv8Problem p, Grid g)
{
    typedef typename T::elem elem;
    __shared__ std::uint32_t wave_max[kThreads / 64];
    const int dim = p.c.dim, block = p.c.block;
    const Lanes lanes(dim);
    for_each_piece(p, g, [&](const Piece &w) {
        const std::int64_t start = w.s.len - w.s.n;  // position of the sequence's first row (may be below 0)
        const std::int64_t t0 = w.page * block;
        const std::int64_t lo = start > t0 ? start : t0, hi = w.s.len < t0 + block ? w.s.len : t0 + block;
        const int kept = int(lo - t0), fresh = int(hi - lo);  // fresh >= 1
        const std::int64_t ld = w.kv ? p.ldv : p.ldk;
        const elem *src = static_cast<const elem *>(w.kv ? p.V : p.K) + (w.s.row0 + (lo - start)) * ld +
                          w.head * (w.kv ? p.hsv : p.hsk) + lanes.at;
        // The first pieces stay in registers; further ones are read again
        // below. They are on their way while the table is read, without
        // conditions (which would make them wait for one another): past the
        // last row it is read again, which changes no maximum.
        Eight<T> held[kHeld];
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int r = lanes.row + i * lanes.step;
            held[i] = load_any<Eight<T>>(src + (r < fresh ? r : fresh - 1) * ld);
        }
        const std::int64_t page = kv8_page(p.c, p.b, w.s.seq, w.page);
        if (page < 0) return;  // the same for the whole work-group
        std::uint8_t *codes = static_cast<std::uint8_t *>(w.kv ? p.c.V : p.c.K) + (page * p.c.heads + w.head) * block * dim + lanes.at;
        float *scale = (w.kv ? p.c.Vs : p.c.Ks) + page * p.c.heads + w.head;
        const float before = kept > 0 ? *scale : 0.0f;

        std::uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) m = largest<T>(held[i].x, m);
        for (int r = lanes.row + kHeld * lanes.step; r < fresh; r += lanes.step) m = largest<T>(load_any<Eight<T>>(src + r * ld).x, m);
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) {
            const std::uint32_t o = std::uint32_t(__shfl_xor(int(m), d));
            m = o > m ? o : m;
        }
        if ((threadIdx.x & 63) == 0) wave_max[threadIdx.x >> 6] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kThreads / 64; ++i) m = wave_max[i] > m ? wave_max[i] : m;
        const float s = __builtin_fmaxf(scale_for(m), before);
        const float inverse = s > 0.0f ? 1.0f / s : 0.0f;
        // A scale that this kernel left is a power of two, whose inverse is
        // exact; one that a caller set need not be (or have an inverse).
        const bool power = __builtin_amdgcn_readfirstlane(s == 0.0f || exact_inverse(s)) != 0;

        if (s != before) {
            // The page's earlier tokens, rounded to the risen scale.
            const float ratio = before * inverse;
            for (int r = lanes.row; r < kept; r += lanes.step) {
                u32x2 *at = reinterpret_cast<u32x2 *>(codes + r * dim);
                u32x2 v = *at;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(int(v[i]), false);
                    const auto b = __builtin_amdgcn_cvt_pk_f32_fp8(int(v[i]), true);
                    v[i] = to_codes(a[0] * ratio, a[1] * ratio, b[0] * ratio, b[1] * ratio);
                }
                *at = v;
            }
        }
        auto store = [&](const Eight<T> &v, int r) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = to_f32<T>(v.x[i]);
            if (power) {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] *= inverse;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] /= s;
            }
            // Finite quotients are at most 448.
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = (f32_bits(x[i]) & 0x7f800000u) == 0x7f800000u ? __builtin_nanf("") : x[i];
            *reinterpret_cast<u32x2 *>(codes + (kept + r) * dim) = u32x2{to_codes(x[0], x[1], x[2], x[3]), to_codes(x[4], x[5], x[6], x[7])};
        };
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            if (lanes.row + i * lanes.step < fresh) store(held[i], lanes.row + i * lanes.step);
        for (int r = lanes.row + kHeld * lanes.step; r < fresh; r += lanes.step) store(load_any<Eight<T>>(src + r * ld), r);
        __syncthreads();  // every thread has read the scale and wave_max
        if (threadIdx.x == 0) *scale = s;
    });
}

template <class T> __global__ __launch_bounds__(kThreads) void kv8_read_kernel(Kv8Problem p, Grid g)
{
    typedef typename T::elem elem;
    const int dim = p.c.dim, block = p.c.block;
    const Lanes lanes(dim);
    for_each_piece(p, g, [&](const Piece &w) {
        const std::int64_t start = w.s.len - w.s.n, t0 = w.page * block;
        const std::int64_t lo = start > t0 ? start : t0, hi = w.s.len < t0 + block ? w.s.len : t0 + block;
        const std::int64_t page = kv8_page(p.c, p.b, w.s.seq, w.page);
        const int count = int(hi - lo);
        const std::int64_t ld = w.kv ? p.ldv : p.ldk;
        elem *dst = static_cast<elem *>(w.kv ? p.V : p.K) + (w.s.row0 + (lo - start)) * ld + w.head * (w.kv ? p.hsv : p.hsk) + lanes.at;
        // A page that is not the cache's is not read; its rows are NaN.
        const std::int64_t at = (page < 0 ? 0 : page) * p.c.heads + w.head;
        const std::uint8_t *codes = static_cast<const std::uint8_t *>(w.kv ? p.c.V : p.c.K) + at * block * dim + (lo - t0) * dim + lanes.at;
        const float s = page < 0 ? __builtin_nanf("") : (w.kv ? p.c.Vs : p.c.Ks)[at];
        for (int r0 = lanes.row; r0 < count; r0 += kHeld * lanes.step) {
            u32x2 v[kHeld];
#pragma unroll
            for (int j = 0; j < kHeld; ++j)
                if (r0 + j * lanes.step < count) v[j] = *reinterpret_cast<const u32x2 *>(codes + (r0 + j * lanes.step) * dim);
#pragma unroll
            for (int j = 0; j < kHeld; ++j) {
                if (r0 + j * lanes.step >= count) continue;
                Eight<T> out;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(int(v[j][i]), false);
                    const auto b = __builtin_amdgcn_cvt_pk_f32_fp8(int(v[j][i]), true);
                    out.x[4 * i] = from_f32<T>(a[0] * s);
                    out.x[4 * i + 1] = from_f32<T>(a[1] * s);
                    out.x[4 * i + 2] = from_f32<T>(b[0] * s);
                    out.x[4 * i + 3] = from_f32<T>(b[1] * s);
                }
                __builtin_memcpy(dst + (r0 + j * lanes.step) * ld, &out, sizeof(out));
            }
        }
    });
}

template <class F> hipError_t launch(const Kv8Problem &p, F f32, F bf16, F f16, hipStream_t stream)
{
    const F kernel = p.dtype == SGEMM_F32 ? f32 : p.dtype == SGEMM_LP_BF16 ? bf16 : f16;
    Kv8Problem q = p;
    Grid g = grid_of(p);
    void *args[] = {&q, &g};
    return hipLaunchKernel(reinterpret_cast<const void *>(kernel), dim3(2u * unsigned(p.c.heads) * g.pieces * g.seqs), dim3(kThreads), args, 0,
                           stream);
}

}  // namespace

hipError_t launch_kv8_write(const Kv8Problem &p, hipStream_t stream)
{
    return launch(p, &kv8_write_kernel<F32>, &kv8_write_kernel<BF16>, &kv8_write_kernel<F16>, stream);
}

hipError_t launch_kv8_read(const Kv8Problem &p, hipStream_t stream)
{
    return launch(p, &kv8_read_kernel<F32>, &kv8_read_kernel<BF16>, &kv8_read_kernel<F16>, stream);
}

}  // namespace sgemm_impl
