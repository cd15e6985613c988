// The 4-bit cache of keys and values: quantising new rows into its pages
// (sgemm_kv4_write) and reading rows back (sgemm_kv4_read).
//
// A token and head has a scale of its own, max |x| / 6 in bfloat16, so that a
// new token changes nothing that the cache holds, no row waits for another,
// and nothing is atomic: a row of a head is a unit of its own, taken by as
// many lanes as it has pieces of eight elements (rounded up to a power of
// two), whose maximum goes round by lane exchanges.
//
// x / scale is needed to the last bit next to the midpoints of e2m1. The
// quotient is formed as y = x r with r = 1 / scale, and corrected once by its
// residual, y + (x - y scale) r. A midpoint m times the scale has at most 11
// significant bits, so x is either m scale itself, and the correction then
// lands on m exactly (the residual is exact, the correction's own error below
// 2^-45), or at least one unit of its last place away, which is more than half
// of a unit of m's: the corrected quotient then does not round to m.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "gemm.hpp"
#include "kv8.hpp"
#include "step.hpp"

namespace sgemm_impl {
namespace {

constexpr int kThreads = 256, kHeld = 4;  // units a thread has in flight

// How a work-group's threads lie over units (rows of one head): `group` lanes
// a unit, `across` heads side by side, rows below one another.
struct Lay {
    int group, across, deep;       // lanes of a unit, heads at once, rows at once
    unsigned chunk;                // rows of a sequence that a work-group takes: kHeld * deep
    unsigned pieces, seqs;         // chunks and sequences that the launch covers at once
};

Lay lay_of(const Kv4Problem &p)
{
    Lay l;
    l.group = 2;
    while (l.group < p.c.dim / 8) l.group *= 2;
    const int units = kThreads / l.group;
    l.across = p.c.heads < units ? p.c.heads : units;
    l.deep = units / l.across;
    l.chunk = unsigned(kHeld * l.deep);
    const std::int64_t n = p.b.max_new < p.b.rows ? p.b.max_new : p.b.rows, most = std::int64_t(1) << 22;
    std::int64_t pieces = (n + l.chunk - 1) / l.chunk;
    pieces = pieces < 1 ? 1 : pieces > most ? most : pieces;
    std::int64_t seqs = most / pieces;
    seqs = seqs < 1 ? 1 : seqs < p.b.seqs ? seqs : p.b.seqs;
    l.pieces = unsigned(pieces);
    l.seqs = unsigned(seqs);
    return l;
}

// The largest value of a unit's lanes, in all of them.
__device__ inline std::uint32_t unit_max(std::uint32_t m, int group)
{
    for (int d = group / 2; d > 0; d >>= 1) {
        const std::uint32_t o = std::uint32_t(__shfl_xor(int(m), d));
        m = o > m ? o : m;
    }
    return m;
}

// The bits of a row's scale, from those of its largest size (at least those of
// infinity: some value is not finite).
__device__ inline std::uint16_t scale_bits(std::uint32_t amax)
{
    if (amax >= 0x7f800000u) return 0x7fc0u;
    if (amax == 0) return 0;
    const std::uint16_t s = from_f32<BF16>(bits_f32(amax) / 6.0f);
    constexpr std::uint16_t kLeast = 27u << 7;  // 2^-100
    return s < kLeast ? kLeast : s;
}

__device__ inline std::uint32_t to_codes(const float *y)
{
    std::uint32_t v = 0;
    v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, y[0], y[1], 1.0f, 0);
    v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, y[2], y[3], 1.0f, 1);
    v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, y[4], y[5], 1.0f, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, y[6], y[7], 1.0f, 3);
}

__device__ inline void from_codes(std::uint32_t v, float *x)
{
    const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, 1.0f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, 1.0f, 1);
    const auto c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, 1.0f, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, 1.0f, 3);
    x[0] = a[0], x[1] = a[1], x[2] = b[0], x[3] = b[1], x[4] = c[0], x[5] = c[1], x[6] = d[0], x[7] = d[1];
}

template <class T> struct Eight {
    typename T::elem x[8];
};

// Where a work-group's thread works, and the walk over the sequences, chunks
// and heads that fall to it: body(sequence, head, first row of the thread).
struct Place {
    int at, head, row, kv;  // first element; head and row within the work-group's; K (0) or V (1)
    bool there;
};

template <class Body> __device__ inline void for_each_chunk(const Kv4Problem &p, const Lay &l, Body &&body)
{
    const int lane = int(threadIdx.x) & (l.group - 1), unit = int(threadIdx.x) / l.group;
    Place w;
    w.at = 8 * lane;
    w.head = unit % l.across;
    w.row = unit / l.across;
    w.there = w.row < l.deep;
    unsigned id = blockIdx.x;
    w.kv = int(id & 1);
    id >>= 1;
    const unsigned piece = id % l.pieces;
    for (unsigned seq = id / l.pieces; seq < unsigned(p.b.seqs); seq += l.seqs) {
        const Kv8Sequence s = kv8_sequence(p.b, int(seq));
        for (std::int64_t row = std::int64_t(piece) * l.chunk; row < s.n; row += std::int64_t(l.pieces) * l.chunk)
            for (int head = w.head; head - w.head < p.c.heads; head += l.across) body(s, w, head, row + w.row);
    }
}

template <class T> __global__ __launch_bounds__(kThreads) void kv4_write_kernel(Kv4Problem p, Lay l)
{
    typedef typename T::elem elem;
    const int dim = p.c.dim, shift = 31 - __builtin_clz(unsigned(p.c.block));
    for_each_chunk(p, l, [&](const Kv8Sequence &s, const Place &w, int head, std::int64_t row0) {
        const std::int64_t ld = w.kv ? p.ldv : p.ldk;
        const bool there = w.there && head < p.c.heads, mine = there && w.at < dim;
        const elem *src = static_cast<const elem *>(w.kv ? p.V : p.K) + s.row0 * ld + (there ? head : 0) * (w.kv ? p.hsv : p.hsk) +
                          (mine ? w.at : 0);
        // All loads first, without conditions: rows past the last repeat it.
        Eight<T> v[kHeld];
        std::int64_t page[kHeld];
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const std::int64_t r = row0 + i * l.deep;
            v[i] = load_any<Eight<T>>(src + (r < s.n ? r : s.n - 1) * ld);
        }
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const std::int64_t r = row0 + i * l.deep, t = s.len - s.n + r;
            page[i] = there && r < s.n && t >= 0 ? kv8_page(p.c, p.b, s.seq, t >> shift) : -1;
        }
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            float x[8];
            std::uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] = to_f32<T>(v[i].x[j]);
                const std::uint32_t a = f32_bits(x[j]) & 0x7fffffffu;
                m = a > m ? a : m;
            }
            m = unit_max(mine ? m : 0, l.group);
            const std::uint16_t sb = scale_bits(m);
            const float scale = to_f32<BF16>(sb), r = m == 0 || m >= 0x7f800000u ? 0.0f : 1.0f / scale;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float y = x[j] * r;
                x[j] = __builtin_fmaf(__builtin_fmaf(-y, scale, x[j]), r, y);
            }
            if (page[i] < 0) continue;
            const std::int64_t t = s.len - s.n + row0 + i * l.deep;
            const std::int64_t token = ((page[i] * p.c.heads + head) << shift) + (t & ((1 << shift) - 1));
            const std::uint32_t codes = m >= 0x7f800000u ? 0u : to_codes(x);
            if (mine) *reinterpret_cast<std::uint32_t *>(static_cast<std::uint8_t *>(w.kv ? p.c.V : p.c.K) + token * (dim / 2) + w.at / 2) = codes;
            if (w.at == 0) static_cast<std::uint16_t *>(w.kv ? p.c.Vs : p.c.Ks)[token] = sb;
        }
    });
}

template <class T> __global__ __launch_bounds__(kThreads) void kv4_read_kernel(Kv4Problem p, Lay l)
{
    typedef typename T::elem elem;
    const int dim = p.c.dim, shift = 31 - __builtin_clz(unsigned(p.c.block));
    for_each_chunk(p, l, [&](const Kv8Sequence &s, const Place &w, int head, std::int64_t row0) {
        if (!w.there || head >= p.c.heads || w.at >= dim) return;
        const std::int64_t ld = w.kv ? p.ldv : p.ldk;
        elem *dst = static_cast<elem *>(w.kv ? p.V : p.K) + s.row0 * ld + head * (w.kv ? p.hsv : p.hsk) + w.at;
        std::int64_t page[kHeld], t[kHeld];
        std::uint32_t v[kHeld];
        float scale[kHeld];
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const std::int64_t r = row0 + i * l.deep;
            t[i] = r < s.n ? s.len - s.n + r : -1;
            page[i] = t[i] >= 0 ? kv8_page(p.c, p.b, s.seq, t[i] >> shift) : -1;
        }
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            // A page that is not the cache's is not read: page 0 is in its place, and the rows are NaN.
            const std::int64_t token = (((page[i] < 0 ? 0 : page[i]) * p.c.heads + head) << shift) + (t[i] & ((1 << shift) - 1));
            v[i] = *reinterpret_cast<const std::uint32_t *>(static_cast<const std::uint8_t *>(w.kv ? p.c.V : p.c.K) + token * (dim / 2) + w.at / 2);
            scale[i] = to_f32<BF16>(static_cast<const std::uint16_t *>(w.kv ? p.c.Vs : p.c.Ks)[token]);
        }
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            if (t[i] < 0) continue;
            float s1 = scale[i];
            if (page[i] < 0 || (f32_bits(s1) & 0x7f800000u) == 0x7f800000u) s1 = __builtin_nanf("");
            float x[8];
            from_codes(v[i], x);
            Eight<T> out;
#pragma unroll
            for (int j = 0; j < 8; ++j) out.x[j] = from_f32<T>(x[j] * s1);
            __builtin_memcpy(dst + (row0 + i * l.deep) * ld, &out, sizeof(out));
        }
    });
}

template <class F> hipError_t launch(const Kv4Problem &p, F f32, F bf16, F f16, hipStream_t stream)
{
    const F kernel = p.dtype == SGEMM_F32 ? f32 : p.dtype == SGEMM_LP_BF16 ? bf16 : f16;
    Kv4Problem q = p;
    Lay l = lay_of(p);
    void *args[] = {&q, &l};
    return hipLaunchKernel(reinterpret_cast<const void *>(kernel), dim3(2u * l.pieces * l.seqs), dim3(kThreads), args, 0, stream);
}

}  // namespace

hipError_t launch_kv4_write(const Kv4Problem &p, hipStream_t stream)
{
    return launch(p, &kv4_write_kernel<F32>, &kv4_write_kernel<BF16>, &kv4_write_kernel<F16>, stream);
}

hipError_t launch_kv4_read(const Kv4Problem &p, hipStream_t stream)
{
    return launch(p, &kv4_read_kernel<F32>, &kv4_read_kernel<BF16>, &kv4_read_kernel<F16>, stream);
}

}  // namespace sgemm_impl
