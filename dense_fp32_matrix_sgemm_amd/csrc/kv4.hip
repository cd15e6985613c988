// The 4-bit cache of keys and values: quantising new rows into its pages
// (sgemm_kv4_write) and reading rows back (sgemm_kv4_read).
//
// A token and head has a scale of its own, max |x| / 6 in bfloat16, so that a
// new token changes nothing that the cache holds, no row waits for another,
// and nothing is atomic: a row of a head is a unit of its own, taken by as
// many lanes as it has pieces of eight elements (rounded up to a power of
// two), whose maximum goes round by lane exchanges. A thread has four units in
// flight: with two or eight, or 512 or 1024 threads, nothing was gained.
//
// 4 prompts of up to 4096 tokens, 8 heads of 128 in bf16: write 17.5 us for 61 MB
// (3.5 TB/s), of which its vector instructions take a third, read 13.3 for 64 MB
// (4.8; 16.0 with outputs through the caches); 64 sequences of one token: write 3.8 us, three round trips, and 128
// tokens of each read into float32 17.6 for 76 MB (4.3). When rows are written
// they are loaded first, as soon as their sequence is known, and only the stores
// wait for their pages; when rows are read back, the loads do. More units in flight
// did not help either. What keeps the write from a copy's rate was not found out: a
// wave stores pieces of 64 bytes for each of four heads, and each scale apart,
// 2 bytes in a line of its own; another order was not tried.
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

// The largest value of a unit's 2 to 32 lanes, in all of them: from the other
// lane of a pair, the other pair of four, then the lanes of an eight and of a
// sixteen in reverse, then the other sixteen.
template <int Ctrl> __device__ inline std::uint32_t max_with(std::uint32_t m)
{
    const std::uint32_t o = std::uint32_t(__builtin_amdgcn_mov_dpp(int(m), Ctrl, 0xf, 0xf, true));
    return o > m ? o : m;
}
__device__ inline std::uint32_t unit_max(std::uint32_t m, int group)
{
    m = max_with<0xb1>(m);
    if (group > 2) m = max_with<0x4e>(m);
    if (group > 4) m = max_with<0x141>(m);
    if (group > 8) m = max_with<0x140>(m);
    if (group > 16) {
        const auto x = __builtin_amdgcn_permlane16_swap(m, m, false, false);
        m = x[0] > x[1] ? x[0] : x[1];
    }
    return m;
}

// The largest size of eight elements, as the bits of a float32 (at least those
// of infinity if one is not finite). The bits of a size grow with it in every
// type, so the 16-bit ones are compared as they are, two at a time.
template <class T> struct Eight {
    typename T::elem x[8];
};
template <class T> __device__ inline std::uint32_t largest(const Eight<T> &v)
{
    if constexpr (sizeof(typename T::elem) == 4) {
        std::uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const std::uint32_t a = f32_bits(v.x[j]) & 0x7fffffffu;
            m = a > m ? a : m;
        }
        return m;
    } else {
        typedef __attribute__((ext_vector_type(2))) std::uint16_t u16x2;
        const u32x4 w = __builtin_bit_cast(u32x4, v) & 0x7fff7fffu;
        u16x2 m = __builtin_bit_cast(u16x2, w[0]);
#pragma unroll
        for (int j = 1; j < 4; ++j) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, std::uint32_t(w[j])));
        return f32_bits(to_f32<T>(m[0] > m[1] ? m[0] : m[1]));
    }
}

// The bits of a row's scale, from those of its largest size (at least those of
// infinity: some value is not finite). The quotient by 6 is corrected by its
// residual as the elements' are, and so rounded as a division's is (where it is
// not among the subnormals, which are far below the least scale).
__device__ inline std::uint16_t scale_bits(std::uint32_t amax)
{
    const float a = bits_f32(amax), sixth = 1.0f / 6.0f, y = a * sixth;
    const std::uint16_t s = from_f32<BF16>(__builtin_fmaf(__builtin_fmaf(-y, 6.0f, a), sixth, y));
    constexpr std::uint16_t kLeast = 27u << 7;  // 2^-100
    return amax >= 0x7f800000u ? 0x7fc0u : amax == 0 ? 0u : s < kLeast ? kLeast : s;
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

// Eight values times s, rounded to T.
template <class T> __device__ inline void rounded(const float *x, float s, Eight<T> &out)
{
    if constexpr (sizeof(typename T::elem) == 4) {
#pragma unroll
        for (int j = 0; j < 8; ++j) out.x[j] = x[j] * s;
    } else {
        u32x4 w;
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = rounded2<T>(x[2 * j] * s, x[2 * j + 1] * s);
        out = __builtin_bit_cast(Eight<T>, w);
    }
}

// A thread's place among its work-group's units, and a chunk of rows: the
// sequence, where its table is, the chunk's first row and its position, and the
// rows of the chunk. All but the thread's place is the same for a work-group.
struct Place {
    int at, head, row, kv;  // first element; head and row within the work-group's; K (0) or V (1)
    bool there;
};
struct Chunk {
    const int *table;
    std::int64_t row0;
    int t0, rows;
};

// Calls body(chunk, place, head) for the chunks and heads that fall to this work-group.
template <class Body> __device__ inline void for_each_chunk(const Kv4Problem &p, const Lay &l, int shift, Body &&body)
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
        for (std::int64_t row = std::int64_t(piece) * l.chunk; row < s.n; row += std::int64_t(l.pieces) * l.chunk) {
            const Chunk c = {p.b.table + std::int64_t(seq) * p.b.table_ld, s.row0 + row, int(s.len - s.n + row),
                             int(s.n - row < l.chunk ? s.n - row : l.chunk)};
            for (int head = 0; head < p.c.heads; head += l.across) body(c, w, head + w.head);
        }
    }
}

// The page of position t, or -1 where there is none or the table names none of the cache's.
__device__ inline int page_of(const Kv4Problem &p, const Chunk &c, int t, int shift)
{
    const int column = t >> shift;
    if (t < 0 || column >= p.b.table_ld) return -1;
    const int page = c.table[column];
    return unsigned(page) < unsigned(p.c.pages) ? page : -1;
}

template <class T> __global__ __launch_bounds__(kThreads) void kv4_write_kernel(Kv4Problem p, Lay l)
{
    typedef typename T::elem elem;
    const int dim = p.c.dim, shift = 31 - __builtin_clz(unsigned(p.c.block)), mask = p.c.block - 1;
    const std::int64_t page_tokens = std::int64_t(p.c.heads) << shift;
    for_each_chunk(p, l, shift, [&](const Chunk &c, const Place &w, int head) {
        const std::int64_t ld = w.kv ? p.ldv : p.ldk;
        const bool there = w.there && head < p.c.heads, mine = there && w.at < dim;
        const elem *const src = static_cast<const elem *>(w.kv ? p.V : p.K) + c.row0 * ld + (there ? head : 0) * (w.kv ? p.hsv : p.hsk) +
                                (mine ? w.at : 0);
        // All loads first, without conditions: rows past the last repeat it.
        Eight<T> v[kHeld];
        int page[kHeld];
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int r = w.row + i * l.deep;
            v[i] = load_any<Eight<T>>(src + (r < c.rows ? r : c.rows - 1) * ld);
        }
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int r = w.row + i * l.deep;
            page[i] = there && r < c.rows ? page_of(p, c, c.t0 + r, shift) : -1;
        }
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const std::uint32_t m = unit_max(mine ? largest(v[i]) : 0u, l.group);
            const std::uint16_t sb = scale_bits(m);
            const float scale = to_f32<BF16>(sb), inverse = m == 0 ? 0.0f : __builtin_amdgcn_rcpf(scale);
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float x = to_f32<T>(v[i].x[j]), q = x * inverse;
                y[j] = __builtin_fmaf(__builtin_fmaf(-q, scale, x), inverse, q);
            }
            if (page[i] < 0) continue;
            const std::int64_t token = page[i] * page_tokens + ((std::int64_t(head) << shift) + ((c.t0 + w.row + i * l.deep) & mask));
            const std::uint32_t codes = m >= 0x7f800000u ? 0u : to_codes(y);
            if (mine) *reinterpret_cast<std::uint32_t *>(static_cast<std::uint8_t *>(w.kv ? p.c.V : p.c.K) + token * (dim / 2) + w.at / 2) = codes;
            if (w.at == 0) static_cast<std::uint16_t *>(w.kv ? p.c.Vs : p.c.Ks)[token] = sb;
        }
    });
}

// Stream: outputs of 16 bits that are kept out of the caches. (Such a store has to
// cover whole lines. A float32 lane's 32 bytes are two stores, 17.9 -> 27.2 us for
// 64 sequences' 128 tokens; with the lanes' halves passed round, so that they do,
// nothing was gained.)
template <class T, bool Stream> __global__ __launch_bounds__(kThreads) void kv4_read_kernel(Kv4Problem p, Lay l)
{
    typedef typename T::elem elem;
    const int dim = p.c.dim, shift = 31 - __builtin_clz(unsigned(p.c.block)), mask = p.c.block - 1;
    const std::int64_t page_tokens = std::int64_t(p.c.heads) << shift;
    for_each_chunk(p, l, shift, [&](const Chunk &c, const Place &w, int head) {
        if (!w.there || head >= p.c.heads || w.at >= dim) return;
        const std::int64_t ld = w.kv ? p.ldv : p.ldk;
        elem *const dst = static_cast<elem *>(w.kv ? p.V : p.K) + c.row0 * ld + head * (w.kv ? p.hsv : p.hsk) + w.at;
        const std::uint8_t *const codes = static_cast<const std::uint8_t *>(w.kv ? p.c.V : p.c.K) + w.at / 2;
        const std::uint16_t *const scales = static_cast<const std::uint16_t *>(w.kv ? p.c.Vs : p.c.Ks);
        int page[kHeld];
        std::uint32_t v[kHeld];
        std::uint16_t scale[kHeld];
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int r = w.row + i * l.deep;
            page[i] = page_of(p, c, c.t0 + (r < c.rows ? r : c.rows - 1), shift);
        }
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            // A page that is not the cache's is not read: page 0 is in its place, and the rows are NaN.
            const std::int64_t token = (page[i] < 0 ? 0 : page[i]) * page_tokens + ((std::int64_t(head) << shift) + ((c.t0 + w.row + i * l.deep) & mask));
            v[i] = *reinterpret_cast<const std::uint32_t *>(codes + token * (dim / 2));
            scale[i] = scales[token];
        }
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int r = w.row + i * l.deep;
            if (r >= c.rows || c.t0 + r < 0) continue;
            const float s = page[i] < 0 || (scale[i] & 0x7f80u) == 0x7f80u ? __builtin_nanf("") : to_f32<BF16>(scale[i]);
            float x[8];
            from_codes(v[i], x);
            Eight<T> out;
            rounded<T>(x, s, out);
            if constexpr (Stream) stream_store(dst + r * ld, __builtin_bit_cast(u32x4, out));
            else __builtin_memcpy(dst + r * ld, &out, sizeof(out));
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
    if (p.stream()) return launch(p, &kv4_read_kernel<F32, false>, &kv4_read_kernel<BF16, true>, &kv4_read_kernel<F16, true>, stream);
    return launch(p, &kv4_read_kernel<F32, false>, &kv4_read_kernel<BF16, false>, &kv4_read_kernel<F16, false>, stream);
}

}  // namespace sgemm_impl
