// C = alpha * A * W^T + beta * C with W held in 4 bits (sgemm_w4): each type
// of A is its own translation unit (w4_f32.hip, w4_bf16.hip, w4_f16.hip).
//
// Per output C[m][n] the sum over k falls into groups that share one scale:
//
//     sum_g S[n][g] * ( sum_{k in g} A[m][k] * (q[n][k] - z[n][g]) )
//
// q - z is a whole number of -15..15, which bf16 and f16 hold exactly, so the
// inner sums run on the 16-bit matrix cores (v_mfma_f32_16x16x32) with exact
// products and float32 sums, and each group's sum is then multiplied by its
// scale in float32: no rounding but those of float32 sums. float32 A enters
// as three bf16 parts that add up to it exactly (split3).
//
// Zero points are subtracted from the codes before the product, not through
// the row sums of A afterwards: that would be cheaper, but a group of codes
// equal to its zero point would leave the rounding of a cancelled sum instead
// of 0, and an infinity in A would give NaN where the product has infinity.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "lowbit.hpp"

namespace sgemm_impl {
namespace {

constexpr int kW4Chunk = 128;  // k that a wave takes at a time: 16 bytes of codes a lane

// (x & m) | c in one v_and_or_b32: with two constants that takes one of them
// in a vector register, which the compiler does not do by itself.
__device__ inline std::uint32_t and_or(std::uint32_t x, std::uint32_t m, std::uint32_t c)
{
    asm("" : "+v"(c));
    return (x & m) | c;
}

// Eight codes of one word as exact 16-bit numbers. `z` is the zero point. The order of k within the eight is the type's own:
// A's operand comes in the same (AOperand).
//
// bf16: without zero points the codes become signed nibbles (q - 8, by
// flipping the top bit) and v_cvt_off_f32_i4 gives nibble / 16 in float32,
// whose upper half is the bf16 number; the 16 multiplies the finished sum (a
// scale from 2^124 on would overflow by it). With zero
// points the four bytes of a word's even (odd) nibbles have z subtracted at
// once, each kept from borrowing by its top bit, and are converted as signed
// bytes. Either takes a conversion a code and a v_perm for two.
// f16: a nibble or'ed into the fraction of 1024 is 1024 + q (the next nibble,
// four bits higher, 1024 + 16 q), and one packed add (multiply-add) leaves
// q - z exactly: three instructions for two codes.
template <class T, bool ZP> struct Codes {
    static constexpr float kUnit = ZP ? 1.0f : 16.0f;  // what the finished sum has to be multiplied by
    std::uint32_t z4;
    __device__ explicit Codes(std::uint32_t z) : z4(z * 0x01010101u) {}
    __device__ Frag operator()(std::uint32_t w) const
    {
        float f[8];
        if (ZP) {
            const std::uint32_t even = (and_or(w, 0x0f0f0f0fu, 0x80808080u) - z4) ^ 0x80808080u;
            const std::uint32_t odd = (and_or(w >> 4, 0x0f0f0f0fu, 0x80808080u) - z4) ^ 0x80808080u;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = float(int(std::int8_t(even >> (8 * i))));
                f[2 * i + 1] = float(int(std::int8_t(odd >> (8 * i))));
            }
        } else {
            const std::uint32_t even = w ^ 0x88888888u;
            std::uint32_t odd = even >> 4;
            asm("" : "+v"(odd));  // its bytes are then selected in the conversions, without more shifts
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __builtin_amdgcn_cvt_off_f32_i4(int(even >> (8 * i)));
                f[2 * i + 1] = __builtin_amdgcn_cvt_off_f32_i4(int(odd >> (8 * i)));
            }
        }
        Frag r;
#pragma unroll
        for (int i = 0; i < 4; ++i) r.v[i] = pack_hi(f[2 * i], f[2 * i + 1]);
        return r;
    }
};
template <bool ZP> struct Codes<F16, ZP> {
    static constexpr float kUnit = 1.0f;
    std::uint32_t lo, hi;  // pairs of -(1024 + z) and -(64 + z), by their bits
    __device__ explicit Codes(std::uint32_t z) : lo((z | z << 16) | 0xe400e400u), hi((z << 4 | z << 20) | 0xd400d400u) {}
    __device__ Frag operator()(std::uint32_t w) const
    {
        const f16x2 sixteenth = {_Float16(0.0625f), _Float16(0.0625f)};
        Frag r;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const std::uint32_t x = w >> (8 * i);
            const f16x2 a = __builtin_bit_cast(f16x2, and_or(x, 0x000f000fu, 0x64006400u)) + __builtin_bit_cast(f16x2, lo);
            const f16x2 b = __builtin_bit_cast(f16x2, and_or(x, 0x00f000f0u, 0x64006400u)) * sixteenth + __builtin_bit_cast(f16x2, hi);
            r.v[2 * i] = __builtin_bit_cast(std::uint32_t, a);      // codes 2i, 2i + 4
            r.v[2 * i + 1] = __builtin_bit_cast(std::uint32_t, b);  // codes 2i + 1, 2i + 5
        }
        return r;
    }
};

// Eight elements of a row of A as operands of the matrix instruction, in
// kPlanes parts that add up to them: what is kept in LDS.
template <class T> struct AOperand;
template <> struct AOperand<BF16> {
    static constexpr int kPlanes = 1;
    typedef std::uint16_t elem;
    Frag f[1];
    __device__ void set(const std::uint16_t *x) { __builtin_memcpy(&f[0], x, 16); }
    __device__ f32x4 times(const Frag &w, f32x4 acc) const { return mfma_bf16(f[0], w, acc); }
};
template <> struct AOperand<F16> {
    static constexpr int kPlanes = 1;
    typedef std::uint16_t elem;
    Frag f[1];
    __device__ void set(const std::uint16_t *x)
    {
        u32x4 r;
        __builtin_memcpy(&r, x, 16);
        // (a0 a1)(a2 a3)(a4 a5)(a6 a7) -> (a0 a4)(a1 a5)(a2 a6)(a3 a7), the codes' order.
        f[0].v[0] = __builtin_amdgcn_perm(r[2], r[0], 0x05040100u);
        f[0].v[1] = __builtin_amdgcn_perm(r[2], r[0], 0x07060302u);
        f[0].v[2] = __builtin_amdgcn_perm(r[3], r[1], 0x05040100u);
        f[0].v[3] = __builtin_amdgcn_perm(r[3], r[1], 0x07060302u);
    }
    __device__ f32x4 times(const Frag &w, f32x4 acc) const { return mfma_f16(f[0], w, acc); }
};
template <> struct AOperand<F32> {
    static constexpr int kPlanes = 3;
    typedef float elem;
    Frag f[3];
    __device__ void set(const float *x) { split3(x, f[0], f[1], f[2]); }
    __device__ f32x4 times(const Frag &w, f32x4 acc) const
    {
        return mfma_bf16(f[0], w, mfma_bf16(f[1], w, mfma_bf16(f[2], w, acc)));
    }
};

// Eight elements of a row from k on, zeros from K on.
template <class T> __device__ inline void load_a(const typename T::elem *row, int k, int K, typename T::elem *x)
{
    struct Eight {
        typename T::elem x[8];
    };
    if (k + 8 <= K) {
        const Eight v = load_any<Eight>(row + k);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = v.x[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = k + i < K ? row[k + i] : typename T::elem(0);
    }
}

// Lanes 16 r + c hold in word j the codes of k = 32 r + 8 j; afterwards those
// of k = 32 j + 8 r: a step of the matrix instruction (word j of all lanes)
// then spans 32 adjacent k, inside one group. Row r's word j goes to row j's
// word r, by gfx950's exchanges of half waves and of rows of 16 lanes.
__device__ inline u32x4 steps_of_codes(u32x4 w)
{
    const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    return u32x4{c[0], c[1], d[0], d[1]};
}

template <int N> struct Words {
    std::uint32_t v[N];
};

// N zero points as they come from memory. One or two stay in a type of their
// size: widening them where they are loaded would wait for the load.
template <int N> struct Bytes {
    Words<(N + 3) / 4> w;
    __device__ void load(const std::uint8_t *p) { w = load_any<Words<(N + 3) / 4>>(p); }
    __device__ std::uint32_t at(int i) const { return w.v[i / 4] >> (8 * (i % 4)); }
};
template <> struct Bytes<1> {
    std::uint8_t w;
    __device__ void load(const std::uint8_t *p) { w = *p; }
    __device__ std::uint32_t at(int) const { return w; }
};
template <> struct Bytes<2> {
    std::uint16_t w;
    __device__ void load(const std::uint8_t *p) { w = load_any<std::uint16_t>(p); }
    __device__ std::uint32_t at(int i) const { return std::uint32_t(w) >> (8 * i); }
};

// N scales of type ST, likewise.
template <class ST, int N> struct ScaleSet {
    Words<N / 2> w;
    __device__ void load(const void *S, std::int64_t i) { w = load_any<Words<N / 2>>(static_cast<const std::uint16_t *>(S) + i); }
    __device__ float at(int i) const { return to_f32<ST>(std::uint16_t(w.v[i / 2] >> (16 * (i % 2)))); }
};
template <class ST> struct ScaleSet<ST, 1> {
    typename ST::elem w;
    __device__ void load(const void *S, std::int64_t i) { w = load_any<typename ST::elem>(static_cast<const typename ST::elem *>(S) + i); }
    __device__ float at(int) const { return to_f32<ST>(w); }
};
template <int N> struct ScaleSet<F32, N> {
    Words<N> w;
    __device__ void load(const void *S, std::int64_t i) { w = load_any<Words<N>>(static_cast<const float *>(S) + i); }
    __device__ float at(int i) const { return bits_f32(w.v[i]); }
};
template <> struct ScaleSet<F32, 1> {
    float w;
    __device__ void load(const void *S, std::int64_t i) { w = static_cast<const float *>(S)[i]; }
    __device__ float at(int) const { return w; }
};

// The scales and zero points of N runs of 32 GS k from k0 on, for one column.
// Run: group == 32 GS, so that they are adjacent and come in one load each;
// otherwise group is a multiple of 32 GS and each run has its own loads.
template <class ST, int GS, int N, bool ZP, bool Run> struct Groups {
    static constexpr int kSets = Run ? 1 : N, kPer = Run ? N : 1;
    ScaleSet<ST, kPer> s[kSets];
    Bytes<kPer> z[kSets];
    __device__ void load(const void *S, std::int64_t srow, const std::uint8_t *zrow, unsigned k0, int group)
    {
#pragma unroll
        for (int i = 0; i < kSets; ++i) {
            const unsigned g = Run ? k0 / (32u * GS) : (k0 + i * (32u * GS)) / unsigned(group);
            s[i].load(S, srow + g);
            if (ZP) z[i].load(zrow + g);
        }
    }
    __device__ float scale(int run) const { return Run ? s[0].at(run) : s[Run ? 0 : run].at(0); }
    __device__ std::uint32_t zero(int run) const { return ZP ? (Run ? z[0].at(run) : z[Run ? 0 : run].at(0)) & 15u : 8u; }
};

// N scales of a runtime type, for the tile kernels: loaded as two runs of N
// 16-bit words without a branch (for a 16-bit type the second repeats the
// first), told apart where they are used.
struct AnyType {};
template <int N> struct ScaleSet<AnyType, N> {
    Words<N / 2> a, b;
    __device__ void load(const void *S, std::int64_t i, bool f32)
    {
        const char *p = static_cast<const char *>(S) + i * (f32 ? 4 : 2);
        a = load_any<Words<N / 2>>(p);
        b = load_any<Words<N / 2>>(p + (f32 ? 2 * N : 0));
    }
    __device__ float at(int i, int stype) const
    {
        const std::uint16_t x = std::uint16_t(a.v[i / 2] >> (16 * (i % 2)));
        const float f = bits_f32(i < N / 2 ? a.v[i < N / 2 ? i : 0] : b.v[i < N / 2 ? 0 : i - N / 2]);
        return stype == SGEMM_F32 ? f : stype == SGEMM_LP_BF16 ? to_f32<BF16>(x) : to_f32<F16>(x);
    }
};
template <> struct ScaleSet<AnyType, 1> {
    std::uint16_t a, b;
    __device__ void load(const void *S, std::int64_t i, bool f32)
    {
        const char *p = static_cast<const char *>(S) + i * (f32 ? 4 : 2);
        a = load_any<std::uint16_t>(p);
        b = load_any<std::uint16_t>(p + (f32 ? 2 : 0));
    }
    __device__ float at(int, int stype) const
    {
        const float f = bits_f32(a | std::uint32_t(b) << 16);
        return stype == SGEMM_F32 ? f : stype == SGEMM_LP_BF16 ? to_f32<BF16>(a) : to_f32<F16>(a);
    }
};

// As Groups; past K (the last slab) scales are 0, as A is (a last group's
// infinite scale would make NaN of it).
template <int GS, int N, bool ZP, bool Run> struct AnyGroups {
    static constexpr int kSets = Run ? 1 : N, kPer = Run ? N : 1;
    ScaleSet<AnyType, kPer> s[kSets];
    Bytes<kPer> z[kSets];
    __device__ void load(const W4Problem &p, std::int64_t srow, const std::uint8_t *zrow, int k0)
    {
#pragma unroll
        for (int i = 0; i < kSets; ++i) {
            const unsigned g = Run ? unsigned(k0) / (32u * GS) : unsigned(k0 + i * (32 * GS)) / unsigned(p.group);
            s[i].load(p.S, srow + g, p.stype == SGEMM_F32);
            if (ZP) z[i].load(zrow + g);
        }
    }
    __device__ void load_last(const W4Problem &p, std::int64_t srow, const std::uint8_t *zrow, int k0)
    {
        const bool f32 = p.stype == SGEMM_F32;
        std::uint16_t a[N], b[N];
        std::uint8_t zz[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const bool past = k0 + 32 * GS * i >= p.K;
            const int k = past ? p.K - 1 : k0 + 32 * GS * i;
            ScaleSet<AnyType, 1> one;
            one.load(p.S, srow + k / p.group, f32);
            a[i] = past ? 0 : one.a, b[i] = past ? 0 : one.b;
            zz[i] = ZP ? zrow[k / p.group] : 0;
        }
        if constexpr (Run && N > 1) {
            // As the adjacent load would have left them.
            std::uint16_t x[2 * N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                x[f32 ? 2 * i : i] = a[i];
                if (f32) x[2 * i + 1] = b[i];
            }
            __builtin_memcpy(&s[0].a, x, 2 * N);
            __builtin_memcpy(&s[0].b, x + N, 2 * N);
        } else {
#pragma unroll
            for (int i = 0; i < kSets; ++i) s[i].a = a[i], s[i].b = b[i];
        }
        __builtin_memcpy(&z, zz, sizeof(zz));
    }
    __device__ float scale(int run, int stype) const { return Run ? s[0].at(run, stype) : s[Run ? 0 : run].at(0, stype); }
    __device__ std::uint32_t zero(int run) const { return ZP ? (Run ? z[0].at(run) : z[Run ? 0 : run].at(0)) & 15u : 8u; }
};

// What a wave loads for U chunks of k; Held: A comes from LDS.
template <class T> struct Eight {
    typename T::elem x[8];
};
template <class T, class ST, int GS, int U, bool ZP, bool Run, bool Held> struct W4Stage {
    u32x4 w[U];
    Groups<ST, GS, 4 * U / GS, ZP, Run> g;
    Eight<T> a[Held ? 1 : 4 * U];  // Held: not used
};

// How a product is laid out over work-groups (plan_w4).
struct W4Layout {
    int wn, wk;  // waves along N and along K
    int slabs;   // runs of K whose A is held in LDS, one after the other
    int pitch;   // bytes from one held row to the next: 16 more than a multiple of 128, so that 16 rows meet in no bank
};

// Up to 16 rows of A. One work-group: all rows of C by 16 wn columns. The
// codes go from memory to registers once: each wave takes a run of K for its
// 16 columns in steps of U chunks of 128, each lane 16 bytes of one column's
// codes per chunk. The wk waves of a column tile add their sums through LDS
// in their order, so the result does not depend on timing. GS: steps of 32 k
// that share a scale.
//
// Held: a slab of A's rows lies in LDS as matrix operands, read by every wave
// (and the runs are the slab's). Otherwise A comes straight to registers,
// eight elements of a row for each lane and matrix instruction: no barriers,
// but more loads in all. plan_w4 chooses.
//
// 1 row of bf16 by 16384 x 4096 with zero points (35 MB) takes 12.5 us on the
// device, 2.8 TB/s; 8 rows by 8192 x 8192 (34 MB) 15.8. Of the 12.5 us the
// loads alone take 8.7 and A's way to LDS 1, neither of which more loads in
// flight shortened (A or codes, one to three steps further ahead: 13.9 to 16.7
// us). With few columns most compute units have no work-group (K is not divided
// over work-groups): 13 rows of float32 by 2047 x 4093 use 128 of 256 and take
// 13.7 us for 5.8 MB, 16 rows by 1024 x 16384 use 64 and take 38.7 for 9.7 MB.
template <class T, class ST, int GS, bool ZP, int U, bool Short, bool Run, bool Held>
__global__ __launch_bounds__(64 * kRowsWaves) void w4_rows_kernel(W4Problem p, W4Layout l)
{
    extern __shared__ __align__(16) char lds[];  // A: [plane][row][k] as 16-bit operands
    typedef typename T::elem elem;
    typedef W4Stage<T, ST, GS, U, ZP, Run, Held> Stage;
    typedef AOperand<T> Operand;
    typedef Codes<T, ZP> Code;
    constexpr int kStep = kW4Chunk * U, kPlanes = Operand::kPlanes;
    float *const part = reinterpret_cast<float *>(lds);  // then the sums: [wave][row][column]
    const int lane = threadIdx.x & 63, c = lane & 15, kq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wk = wave % l.wk, wn = wave / l.wk, cols = 16 * l.wn, rows = p.M;
    const std::int64_t c0 = std::int64_t(blockIdx.x) * cols;
    const int bytes = p.K / 2 + p.K % 2;

    // Columns past the last read it again; their sums are not stored.
    const std::int64_t n = c0 + wn * 16 + c < p.N ? c0 + wn * 16 + c : p.N - 1, srow = n * p.lds;
    const std::uint8_t *const wrow = p.W + n * p.ldw, *const zrow = ZP ? p.Z + n * p.ldz : nullptr;

    // Likewise rows past the last.
    const int my_row = c < rows ? c : rows - 1;
    const elem *const arow = static_cast<const elem *>(p.A) + my_row * p.lda;

    auto load = [&](Stage &st, unsigned k0) {
#pragma unroll
        for (int u = 0; u < U; ++u) st.w[u] = load_any<u32x4>(wrow + (k0 / 2 + 64 * u + 16 * kq));
        if constexpr (!Held) {
#pragma unroll
            for (int s = 0; s < 4 * U; ++s) st.a[s] = load_any<Eight<T>>(arow + (k0 + 32 * s + 8 * kq));
        }
        st.g.load(p.S, srow, zrow, k0, p.group);
    };

    const char *held[kPlanes];
#pragma unroll
    for (int f = 0; f < kPlanes; ++f) held[f] = lds + (f * rows + my_row) * l.pitch + 16 * kq;
    f32x4 out = {0, 0, 0, 0};

    auto operand = [&](int k) {  // A's operand of the step of 32 that starts at k of the held slab
        Operand a;
#pragma unroll
        for (int f = 0; f < kPlanes; ++f) a.f[f].v = *reinterpret_cast<const u32x4 *>(held[f] + 2 * k);
        return a;
    };
    auto multiply = [&](const Stage &st, int k0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const u32x4 w = steps_of_codes(st.w[u]);
#pragma unroll
            for (int g = 0; g < 4 / GS; ++g) {
                const int run = u * (4 / GS) + g;
                f32x4 acc;
#pragma unroll
                for (int s = 0; s < GS; ++s) {
                    const Frag wf = Code(st.g.zero(run))(w[g * GS + s]);
                    Operand a;
                    if constexpr (Held) {
                        a = operand(k0 + 128 * u + 32 * (g * GS + s));
                    } else {
                        a.set(st.a[4 * u + g * GS + s].x);
                    }
                    acc = a.times(wf, s == 0 ? f32x4{0, 0, 0, 0} : acc);
                }
                float s = st.g.scale(run);
                // Widened once, not in each of the multiply-adds (v_fma_mix_f32: 8 rows by 8192 x 8192 15.8 -> 16.5 us).
                if (!ZP) asm("" : "+v"(s));
#pragma unroll
                for (int r = 0; r < 4; ++r) out[r] += s * acc[r];
            }
        }
    };

    // Slabs share K's whole steps evenly; the last has the rest of K as well.
    const int k_steps = p.K / kStep, base = k_steps / l.slabs, extra = k_steps % l.slabs;
    int slab0 = 0;
    for (int j = 0; j < l.slabs; ++j) {
        const int all = Short ? 0 : base + (j < extra), slab_k = j + 1 < l.slabs ? all * kStep : p.K - slab0;
        // This wave's run of the slab's whole steps: at least one unless
        // Short. The first loads are on their way while A goes to LDS.
        const int s0 = wk * all / l.wk, steps = (wk + 1) * all / l.wk - s0;
        Stage st;
        if constexpr (!Short) load(st, slab0 + s0 * kStep);

        if constexpr (Held) {
            if (j > 0) __syncthreads();  // the last slab has been read
            const int eights = (slab_k + 31) / 32 * 4;
            for (int e = threadIdx.x; e < rows * eights; e += blockDim.x) {
                const int r = e / eights, at = e % eights;
                elem x[8];
                load_a<T>(static_cast<const elem *>(p.A) + r * p.lda + slab0, 8 * at, slab_k, x);
                Operand a;
                a.set(x);
#pragma unroll
                for (int f = 0; f < kPlanes; ++f) *reinterpret_cast<u32x4 *>(lds + (f * rows + r) * l.pitch + 16 * at) = a.f[f].v;
            }
            __syncthreads();
        }

        if constexpr (!Short) {
            for (int i = 0; i + 1 < steps; ++i) {
                multiply(st, (s0 + i) * kStep);
                load(st, slab0 + (s0 + i + 1) * kStep);
            }
            multiply(st, (s0 + steps - 1) * kStep);
        }
        // What is left of the slab, 32 k at a time in turns, the codes
        // guarded (A is 0 past K).
        for (int k0 = all * kStep + 32 * wk; k0 < slab_k; k0 += 32 * l.wk) {
            const int group = (slab0 + k0) / p.group, at = (slab0 + k0) / 2 + 4 * kq;
            std::uint32_t w = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) w |= at + i < bytes ? std::uint32_t(wrow[at + i]) << (8 * i) : 0u;
            const Frag wf = Code(ZP ? zrow[group] & 15u : 8u)(w);
            const float s = to_f32<ST>(static_cast<const typename ST::elem *>(p.S)[srow + group]);
            Operand a;
            if constexpr (Held) {
                a = operand(k0);
            } else {
                elem x[8];
                load_a<T>(arow, slab0 + k0 + 8 * kq, p.K, x);
                a.set(x);
            }
            const f32x4 acc = a.times(wf, f32x4{0, 0, 0, 0});
#pragma unroll
            for (int r = 0; r < 4; ++r) out[r] += s * acc[r];
        }
        slab0 += slab_k;
    }

    // D of the matrix instruction: lane 16 q + c, register r: row 4 q + r, column c.
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 4; ++r) part[(wave * 16 + 4 * kq + r) * 16 + c] = out[r] * Code::kUnit;
    __syncthreads();
    for (int e = threadIdx.x; e < rows * cols; e += blockDim.x) {
        const int i = e / cols, j = e % cols;
        if (c0 + j >= p.N) continue;
        const float *src = part + (j / 16 * l.wk * 16 + i) * 16 + j % 16;
        float sum = 0.0f;
        for (int w = 0; w < l.wk; ++w) sum += src[w * 256];
        float *dst = p.C + i * p.ldc + c0 + j;
        *dst = p.beta == 0.0f ? p.alpha * sum : __builtin_fmaf(p.alpha, sum, p.beta * *dst);
    }
}

template <class T, class ST, int GS, bool ZP, bool Run> hipError_t launch_rows(const W4Problem &p, const W4Plan &plan, hipStream_t stream)
{
    constexpr int U = sizeof(typename T::elem) == 2 ? 2 : 1, kStep = kW4Chunk * U;
    static_assert(kStep == w4_step(AOperand<T>::kPlanes > 1), "the plan's step");
    const bool straight = plan.slabs == 0;
    W4Layout l{plan.wn, plan.wk, straight ? 1 : plan.slabs, plan.pitch};
    const int steps = p.K / kStep, waves = l.wn * l.wk, width = 16 * l.wn;
    const std::size_t sums = std::size_t(waves) * 1024, shared = std::size_t(plan.held) < sums ? sums : std::size_t(plan.held);
    const std::int64_t tiles_n = (std::int64_t(p.N) + width - 1) / width;
    const void *kernel = steps == 0 ? reinterpret_cast<const void *>(&w4_rows_kernel<T, ST, 1, ZP, U, true, false, true>)
                         : straight ? reinterpret_cast<const void *>(&w4_rows_kernel<T, ST, GS, ZP, U, false, Run, false>)
                                    : reinterpret_cast<const void *>(&w4_rows_kernel<T, ST, GS, ZP, U, false, Run, true>);
    if (shared > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
        if (e != hipSuccess) return e;
    }
    // Bands of columns keep the launch under 2^32 work-items.
    constexpr std::int64_t kBand = std::int64_t(1) << 21;
    for (std::int64_t t0 = 0; t0 < tiles_n; t0 += kBand) {
        const std::int64_t n0 = t0 * width, tn = tiles_n - t0 < kBand ? tiles_n - t0 : kBand;
        W4Problem q = p;
        q.N = int(p.N - n0 < kBand * width ? p.N - n0 : kBand * width);
        q.W = p.W + n0 * p.ldw;
        q.S = static_cast<const char *>(p.S) + n0 * p.lds * (p.stype == SGEMM_F32 ? 4 : 2);
        if (p.Z) q.Z = p.Z + n0 * p.ldz;
        q.C = p.C + n0;
        void *args[] = {&q, &l};
        const hipError_t e = hipLaunchKernel(kernel, dim3(unsigned(tn)), dim3(64 * waves), args, shared, stream);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// Products with more rows, on v_mfma_f32_32x32x16: each wave a tile of 32 MT
// rows by 32 NT columns. A's rows of 128 k at a time (a slab) lie in LDS, the
// next slab's in registers while this one is multiplied; each wave's codes go
// from memory straight to its registers and are converted once for all rows.
// WN > 1: WN waves divide the columns and share the slab (two buffers, one
// barrier a slab). WN == 1: WK waves divide K, each with a buffer of its own
// and no barrier, and add their sums through LDS in their order: for products
// with too few tiles to fill the device.
//
// Within a slab the loops run over groups, then row tiles, then k: a group's
// sum of one row tile is complete, scaled and added to the result before the
// next begins, so that it takes 16 NT registers and not another result tile.
// Lane 32 h + c supplies column (row) c; which k it supplies in a step is free
// as long as both operands agree and stay inside a group: k = 16 GS h + 8 j of
// the group in step j, so that a lane's codes of a group are adjacent.
//
// The matrix cores bound it: what shares their time is the conversion (7
// cycles a code and column, so tall tiles) and the reads of A from LDS (4
// cycles a row and 64 k for four waves against MT NT matrix instructions, so
// wide ones). 2048 x 4096 x 4096 in bf16: 85 us in a run of calls (810
// TFLOP/s), 98 in a replayed graph; matrix instructions take 37% of the cycles
// a compute unit is busy, the other vector instructions 53%. 128 x 64 a wave,
// one wave a SIMD: 121 us; 16x16x32 instructions: 571.
// The shared-slab tile takes all 256 registers of two waves a SIMD: with 16-bit
// rows it spills 5 to 20 vector registers (24 to 84 bytes of scratch a lane) for
// groups of 128 and more, 1 to 15 for groups of 32 or 96 with zero points, none
// for the others; float32 rows have a SIMD to themselves and spill none.
typedef __attribute__((ext_vector_type(16))) float f32x16;
template <class T> __device__ inline f32x16 mfma32(const Frag &a, const Frag &b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a.v), __builtin_bit_cast(bf16x8, b.v), c, 0, 0, 0);
}
template <> __device__ inline f32x16 mfma32<F16>(const Frag &a, const Frag &b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a.v), __builtin_bit_cast(f16x8, b.v), c, 0, 0, 0);
}

constexpr int kTilePitch = 2 * kW4Chunk + 16;  // bytes of a row of A's slab in LDS: 8 rows meet in no bank

template <class T, int MT, int NT, int WN, int WK> constexpr int tile_lds()
{
    const int slabs = (WN > 1 ? 2 : WK) * AOperand<T>::kPlanes * 32 * MT * kTilePitch, sums = WK > 1 ? WK * MT * NT * 4096 : 0;
    return slabs > sums ? slabs : sums;
}

template <class T, int MT, int NT, int GS, bool ZP, bool Run, int WN, int WK>
__global__ __launch_bounds__(64 * WN * WK, WN > 1 && AOperand<T>::kPlanes == 1 ? 2 : 1) void w4_tile_kernel(W4Problem p, int tiles_m)
{
    static_assert(WN == 1 || WK == 1, "waves divide the columns or K");
    extern __shared__ __align__(16) char lds[];  // [buffer][plane][row][k]
    typedef typename T::elem elem;
    typedef AOperand<T> Operand;
    typedef Codes<T, ZP> Code;
    constexpr int kPlanes = Operand::kPlanes, BM = 32 * MT, BN = 32 * NT * WN, kPieces = BM * 16 / (64 * WN);
    constexpr int kBuffer = kPlanes * BM * kTilePitch;
    const int lane = threadIdx.x & 63, c = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = WN > 1 ? wave : 0, wk = WN > 1 ? 0 : wave;
    const std::int64_t m0 = std::int64_t(blockIdx.x % unsigned(tiles_m)) * BM;
    const std::int64_t c0 = std::int64_t(blockIdx.x / unsigned(tiles_m)) * BN, n0 = c0 + wn * (32 * NT);
    const int bytes = p.K / 2 + p.K % 2;

    const std::uint8_t *wrow[NT], *zrow[NT];
    std::int64_t srow[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        // Columns (and rows) past the last read it again; they are not stored.
        const std::int64_t n = n0 + 32 * t + c < p.N ? n0 + 32 * t + c : p.N - 1;
        wrow[t] = p.W + n * p.ldw;
        srow[t] = n * p.lds;
        zrow[t] = ZP ? p.Z + n * p.ldz : nullptr;
    }
    // A's slab in pieces of 8 k: a thread takes piece t % 16 of rows t / 16, t / 16 + 4 WN, ...
    const int piece = threadIdx.x & 15, prow = (WN > 1 ? threadIdx.x : lane) >> 4;
    const elem *arow[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const std::int64_t r = m0 + prow + 4 * WN * i < p.M ? m0 + prow + 4 * WN * i : p.M - 1;
        arow[i] = static_cast<const elem *>(p.A) + r * p.lda;
    }
    struct Eight {
        elem x[8];
    };
    Eight araw[kPieces];
    std::uint32_t w[NT][16];  // a lane's codes: word 2 GS g + j holds k = 32 GS g + 16 GS h + 8 j
    AnyGroups<GS, 4 / GS, ZP, Run> groups[NT];
    f32x16 out[MT][NT] = {};

    auto load = [&](int k0, auto tail) {
        constexpr bool Tail = decltype(tail)::value;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            if constexpr (Tail) {
                load_a<T>(arow[i], k0 + 8 * piece, p.K, araw[i].x);
            } else {
                araw[i] = load_any<Eight>(arow[i] + k0 + 8 * piece);
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int g = 0; g < 4 / GS; ++g) {
                const int at = k0 / 2 + 16 * GS * g + 8 * GS * h;
                if constexpr (Tail) {
#pragma unroll
                    for (int j = 0; j < 2 * GS; ++j) {
                        std::uint32_t x = 0;
#pragma unroll
                        for (int i = 0; i < 4; ++i) x |= at + 4 * j + i < bytes ? std::uint32_t(wrow[t][at + 4 * j + i]) << (8 * i) : 0u;
                        w[t][2 * GS * g + j] = x;
                    }
                } else {
                    const Words<2 * GS> x = load_any<Words<2 * GS>>(wrow[t] + at);
#pragma unroll
                    for (int j = 0; j < 2 * GS; ++j) w[t][2 * GS * g + j] = x.v[j];
                }
            }
            if constexpr (Tail) {
                groups[t].load_last(p, srow[t], zrow[t], k0);
            } else {
                groups[t].load(p, srow[t], zrow[t], k0);
            }
        }
    };
    // A wave with a buffer of its own writes what its other lanes read: the
    // hardware runs one wave's LDS accesses in order, the fences keep the
    // compiler to that order (no instruction). WN > 1 has the barrier.
    auto own_order = [] {
        if constexpr (WN == 1) {
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
            __builtin_amdgcn_wave_barrier();
        }
    };
    auto hold = [&](char *buffer) {
        own_order();
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            Operand a;
            a.set(araw[i].x);
#pragma unroll
            for (int f = 0; f < kPlanes; ++f)
                *reinterpret_cast<u32x4 *>(buffer + (f * BM + prow + 4 * WN * i) * kTilePitch + 16 * piece) = a.f[f].v;
        }
        own_order();
    };

    const int slabs = (p.K + kW4Chunk - 1) / kW4Chunk, whole = p.K / kW4Chunk;
    const int first = int(std::int64_t(slabs) * wk / WK), end = int(std::int64_t(slabs) * (wk + 1) / WK);
    char *const own = lds + wk * kBuffer;
    if (first < end) {
        if (first < whole) {
            load(first * kW4Chunk, std::false_type{});
        } else {
            load(first * kW4Chunk, std::true_type{});
        }
        hold(own);
    }
    for (int s = first; s < end; ++s) {
        if (WN > 1) __syncthreads();  // this slab is in LDS; the one before has been read
        const char *const buffer = own + (WN > 1 ? (s - first) % 2 * kBuffer : 0) + c * kTilePitch + 32 * GS * h;
        // The slab's operands and scales, then (their registers free) the next slab's loads.
        Frag b[NT][8];
        float scale[NT][4 / GS];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int g = 0; g < 4 / GS; ++g) {
                scale[t][g] = groups[t].scale(g, p.stype);
#pragma unroll
                for (int j = 0; j < 2 * GS; ++j) b[t][2 * GS * g + j] = Code(groups[t].zero(g))(w[t][2 * GS * g + j]);
            }
        if (s + 1 < end) {
            if (s + 1 < whole) {
                load((s + 1) * kW4Chunk, std::false_type{});
            } else {
                load((s + 1) * kW4Chunk, std::true_type{});
            }
        }
#pragma unroll
        for (int g = 0; g < 4 / GS; ++g)
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                f32x16 acc[NT];
#pragma unroll
                for (int j = 0; j < 2 * GS; ++j) {
#pragma unroll
                    for (int f = kPlanes - 1; f >= 0; --f) {
                        Frag a;
                        a.v = *reinterpret_cast<const u32x4 *>(buffer + (f * BM + 32 * i) * kTilePitch + 64 * GS * g + 16 * j);
#pragma unroll
                        for (int t = 0; t < NT; ++t)
                            acc[t] = mfma32<T>(a, b[t][2 * GS * g + j], j == 0 && f == kPlanes - 1 ? f32x16{} : acc[t]);
                    }
                }
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int r = 0; r < 16; ++r) out[i][t][r] += scale[t][g] * acc[t][r];
                if (GS < 4) {
                    // Without a fence the compiler keeps many short groups' sums at once and spills.
#pragma unroll
                    for (int t = 0; t < NT; ++t) asm volatile("" : "+v"(out[i][t]));
                }
            }
        if (s + 1 < end) hold(own + (WN > 1 ? (s + 1 - first) % 2 * kBuffer : 0));
    }
    // D: lane 32 h + c, register r: row 8 (r / 4) + 4 h + r % 4, column c.
    auto store = [&](std::int64_t m, std::int64_t n, float x) {
        float *dst = p.C + m * p.ldc + n;
        x *= Code::kUnit;
        *dst = p.beta == 0.0f ? p.alpha * x : __builtin_fmaf(p.alpha, x, p.beta * *dst);
    };
    if constexpr (WK > 1) {
        float *const part = reinterpret_cast<float *>(lds);  // [wave][row][column]
        __syncthreads();
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    part[(wk * BM + 32 * i + 8 * (r / 4) + 4 * h + r % 4) * BN + 32 * t + c] = out[i][t][r];
        __syncthreads();
        for (int e = threadIdx.x; e < BM * BN; e += 64 * WK) {
            const std::int64_t m = m0 + e / BN, n = c0 + e % BN;
            if (m >= p.M || n >= p.N) continue;
            float sum = 0.0f;
#pragma unroll
            for (int x = 0; x < WK; ++x) sum += part[x * BM * BN + e];
            store(m, n, sum);
        }
    } else {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const std::int64_t n = n0 + 32 * t + c;
            if (n >= p.N) continue;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const std::int64_t m = m0 + 32 * i + 8 * (r / 4) + 4 * h + r % 4;
                    if (m < p.M) store(m, n, out[i][t][r]);
                }
        }
    }
}

template <class T, int MT, int NT, int GS, bool ZP, bool Run, int WN, int WK>
hipError_t launch_tile_shape(const W4Problem &p, hipStream_t stream)
{
    constexpr int BM = 32 * MT, BN = 32 * NT * WN, kLds = tile_lds<T, MT, NT, WN, WK>();
    static_assert(kLds <= 160 * 1024, "fits the LDS");
    const void *kernel = reinterpret_cast<const void *>(&w4_tile_kernel<T, MT, NT, GS, ZP, Run, WN, WK>);
    if (kLds > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
        if (e != hipSuccess) return e;
    }
    // Bands of rows and columns keep the launch under 2^32 work-items.
    constexpr std::int64_t kBand = 2048;
    for (std::int64_t r0 = 0; r0 < p.M; r0 += kBand * BM)
        for (std::int64_t c0 = 0; c0 < p.N; c0 += kBand * BN) {
            W4Problem q = p;
            q.M = int(p.M - r0 < kBand * BM ? p.M - r0 : kBand * BM);
            q.N = int(p.N - c0 < kBand * BN ? p.N - c0 : kBand * BN);
            q.A = static_cast<const char *>(p.A) + r0 * p.lda * std::int64_t(sizeof(typename T::elem));
            q.W = p.W + c0 * p.ldw;
            q.S = static_cast<const char *>(p.S) + c0 * p.lds * (p.stype == SGEMM_F32 ? 4 : 2);
            if (p.Z) q.Z = p.Z + c0 * p.ldz;
            q.C = p.C + r0 * p.ldc + c0;
            int tiles_m = (q.M + BM - 1) / BM;
            const int tiles_n = (q.N + BN - 1) / BN;
            void *args[] = {&q, &tiles_m};
            const hipError_t e = hipLaunchKernel(kernel, dim3(unsigned(tiles_m) * unsigned(tiles_n)), dim3(64 * WN * WK), args, kLds, stream);
            if (e != hipSuccess) return e;
        }
    return hipSuccess;
}

template <class T, int GS, bool ZP, bool Run> hipError_t launch_tile(const W4Problem &p, const W4Plan &plan, hipStream_t stream)
{
    if (plan.wn == 4) return launch_tile_shape<T, 2, 2, GS, ZP, Run, 4, 1>(p, stream);
    if constexpr (AOperand<T>::kPlanes == 1) {
        if (plan.nt == 2) return launch_tile_shape<T, 2, 2, GS, ZP, Run, 1, 4>(p, stream);
        if (plan.mt == 2) return launch_tile_shape<T, 2, 1, GS, ZP, Run, 1, 8>(p, stream);
        return launch_tile_shape<T, 1, 1, GS, ZP, Run, 1, 8>(p, stream);
    } else {
        return launch_tile_shape<T, 1, 1, GS, ZP, Run, 1, 4>(p, stream);
    }
}

// k whose groups one wave adds up in one float32 sum at most: up to 2048 terms.
// A longer sum would take on the roundings of all its terms, and stop growing
// from 2^24 of them on.
constexpr std::int64_t kW4SumK = 1 << 16;

template <class T, class ST, int GS, bool ZP, bool Run> hipError_t launch_shape(const W4Problem &p, hipStream_t stream)
{
    const int dtype = std::is_same<T, F32>::value ? SGEMM_F32 : std::is_same<T, BF16>::value ? SGEMM_LP_BF16 : SGEMM_LP_F16;
    const W4Plan plan = plan_w4(dtype, p.M, p.N, p.K, p.cus);
    const std::int64_t most = kW4SumK * plan.wk;
    if (p.K <= most) return plan.few ? launch_rows<T, ST, GS, ZP, Run>(p, plan, stream) : launch_tile<T, GS, ZP, Run>(p, plan, stream);
    // Longer K in pieces, each added to C: they end where a group ends, or lie inside one.
    for (std::int64_t k0 = 0; k0 < p.K;) {
        const std::int64_t left = p.group - k0 % p.group, inside = left < most ? left : most;
        std::int64_t n = k0 % p.group != 0 || p.group > most ? inside : most / p.group * p.group;
        if (n > p.K - k0) n = p.K - k0;
        W4Problem q = p;
        q.K = int(n);
        q.A = static_cast<const char *>(p.A) + k0 * std::int64_t(sizeof(typename T::elem));
        q.W = p.W + k0 / 2;  // k0 is a multiple of 32
        q.S = static_cast<const char *>(p.S) + k0 / p.group * (p.stype == SGEMM_F32 ? 4 : 2);
        if (p.Z) q.Z = p.Z + k0 / p.group;
        if (k0 > 0) q.beta = 1.0f;
        const W4Plan part = plan_w4(dtype, p.M, p.N, q.K, p.cus);
        const hipError_t e = part.few ? launch_rows<T, ST, GS, ZP, Run>(q, part, stream) : launch_tile<T, GS, ZP, Run>(q, part, stream);
        if (e != hipSuccess) return e;
        k0 += n;
    }
    return hipSuccess;
}

template <class T, class ST, bool ZP> hipError_t launch_group(const W4Problem &p, hipStream_t stream)
{
    switch (p.group) {
    case 32: return launch_shape<T, ST, 1, ZP, true>(p, stream);
    case 64: return launch_shape<T, ST, 2, ZP, true>(p, stream);
    case 128: return launch_shape<T, ST, 4, ZP, true>(p, stream);
    }
    return p.group % 128 == 0 ? launch_shape<T, ST, 4, ZP, false>(p, stream) : launch_shape<T, ST, 1, ZP, false>(p, stream);
}

template <class T, class ST> hipError_t launch_zeros(const W4Problem &p, hipStream_t stream)
{
    return p.Z ? launch_group<T, ST, true>(p, stream) : launch_group<T, ST, false>(p, stream);
}

template <class T> hipError_t launch_w4(const W4Problem &p, hipStream_t stream)
{
    return p.stype == SGEMM_F32       ? launch_zeros<T, F32>(p, stream)
           : p.stype == SGEMM_LP_BF16 ? launch_zeros<T, BF16>(p, stream)
                                      : launch_zeros<T, F16>(p, stream);
}

}  // namespace
}  // namespace sgemm_impl
