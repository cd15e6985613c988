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
// whose upper half is the bf16 number; the 16 goes into the scale. With zero
// points the four bytes of a word's even (odd) nibbles have z subtracted at
// once, each kept from borrowing by its top bit, and are converted as signed
// bytes. Either takes a conversion a code and a v_perm for two.
// f16: a nibble or'ed into the fraction of 1024 is 1024 + q (the next nibble,
// four bits higher, 1024 + 16 q), and one packed add (multiply-add) leaves
// q - z exactly: three instructions for two codes.
template <class T, bool ZP> struct Codes {
    static constexpr float kUnit = ZP ? 1.0f : 16.0f;  // what a code's number has to be multiplied by
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

// N 16-bit scales, likewise.
template <int N> struct Halves {
    Words<N / 2> w;
    __device__ void load(const void *p) { w = load_any<Words<N / 2>>(p); }
    __device__ std::uint16_t at(int i) const { return std::uint16_t(w.v[i / 2] >> (16 * (i % 2))); }
};
template <> struct Halves<1> {
    std::uint16_t w;
    __device__ void load(const void *p) { w = load_any<std::uint16_t>(p); }
    __device__ std::uint16_t at(int) const { return w; }
};

// How a kernel meets the scales. The first three: group == 32 GS, so that a
// wave's scales (of that type) and zero points are adjacent in memory and
// come in one load for U chunks; Any: one load each.
enum class Scales { RunF32, RunBF16, RunF16, Any };

// N scales as loaded.
template <Scales SC, int N> struct ScaleSet {
    typedef typename std::conditional<SC == Scales::RunBF16, BF16, F16>::type T16;
    Halves<N> h;
    __device__ void load(const void *S, std::int64_t i) { h.load(static_cast<const std::uint16_t *>(S) + i); }
    __device__ float at(int i) const { return to_f32<T16>(h.at(i)); }
};
template <int N> struct ScaleSet<Scales::RunF32, N> {
    Words<N> w;
    __device__ void load(const void *S, std::int64_t i) { w = load_any<Words<N>>(static_cast<const float *>(S) + i); }
    __device__ float at(int i) const { return bits_f32(w.v[i]); }
};
template <int N> struct ScaleSet<Scales::Any, N> {
    float f[N];
    __device__ float at(int i) const { return f[i]; }
};

// What a wave loads for U chunks of k.
template <int NT, int GS, int U, Scales SC> struct W4Stage {
    static constexpr int kRuns = 4 * U / GS;  // runs of 32 GS k that share a scale
    u32x4 w[U][NT];
    ScaleSet<SC, kRuns> s[NT];
    Bytes<kRuns> z[NT];
};

// How a product is laid out over work-groups (launch_rows).
struct W4Layout {
    int wn, wk;  // waves along N and along K
    int slabs;   // runs of K whose A is held in LDS, one after the other
    int rows;    // rows of A held, at most 16 MT
    int pitch;   // bytes from one held row to the next: 16 more than a multiple of 128, so that 16 rows meet in no bank
};

// One work-group: 16 MT rows of C by 16 NT wn columns. A slab of A's rows
// lies in LDS as matrix operands, read by every wave; the codes go from
// memory to registers once: each wave takes a run of the slab's k for its 16
// NT columns in steps of U chunks of 128, each lane 16 bytes of one column's
// codes per chunk. The wk waves of a column tile add their sums through LDS
// in their order, so the result does not depend on timing. GS: steps of 32 k
// that share a scale.
template <class T, int MT, int NT, int GS, bool ZP, int U, bool Short, Scales SC, int MaxWaves>
__global__ __launch_bounds__(64 * MaxWaves) void w4_rows_kernel(W4Problem p, W4Layout l)
{
    extern __shared__ __align__(16) char lds[];  // A: [plane][row][k] as 16-bit operands
    typedef typename T::elem elem;
    typedef W4Stage<NT, GS, U, SC> Stage;
    typedef AOperand<T> Operand;
    typedef Codes<T, ZP> Code;
    constexpr int kStep = kW4Chunk * U, kPlanes = Operand::kPlanes, kRuns = Stage::kRuns;
    float *const part = reinterpret_cast<float *>(lds);  // then the sums: [wave][16 MT][16 NT]
    const int lane = threadIdx.x & 63, c = lane & 15, kq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wk = wave % l.wk, wn = wave / l.wk, cols = 16 * NT * l.wn;
    const std::int64_t c0 = std::int64_t(blockIdx.x) * cols, n0 = c0 + wn * (16 * NT);
    const int bytes = p.K / 2 + p.K % 2;

    const std::uint8_t *wrow[NT], *zrow[NT];
    std::int64_t srow[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        // Columns past the last read it again; their sums are not stored.
        const std::int64_t n = n0 + 16 * t + c < p.N ? n0 + 16 * t + c : p.N - 1;
        wrow[t] = p.W + n * p.ldw;
        srow[t] = n * p.lds;
        zrow[t] = ZP ? p.Z + n * p.ldz : nullptr;
    }

    auto load = [&](Stage &st, unsigned k0) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int t = 0; t < NT; ++t) st.w[u][t] = load_any<u32x4>(wrow[t] + (k0 / 2 + 64 * u + 16 * kq));
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if constexpr (SC != Scales::Any) {
                const unsigned g0 = k0 / (32u * GS);
                st.s[t].load(p.S, srow[t] + g0);
                if (ZP) st.z[t].load(zrow[t] + g0);
            } else {
                std::uint8_t z[(kRuns + 3) / 4 * 4] = {};
#pragma unroll
                for (int g = 0; g < kRuns; ++g) {
                    const unsigned group = (k0 + g * (32 * GS)) / unsigned(p.group);
                    st.s[t].f[g] = load_scale(p.S, p.stype, srow[t] + group);
                    if (ZP) z[g] = zrow[t][group];
                }
                if (ZP) __builtin_memcpy(&st.z[t], z, sizeof(st.z[t]));
            }
        }
    };

    for (std::int64_t m0 = std::int64_t(blockIdx.y) * (16 * MT); m0 < p.M; m0 += std::int64_t(gridDim.y) * (16 * MT)) {
        const int rows = p.M - m0 < l.rows ? int(p.M - m0) : l.rows;
        const char *arow[kPlanes][MT];  // rows past the last repeat it; their sums are not stored
#pragma unroll
        for (int f = 0; f < kPlanes; ++f)
#pragma unroll
            for (int i = 0; i < MT; ++i) arow[f][i] = lds + (f * l.rows + (16 * i + c < rows ? 16 * i + c : rows - 1)) * l.pitch + 16 * kq;
        f32x4 out[MT][NT] = {};

        auto operand = [&](int k, int i) {  // A's operand of the step of 32 that starts at k of the slab
            Operand a;
#pragma unroll
            for (int f = 0; f < kPlanes; ++f) a.f[f].v = *reinterpret_cast<const u32x4 *>(arow[f][i] + 2 * k);
            return a;
        };
        auto multiply = [&](const Stage &st, int k0) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                u32x4 w[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t) w[t] = steps_of_codes(st.w[u][t]);
#pragma unroll
                for (int g = 0; g < 4 / GS; ++g) {
                    const int run = u * (4 / GS) + g;
                    f32x4 acc[MT][NT];
#pragma unroll
                    for (int s = 0; s < GS; ++s) {
                        Frag wf[NT];
#pragma unroll
                        for (int t = 0; t < NT; ++t) wf[t] = Code(ZP ? st.z[t].at(run) & 15u : 8u)(w[t][g * GS + s]);
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            const Operand a = operand(k0 + 128 * u + 32 * (g * GS + s), i);
#pragma unroll
                            for (int t = 0; t < NT; ++t) acc[i][t] = a.times(wf[t], s == 0 ? f32x4{0, 0, 0, 0} : acc[i][t]);
                        }
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const float s = st.s[t].at(run) * Code::kUnit;
#pragma unroll
                        for (int i = 0; i < MT; ++i)
#pragma unroll
                            for (int r = 0; r < 4; ++r) out[i][t][r] += s * acc[i][t][r];
                    }
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

            if (j > 0 || m0 >= 16 * MT) __syncthreads();  // the last slab (or sums) in LDS has been read
            const int eights = (slab_k + 31) / 32 * 4;
            for (int e = threadIdx.x; e < rows * eights; e += blockDim.x) {
                const int r = e / eights, at = e % eights;
                elem x[8];
                load_a<T>(static_cast<const elem *>(p.A) + (m0 + r) * p.lda + slab0, 8 * at, slab_k, x);
                Operand a;
                a.set(x);
#pragma unroll
                for (int f = 0; f < kPlanes; ++f) *reinterpret_cast<u32x4 *>(lds + (f * l.rows + r) * l.pitch + 16 * at) = a.f[f].v;
            }
            __syncthreads();

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
                Frag wf[NT];
                float s[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    std::uint32_t w = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) w |= at + i < bytes ? std::uint32_t(wrow[t][at + i]) << (8 * i) : 0u;
                    wf[t] = Code(ZP ? zrow[t][group] & 15u : 8u)(w);
                    s[t] = load_scale(p.S, p.stype, srow[t] + group) * Code::kUnit;
                }
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const Operand a = operand(k0, i);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const f32x4 acc = a.times(wf[t], f32x4{0, 0, 0, 0});
#pragma unroll
                        for (int r = 0; r < 4; ++r) out[i][t][r] += s[t] * acc[r];
                    }
                }
            }
            slab0 += slab_k;
        }

        // D of the matrix instruction: lane 16 q + c, register r: row 4 q + r, column c.
        __syncthreads();
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    part[(wave * (16 * MT) + 16 * i + 4 * kq + r) * (16 * NT) + 16 * t + c] = out[i][t][r];
        __syncthreads();
        for (int e = threadIdx.x; e < rows * cols; e += blockDim.x) {
            const int i = e / cols, j = e % cols;
            if (c0 + j >= p.N) continue;
            const float *src = part + (j / (16 * NT) * l.wk * (16 * MT) + i) * (16 * NT) + j % (16 * NT);
            float sum = 0.0f;
            for (int w = 0; w < l.wk; ++w) sum += src[w * (256 * MT * NT)];
            float *dst = p.C + (m0 + i) * p.ldc + c0 + j;
            *dst = p.beta == 0.0f ? p.alpha * sum : __builtin_fmaf(p.alpha, sum, p.beta * *dst);
        }
    }
}

template <class T, int MT, int NT, int GS, bool ZP, Scales SC> hipError_t launch_rows(const W4Problem &p, hipStream_t stream)
{
    constexpr int U = MT * NT <= 2 && sizeof(typename T::elem) == 2 ? 2 : 1, kStep = kW4Chunk * U, kWaves = MT * NT <= 2 ? 16 : 8;
    constexpr std::int64_t kLds = 160 * 1024;
    const std::int64_t tiles_m = (std::int64_t(p.M) + 16 * MT - 1) / (16 * MT);
    W4Layout l;
    l.rows = p.M < 16 * MT ? p.M : 16 * MT;
    // Waves along K while there are too few columns to fill the device.
    std::int64_t tiles_n = (std::int64_t(p.N) + 16 * NT - 1) / (16 * NT);
    l.wn = 1;
    while (l.wn < 4 && tiles_n >= 2 * l.wn * std::int64_t(p.cus)) l.wn *= 2;
    // K in as few slabs as the LDS holds, of even length, each with a whole
    // step for every wave. (A slab of one step and the rest always fits: 64
    // float32 rows take 100 KB of it.)
    const int steps = p.K / kStep, rest = p.K % kStep;
    const auto held = [&](std::int64_t slab_steps) {
        l.pitch = int((2 * (slab_steps * kStep + (rest + 31) / 32 * 32) + 127) / 128 * 128 + 16);
        return AOperand<T>::kPlanes * l.rows * std::int64_t(l.pitch);
    };
    l.slabs = 1;
    while (l.slabs < steps && held((std::int64_t(steps) + l.slabs - 1) / l.slabs) > kLds) ++l.slabs;
    std::size_t shared = std::size_t(held((std::int64_t(steps) + l.slabs - 1) / l.slabs));
    l.wk = 1;
    while (2 * l.wk * l.wn <= kWaves && 2 * l.wk <= steps / l.slabs) l.wk *= 2;
    const int waves = l.wn * l.wk, width = 16 * NT * l.wn;
    const std::size_t sums = std::size_t(waves) * MT * NT * 1024;
    if (shared < sums) shared = sums;
    tiles_n = (tiles_n + l.wn - 1) / l.wn;
    const void *kernel = steps > 0 ? reinterpret_cast<const void *>(&w4_rows_kernel<T, MT, NT, GS, ZP, U, false, SC, kWaves>)
                                   : reinterpret_cast<const void *>(&w4_rows_kernel<T, MT, NT, 1, ZP, U, true, Scales::Any, kWaves>);
    if (shared > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, int(kLds));
        if (e != hipSuccess) return e;
    }
    // Bands of columns keep the launch under 2^32 work-items.
    constexpr std::int64_t kBand = std::int64_t(1) << 21;
    for (std::int64_t t0 = 0; t0 < tiles_n; t0 += kBand) {
        const std::int64_t n0 = t0 * width, tn = tiles_n - t0 < kBand ? tiles_n - t0 : kBand;
        std::int64_t tm = (std::int64_t(1) << 22) / tn / waves;
        tm = tm < 1 ? 1 : tm < 65535 ? tm : 65535;
        W4Problem q = p;
        q.N = int(p.N - n0 < kBand * width ? p.N - n0 : kBand * width);
        q.W = p.W + n0 * p.ldw;
        q.S = static_cast<const char *>(p.S) + n0 * p.lds * (p.stype == SGEMM_F32 ? 4 : 2);
        if (p.Z) q.Z = p.Z + n0 * p.ldz;
        q.C = p.C + n0;
        const dim3 grid(unsigned(tn), unsigned(tiles_m < tm ? tiles_m : tm));
        void *args[] = {&q, &l};
        const hipError_t e = hipLaunchKernel(kernel, grid, dim3(64 * waves), args, shared, stream);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <class T, int GS, bool ZP, Scales SC> hipError_t launch_shape(const W4Problem &p, hipStream_t stream)
{
    if (p.M <= 16) return launch_rows<T, 1, 1, GS, ZP, SC>(p, stream);
    return p.M <= 32 ? launch_rows<T, 2, 1, GS, ZP, SC>(p, stream) : launch_rows<T, 4, 1, GS, ZP, SC>(p, stream);
}

template <class T, int GS, bool ZP> hipError_t launch_run(const W4Problem &p, hipStream_t stream)
{
    return p.stype == SGEMM_F32       ? launch_shape<T, GS, ZP, Scales::RunF32>(p, stream)
           : p.stype == SGEMM_LP_BF16 ? launch_shape<T, GS, ZP, Scales::RunBF16>(p, stream)
                                      : launch_shape<T, GS, ZP, Scales::RunF16>(p, stream);
}

template <class T, bool ZP> hipError_t launch_group(const W4Problem &p, hipStream_t stream)
{
    switch (p.group) {
    case 32: return launch_run<T, 1, ZP>(p, stream);
    case 64: return launch_run<T, 2, ZP>(p, stream);
    case 128: return launch_run<T, 4, ZP>(p, stream);
    }
    return p.group % 128 == 0 ? launch_shape<T, 4, ZP, Scales::Any>(p, stream) : launch_shape<T, 1, ZP, Scales::Any>(p, stream);
}

template <class T> hipError_t launch_w4(const W4Problem &p, hipStream_t stream)
{
    return p.Z ? launch_group<T, true>(p, stream) : launch_group<T, false>(p, stream);
}

}  // namespace
}  // namespace sgemm_impl
