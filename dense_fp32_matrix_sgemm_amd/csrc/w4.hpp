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

#include "lowbit.hpp"

namespace sgemm_impl {
namespace {

constexpr int kW4Chunk = 128;  // k that a wave takes at a time: 16 bytes of codes a lane

// Eight codes of one word as exact 16-bit numbers. `z` is the zero point
// prepared by w4_zero. The order of k within the eight is the type's own:
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
            std::uint32_t even = (((w & 0x0f0f0f0fu) | 0x80808080u) - z4) ^ 0x80808080u;
            std::uint32_t odd = ((((w >> 4) & 0x0f0f0f0fu) | 0x80808080u) - z4) ^ 0x80808080u;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = float(int(std::int8_t(even >> (8 * i))));
                f[2 * i + 1] = float(int(std::int8_t(odd >> (8 * i))));
            }
        } else {
            const std::uint32_t even = w ^ 0x88888888u;
            const std::uint32_t odd = even >> 4;
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
    f16x2 lo, hi;  // -(1024 + z), -(64 + z)
    __device__ explicit Codes(std::uint32_t z)
    {
        const _Float16 a = _Float16(-1024.0f - float(z)), b = _Float16(-64.0f - float(z));
        lo = f16x2{a, a};
        hi = f16x2{b, b};
    }
    __device__ Frag operator()(std::uint32_t w) const
    {
        const f16x2 sixteenth = {_Float16(0.0625f), _Float16(0.0625f)};
        Frag r;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const std::uint32_t x = w >> (8 * i);
            const f16x2 a = __builtin_bit_cast(f16x2, (x & 0x000f000fu) | 0x64006400u) + lo;
            const f16x2 b = __builtin_bit_cast(f16x2, (x & 0x00f000f0u) | 0x64006400u) * sixteenth + hi;
            r.v[2 * i] = __builtin_bit_cast(std::uint32_t, a);      // codes 2i, 2i + 4
            r.v[2 * i + 1] = __builtin_bit_cast(std::uint32_t, b);  // codes 2i + 1, 2i + 5
        }
        return r;
    }
};

// One lane's eight elements of A's row, as loaded (Raw), and as operands of
// the matrix instruction.
template <class T> struct AOperand;
template <> struct AOperand<BF16> {
    struct Raw {
        u32x4 v;
    };
    Frag f;
    __device__ explicit AOperand(const Raw &r) { f.v = r.v; }
    __device__ f32x4 times(const Frag &w, f32x4 acc) const { return mfma_bf16(f, w, acc); }
};
template <> struct AOperand<F16> {
    struct Raw {
        u32x4 v;
    };
    Frag f;
    __device__ explicit AOperand(const Raw &r)
    {
        // (a0 a1)(a2 a3)(a4 a5)(a6 a7) -> (a0 a4)(a1 a5)(a2 a6)(a3 a7), the codes' order.
        f.v[0] = __builtin_amdgcn_perm(r.v[2], r.v[0], 0x05040100u);
        f.v[1] = __builtin_amdgcn_perm(r.v[2], r.v[0], 0x07060302u);
        f.v[2] = __builtin_amdgcn_perm(r.v[3], r.v[1], 0x05040100u);
        f.v[3] = __builtin_amdgcn_perm(r.v[3], r.v[1], 0x07060302u);
    }
    __device__ f32x4 times(const Frag &w, f32x4 acc) const { return mfma_f16(f, w, acc); }
};
template <> struct AOperand<F32> {
    struct Raw {
        float v[8];
    };
    Frag hi, mid, lo;
    __device__ explicit AOperand(const Raw &r) { split3(r.v, hi, mid, lo); }
    __device__ f32x4 times(const Frag &w, f32x4 acc) const
    {
        return mfma_bf16(hi, w, mfma_bf16(mid, w, mfma_bf16(lo, w, acc)));
    }
};

// Eight elements of a row from k on; zeros from K on when Tail (a partial
// chunk), and everywhere when the row is not there.
template <class T, bool Tail>
__device__ inline typename AOperand<T>::Raw load_a(const typename T::elem *row, std::int64_t k, int K, bool there)
{
    typedef typename AOperand<T>::Raw Raw;
    Raw r;
    __builtin_memset(&r, 0, sizeof(Raw));
    if (!there) return r;
    if (!Tail || k + 8 <= K) return load_any<Raw>(row + k);
    typename T::elem e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = k + i < K ? row[k + i] : typename T::elem(0);
    __builtin_memcpy(&r, e, sizeof(Raw));
    return r;
}

// Sixteen bytes of a row of codes; zeros from the row's end on when Tail.
template <bool Tail> __device__ inline u32x4 load_codes(const std::uint8_t *row, std::int64_t at, int bytes)
{
    if (!Tail || at + 16 <= bytes) return load_any<u32x4>(row + at);
    u32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (at + i < bytes) v[i / 4] |= std::uint32_t(row[at + i]) << (8 * (i % 4));
    return v;
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

// One work-group: 16 MT rows of C by 16 NT columns. Its waves take K in
// chunks of 128 in turn, each lane 16 bytes of one of its 16 columns' codes
// (64 adjacent bytes a column), every A operand used for NT column tiles;
// the waves' sums are added through LDS in the waves' order, so the result
// does not depend on timing. GS: steps of 32 k that share a scale.
template <class T, int MT, int NT, int GS, bool ZP>
__global__ __launch_bounds__(1024) void w4_rows_kernel(W4Problem p)
{
    extern __shared__ float part[];  // [wave][16 MT][16 NT]
    typedef typename T::elem elem;
    const int lane = threadIdx.x & 63, c = lane & 15, kq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const std::int64_t n0 = std::int64_t(blockIdx.x) * (16 * NT);
    const int bytes = (p.K + 1) / 2;

    const std::uint8_t *wrow[NT];
    std::int64_t srow[NT], zrow[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        // Columns past the last read it again; their sums are not stored.
        const std::int64_t n = n0 + 16 * t + c < p.N ? n0 + 16 * t + c : p.N - 1;
        wrow[t] = p.W + n * p.ldw;
        srow[t] = n * p.lds;
        zrow[t] = n * p.ldz;
    }
    for (std::int64_t m0 = std::int64_t(blockIdx.y) * (16 * MT); m0 < p.M; m0 += std::int64_t(gridDim.y) * (16 * MT)) {
        const elem *arow[MT];
        bool there[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            there[t] = m0 + 16 * t + c < p.M;
            arow[t] = static_cast<const elem *>(p.A) + (there[t] ? m0 + 16 * t + c : 0) * p.lda;
        }
        f32x4 out[MT][NT] = {};

        auto chunk = [&](std::int64_t k0, auto tail) {
            constexpr bool Tail = decltype(tail)::value;
            u32x4 w[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) w[t] = steps_of_codes(load_codes<Tail>(wrow[t], k0 / 2 + 16 * kq, bytes));
#pragma unroll
            for (int g = 0; g < 4 / GS; ++g) {
                const std::int64_t k1 = k0 + g * (32 * GS);
                if (Tail && k1 >= p.K) break;
                const int group = int(k1 / p.group);
                f32x4 acc[MT][NT] = {};
#pragma unroll
                for (int s = 0; s < GS; ++s) {
                    typename AOperand<T>::Raw raw[MT];
#pragma unroll
                    for (int i = 0; i < MT; ++i)
                        raw[i] = load_a<T, Tail>(arow[i], k1 + 32 * s + 8 * kq, p.K, there[i]);
                    Frag wf[NT];
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        wf[t] = Codes<T, ZP>(ZP ? p.Z[zrow[t] + group] & 15u : 8u)(w[t][g * GS + s]);
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        const AOperand<T> a(raw[i]);
#pragma unroll
                        for (int t = 0; t < NT; ++t) acc[i][t] = a.times(wf[t], acc[i][t]);
                    }
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const float s = load_scale(p.S, p.stype, srow[t] + group) * Codes<T, ZP>::kUnit;
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int r = 0; r < 4; ++r) out[i][t][r] += s * acc[i][t][r];
                }
            }
        };
        std::int64_t k0 = std::int64_t(wave) * kW4Chunk;
        for (; k0 + kW4Chunk <= p.K; k0 += std::int64_t(waves) * kW4Chunk) chunk(k0, std::false_type{});
        if (k0 < p.K) chunk(k0, std::true_type{});

        // D of the matrix instruction: lane 16 q + c, register r: row 4 q + r, column c.
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    part[(wave * (16 * MT) + 16 * i + 4 * kq + r) * (16 * NT) + 16 * t + c] = out[i][t][r];
        __syncthreads();
        for (int e = threadIdx.x; e < 256 * MT * NT; e += blockDim.x) {
            const int i = e / (16 * NT), j = e % (16 * NT);
            if (m0 + i >= p.M || n0 + j >= p.N) continue;
            float sum = 0.0f;
            for (int w = 0; w < waves; ++w) sum += part[w * (256 * MT * NT) + e];
            float *dst = p.C + (m0 + i) * p.ldc + n0 + j;
            *dst = p.beta == 0.0f ? p.alpha * sum : __builtin_fmaf(p.alpha, sum, p.beta * *dst);
        }
        __syncthreads();
    }
}

template <class T, int MT, int NT, int GS, bool ZP> hipError_t launch_rows(const W4Problem &p, hipStream_t stream)
{
    const std::int64_t tiles_n = (std::int64_t(p.N) + 16 * NT - 1) / (16 * NT);
    const std::int64_t tiles_m = (std::int64_t(p.M) + 16 * MT - 1) / (16 * MT);
    const int chunks = (p.K + kW4Chunk - 1) / kW4Chunk;
    int waves = 4;
    while (waves < 16 && waves < chunks && tiles_n * waves < 16 * std::int64_t(p.cus) && 2 * waves * MT * NT <= 64) waves *= 2;
    // Bands of columns keep the launch under 2^32 work-items.
    constexpr std::int64_t kBand = std::int64_t(1) << 21;
    for (std::int64_t t0 = 0; t0 < tiles_n; t0 += kBand) {
        const std::int64_t n0 = t0 * (16 * NT), tn = tiles_n - t0 < kBand ? tiles_n - t0 : kBand;
        std::int64_t tm = (std::int64_t(1) << 22) / tn / waves;
        tm = tm < 1 ? 1 : tm < 65535 ? tm : 65535;
        W4Problem q = p;
        q.N = int(p.N - n0 < kBand * (16 * NT) ? p.N - n0 : kBand * (16 * NT));
        q.W = p.W + n0 * p.ldw;
        q.S = static_cast<const char *>(p.S) + n0 * p.lds * (p.stype == SGEMM_F32 ? 4 : 2);
        if (p.Z) q.Z = p.Z + n0 * p.ldz;
        q.C = p.C + n0;
        const dim3 grid(unsigned(tn), unsigned(tiles_m < tm ? tiles_m : tm));
        void *args[] = {&q};
        const hipError_t e = hipLaunchKernel(reinterpret_cast<const void *>(&w4_rows_kernel<T, MT, NT, GS, ZP>), grid,
                                             dim3(64 * waves), args, std::size_t(waves) * MT * NT * 1024, stream);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <class T, int GS, bool ZP> hipError_t launch_shape(const W4Problem &p, hipStream_t stream)
{
    return p.M <= 16 ? launch_rows<T, 1, 1, GS, ZP>(p, stream) : launch_rows<T, 4, 1, GS, ZP>(p, stream);
}

template <class T> hipError_t launch_w4(const W4Problem &p, hipStream_t stream)
{
    const bool zp = p.Z != nullptr;
    if (p.group % 128 == 0) return zp ? launch_shape<T, 4, true>(p, stream) : launch_shape<T, 4, false>(p, stream);
    if (p.group % 64 == 0) return zp ? launch_shape<T, 2, true>(p, stream) : launch_shape<T, 2, false>(p, stream);
    return zp ? launch_shape<T, 1, true>(p, stream) : launch_shape<T, 1, false>(p, stream);
}

}  // namespace
}  // namespace sgemm_impl
