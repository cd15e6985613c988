// Quantising a matrix to the W4 form (sgemm_w4_quantize) and reading it back
// (sgemm_w4_dequantize). Each matrix is moved once. 4096 x 4096 in bf16 (42
// MB, 8.2 us at the 5.1 TB/s of a large copy): quantising takes 16.3 us, bound
// by its arithmetic (8600 vector instructions a SIMD, at four cycles each most
// of that time); reading back 14.2 us, 2.9 TB/s, with 3400 instructions a SIMD
// (105 for eight elements, the run-time divisions for the most part): neither
// the memory nor the instructions are used up, and a launch of 14 us has
// little time at its full rate.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "lowbit.hpp"

namespace sgemm_impl {
namespace {

constexpr int kThreads = 256;

template <class T> struct Eight {
    typename T::elem x[8];
};

// Eight elements of a row from k on as float32; zeros from the row's end on.
template <class T> __device__ inline void load8(const typename T::elem *row, int k, int K, float *x)
{
    Eight<T> v;
    if (k + 8 <= K) {
        v = load_any<Eight<T>>(row + k);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v.x[i] = k + i < K ? row[k + i] : typename T::elem(0);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_f32<T>(v.x[i]);
}

__device__ inline float store_scale(void *S, int stype, std::int64_t i, float s)
{
    if (stype == SGEMM_F32) {
        static_cast<float *>(S)[i] = s;
        return s;
    }
    const std::uint16_t b = stype == SGEMM_LP_BF16 ? from_f32<BF16>(s) : from_f32<F16>(s);
    static_cast<std::uint16_t *>(S)[i] = b;
    return stype == SGEMM_LP_BF16 ? to_f32<BF16>(b) : to_f32<F16>(b);
}

// round(x / s) with ties to even, as if the quotient were exact, for |x / s|
// up to 32 or so, of N values: the float32 quotient may round onto or over a
// tie, so its nearest integer r is held against the exact remainder x - r s
// (one fused multiply-add; next to a tie it is a multiple of x's or s's last
// place and fits float32). Only a remainder of half of s or more needs the
// correction, which is rare and left to a branch.
template <int N> __device__ inline void rounded_quotients(const float *x, float s, float inverse, float *r)
{
    const float half = 0.5f * s;
    float d[N], worst = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        r[i] = __builtin_rintf(x[i] * inverse);
        d[i] = __builtin_fmaf(-r[i], s, x[i]);
        worst = __builtin_fmaxf(worst, __builtin_fabsf(d[i]));
    }
    if (worst < half) return;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const bool odd = (int(r[i]) & 1) != 0;
        if (d[i] > half || (d[i] == half && odd)) r[i] += 1.0f;
        else if (d[i] < -half || (d[i] == -half && odd)) r[i] -= 1.0f;
    }
}

// LG lanes (a power of two) share one group and take eight k each in turn.
// Once: group == 8 LG, so that a lane's eight stay in registers between the
// search for the extremes and the rounding. `all` groups, fewer than 2^31.
template <class T, int LG, bool ZP, bool Once>
__global__ __launch_bounds__(kThreads) void w4_quantize_kernel(W4PackProblem p, unsigned groups, unsigned all)
{
    const int part = threadIdx.x % LG;
    for (unsigned id = blockIdx.x * (kThreads / LG) + threadIdx.x / LG; id < all; id += gridDim.x * (kThreads / LG)) {
        const std::int64_t n = id / groups;
        const int g = int(id % groups);
        const int k0 = g * p.group, k1 = p.K - k0 < p.group ? p.K : k0 + p.group;
        const typename T::elem *row = static_cast<const typename T::elem *>(p.B) + n * p.ldb;
        // The largest and the least of the values and 0 by their bits: as
        // signed numbers positive floats are in order and above the negative,
        // as unsigned ones negative floats lie above the positive, the largest
        // magnitude on top. What is not finite ends above either range.
        int top = 0;
        std::uint32_t bottom = 0x80000000u;
        float x[8];
        for (int k = k0 + 8 * part; k < k1; k += 8 * LG) {
            load8<T>(row, k, k1, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const std::uint32_t bits = f32_bits(x[i]);
                top = int(bits) > top ? int(bits) : top;
                bottom = bits > bottom ? bits : bottom;
            }
            if (Once) break;
        }
#pragma unroll
        for (int d = LG / 2; d > 0; d /= 2) {
            const int t = __shfl_xor(top, d);
            const std::uint32_t b = std::uint32_t(__shfl_xor(int(bottom), d));
            top = t > top ? t : top;
            bottom = b > bottom ? b : bottom;
        }
        const float lo = bits_f32(bottom), hi = bits_f32(std::uint32_t(top));
        const bool fine = top < 0x7f800000 && bottom < 0xff800000u;
        float s = ZP ? (hi - lo) / 15.0f : __builtin_fmaxf(hi, -lo) / 7.0f;
        if (!fine) s = __builtin_nanf("");
        // Every lane of the group rounds the scale; the first stores it.
        if (p.stype == SGEMM_LP_BF16) s = to_f32<BF16>(from_f32<BF16>(s));
        if (p.stype == SGEMM_LP_F16) s = to_f32<F16>(from_f32<F16>(s));
        const bool endless = __builtin_isinf(s), flat = !(s > 0.0f) || endless;
        // Quotients are formed on values moved away from the subnormals.
        const float up = s < 0x1p-90f ? 0x1p90f : 1.0f, scale = s * up;
        const float inverse = flat ? 0.0f : 1.0f / scale;
        float z = ZP && endless ? 0.0f : 8.0f;  // every quotient by an infinite scale is 0
        if (ZP && !flat) {
            const float low = -lo * up;
            rounded_quotients<1>(&low, scale, inverse, &z);
            z = __builtin_fminf(z, 15.0f);
        }
        if (part == 0) {
            store_scale(p.S, p.stype, n * p.lds + g, s);
            if (ZP) p.Z[n * p.ldz + g] = std::uint8_t(z);
        }
        for (int k = k0 + 8 * part; k < k1; k += 8 * LG) {
            if (!Once) load8<T>(row, k, k1, x);
            float q[8];
            if (up != 1.0f) {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] *= up;
            }
            rounded_quotients<8>(x, scale, inverse, q);
            std::uint32_t w = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) w |= std::uint32_t(__builtin_amdgcn_fmed3f(q[i] + z, 0.0f, 15.0f)) << (4 * i);
            w = flat ? (ZP && endless ? 0u : 0x88888888u) : w;
            if (k + 8 > k1) w &= (1u << (4 * (k1 - k))) - 1u;  // past the row's end: 0
            std::uint8_t *dst = p.W + n * p.ldw + k / 2;
            if (k + 8 <= k1) {
                __builtin_memcpy(dst, &w, 4);
            } else {
                for (int i = 0; k + 2 * i < k1; ++i) dst[i] = std::uint8_t(w >> (8 * i));
            }
            if (Once) break;
        }
    }
}

constexpr int kEights = 4;  // eights of codes that a thread has in flight

template <class T, bool ZP>
__global__ __launch_bounds__(kThreads) void w4_dequantize_kernel(W4PackProblem p, unsigned eights, unsigned all)
{
    for (unsigned first = blockIdx.x * (kEights * kThreads) + threadIdx.x; first < all; first += gridDim.x * (kEights * kThreads)) {
        std::uint32_t w[kEights];
        float s[kEights];
        int z[kEights], rest[kEights];
        typename T::elem *dst[kEights];
#pragma unroll
        for (int j = 0; j < kEights; ++j) {
            const unsigned id = first + j * kThreads < all ? first + j * kThreads : all - 1;  // past the last: that one again
            const std::int64_t n = id / eights;
            const int k = int(id % eights) * 8, g = int(unsigned(k) / unsigned(p.group));
            const std::uint8_t *src = p.W + n * p.ldw + k / 2;
            rest[j] = p.K - k;
            if (rest[j] >= 7) {
                w[j] = load_any<std::uint32_t>(src);
            } else {
                w[j] = 0;
                for (int i = 0; 2 * i < rest[j]; ++i) w[j] |= std::uint32_t(src[i]) << (8 * i);
            }
            s[j] = load_scale(p.S, p.stype, n * p.lds + g);
            z[j] = ZP ? p.Z[n * p.ldz + g] & 15 : 8;
            dst[j] = static_cast<typename T::elem *>(p.B) + n * p.ldb + k;
        }
#pragma unroll
        for (int j = 0; j < kEights; ++j) {
            if (first + j * kThreads >= all) continue;
            Eight<T> v;
#pragma unroll
            for (int i = 0; i < 8; ++i) v.x[i] = from_f32<T>(s[j] * float(int((w[j] >> (4 * i)) & 15u) - z[j]));
            if (rest[j] >= 8) {
                __builtin_memcpy(dst[j], &v, sizeof(v));
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < rest[j]) dst[j][i] = v.x[i];
            }
        }
    }
}

// Runs launch(part) over bands of rows of fewer than 2^30 pieces each, `per_row`
// of them a row.
template <class Launch> hipError_t for_each_rows(const W4PackProblem &p, std::int64_t per_row, Launch &&launch)
{
    std::int64_t rows = (std::int64_t(1) << 30) / per_row;
    rows = rows < 1 ? 1 : rows;
    const int bsize = p.dtype == SGEMM_F32 ? 4 : 2, ssize = p.stype == SGEMM_F32 ? 4 : 2;
    for (std::int64_t n0 = 0; n0 < p.N; n0 += rows) {
        W4PackProblem q = p;
        q.N = int(p.N - n0 < rows ? p.N - n0 : rows);
        q.B = static_cast<char *>(p.B) + n0 * p.ldb * bsize;
        q.W = p.W + n0 * p.ldw;
        q.S = static_cast<char *>(p.S) + n0 * p.lds * ssize;
        if (p.Z) q.Z = p.Z + n0 * p.ldz;
        const hipError_t e = launch(q);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

unsigned grid_for(std::int64_t pieces, int each)
{
    const std::int64_t n = (pieces + each - 1) / each;
    return unsigned(n < (1 << 22) ? n : (1 << 22));
}

template <class T, int LG> hipError_t quantize(const W4PackProblem &p, hipStream_t stream)
{
    unsigned groups = unsigned((std::int64_t(p.K) + p.group - 1) / p.group);
    const bool once = p.group == 8 * LG;
    const void *kernel = p.Z ? once ? reinterpret_cast<const void *>(&w4_quantize_kernel<T, LG, true, true>)
                                    : reinterpret_cast<const void *>(&w4_quantize_kernel<T, LG, true, false>)
                         : once ? reinterpret_cast<const void *>(&w4_quantize_kernel<T, LG, false, true>)
                                : reinterpret_cast<const void *>(&w4_quantize_kernel<T, LG, false, false>);
    return for_each_rows(p, groups, [&](W4PackProblem &q) {
        unsigned all = unsigned(q.N) * groups;
        void *args[] = {&q, &groups, &all};
        return hipLaunchKernel(kernel, dim3(grid_for(all, kThreads / LG)), dim3(kThreads), args, 0, stream);
    });
}

template <class T> hipError_t quantize(const W4PackProblem &p, hipStream_t stream)
{
    if (p.group <= 32) return quantize<T, 4>(p, stream);
    if (p.group <= 64) return quantize<T, 8>(p, stream);
    if (p.group <= 128) return quantize<T, 16>(p, stream);
    return quantize<T, 32>(p, stream);
}

template <class T> hipError_t dequantize(const W4PackProblem &p, hipStream_t stream)
{
    unsigned eights = unsigned((std::int64_t(p.K) + 7) / 8);
    const void *kernel = p.Z ? reinterpret_cast<const void *>(&w4_dequantize_kernel<T, true>)
                             : reinterpret_cast<const void *>(&w4_dequantize_kernel<T, false>);
    return for_each_rows(p, eights, [&](W4PackProblem &q) {
        unsigned all = unsigned(q.N) * eights;
        void *args[] = {&q, &eights, &all};
        return hipLaunchKernel(kernel, dim3(grid_for(all, kEights * kThreads)), dim3(kThreads), args, 0, stream);
    });
}

}  // namespace

hipError_t launch_w4_quantize(const W4PackProblem &p, hipStream_t stream)
{
    return p.dtype == SGEMM_F32 ? quantize<F32>(p, stream) : p.dtype == SGEMM_LP_BF16 ? quantize<BF16>(p, stream) : quantize<F16>(p, stream);
}

hipError_t launch_w4_dequantize(const W4PackProblem &p, hipStream_t stream)
{
    return p.dtype == SGEMM_F32 ? dequantize<F32>(p, stream) : p.dtype == SGEMM_LP_BF16 ? dequantize<BF16>(p, stream) : dequantize<F16>(p, stream);
}

}  // namespace sgemm_impl
