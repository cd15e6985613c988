// Products whose stored operand is held in few bits: what the W4 kernels
// (w4.hpp, w4_pack.hip) and the 8-bit cache's kernels (kv8.hip,
// kv8_attend.hpp) share, and their launchers.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstring>

#include "lowbit_plan.hpp"
#include "sgemm.h"

namespace sgemm_impl {

// C = alpha * A * W^T + beta * C with W in the W4 form (sgemm.h). Checked,
// with work to do: M, N, K > 0 and alpha != 0.
struct W4Problem {
    const void *A;
    const std::uint8_t *W;
    const void *S;
    const std::uint8_t *Z;  // nullptr: every zero point is 8
    float *C;
    std::int64_t lda, ldw, lds, ldz, ldc;
    int M, N, K, group;
    int stype;  // sgemm_type of the scales
    int cus;
    float alpha, beta;
};
hipError_t launch_w4_f32(const W4Problem &p, hipStream_t stream);
hipError_t launch_w4_bf16(const W4Problem &p, hipStream_t stream);
hipError_t launch_w4_f16(const W4Problem &p, hipStream_t stream);

// Quantising to the W4 form and reading back (N, K > 0).
struct W4PackProblem {
    void *B;  // read by quantise, written by dequantise
    std::uint8_t *W;
    void *S;
    std::uint8_t *Z;
    std::int64_t ldb, ldw, lds, ldz;
    int N, K, group, dtype, stype;
};
hipError_t launch_w4_quantize(const W4PackProblem &p, hipStream_t stream);
hipError_t launch_w4_dequantize(const W4PackProblem &p, hipStream_t stream);

// Writing and reading the 8-bit cache (seqs, rows > 0); `x` strides in
// elements.
struct Kv8Problem {
    sgemm_kv8_cache c;
    sgemm_kv8_batch b;
    void *K, *V;
    std::int64_t ldk, hsk, ldv, hsv;
    int dtype;
};
hipError_t launch_kv8_write(const Kv8Problem &p, hipStream_t stream);
hipError_t launch_kv8_read(const Kv8Problem &p, hipStream_t stream);

struct Kv8AttendProblem {
    sgemm_kv8_cache c;
    sgemm_kv8_batch b;
    const void *Q;
    float *O;
    float *ws;  // splits > 1
    std::int64_t ldq, hsq, ldo, hso;
    int heads_q;
    float scale;
    int causal, window;
    Kv8Plan plan;
};
hipError_t launch_kv8_attend_f32(const Kv8AttendProblem &p, hipStream_t stream);
hipError_t launch_kv8_attend_bf16(const Kv8AttendProblem &p, hipStream_t stream);
hipError_t launch_kv8_attend_f16(const Kv8AttendProblem &p, hipStream_t stream);

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) std::uint32_t u32x4;
typedef __attribute__((ext_vector_type(2))) std::uint32_t u32x2;

// The element types an operand comes in, as tags.
struct F32 {
    typedef float elem;
};
struct BF16 {
    typedef std::uint16_t elem;
};
struct F16 {
    typedef std::uint16_t elem;
};

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;
typedef __attribute__((ext_vector_type(2))) _Float16 f16x2;

__device__ inline float bits_f32(std::uint32_t u) { return __builtin_bit_cast(float, u); }
__device__ inline std::uint32_t f32_bits(float f) { return __builtin_bit_cast(std::uint32_t, f); }

// One element as float32 (exact), and rounded back.
template <class T> __device__ inline float to_f32(typename T::elem x);
template <> __device__ inline float to_f32<F32>(float x) { return x; }
template <> __device__ inline float to_f32<BF16>(std::uint16_t x) { return bits_f32(std::uint32_t(x) << 16); }
template <> __device__ inline float to_f32<F16>(std::uint16_t x) { return float(__builtin_bit_cast(_Float16, x)); }
template <class T> __device__ inline typename T::elem from_f32(float x);
template <> __device__ inline float from_f32<F32>(float x) { return x; }
template <> __device__ inline std::uint16_t from_f32<BF16>(float x) { return __builtin_bit_cast(std::uint16_t, __bf16(x)); }
template <> __device__ inline std::uint16_t from_f32<F16>(float x)
{
    // A product and its rounding to f16 must not become one v_fma_mixlo_f16,
    // which would round once where the definitions round to float32 first.
    asm("" : "+v"(x));
    return __builtin_bit_cast(std::uint16_t, _Float16(x));
}

// Two float32 rounded to a pair of a 16-bit type, the first in the low half.
template <class T> __device__ inline std::uint32_t rounded2(float a, float b);
template <> __device__ inline std::uint32_t rounded2<BF16>(float a, float b)
{
    typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
    return __builtin_bit_cast(std::uint32_t, bf16x2{__bf16(a), __bf16(b)});
}
template <> __device__ inline std::uint32_t rounded2<F16>(float a, float b)
{
    // As from_f32<F16>: a product is rounded to float32 first.
    asm("" : "+v"(a), "+v"(b));
    return __builtin_bit_cast(std::uint32_t, f16x2{_Float16(a), _Float16(b)});
}

// A scale of a runtime type.
__device__ inline float load_scale(const void *S, int stype, std::int64_t i)
{
    if (stype == SGEMM_F32) return static_cast<const float *>(S)[i];
    const std::uint16_t b = static_cast<const std::uint16_t *>(S)[i];
    return stype == SGEMM_LP_BF16 ? to_f32<BF16>(b) : to_f32<F16>(b);
}

// N bytes from any byte address (the compiler makes one access of it).
template <class V> __device__ inline V load_any(const void *p)
{
    V v;
    __builtin_memcpy(&v, p, sizeof(V));
    return v;
}

// Eight 16-bit elements that are not to stay in the caches.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
__device__ inline u32x4 stream_load(const void *p) { return __builtin_nontemporal_load(static_cast<const u32x4_any *>(p)); }
__device__ inline void stream_store(void *p, u32x4 v) { __builtin_nontemporal_store(v, static_cast<u32x4_any *>(p)); }

// The upper halves of two float32, as a pair of bf16 (a in the low half):
// truncation, so exact when the lower halves are zero.
__device__ inline std::uint32_t pack_hi(float a, float b) { return __builtin_amdgcn_perm(f32_bits(b), f32_bits(a), 0x07060302u); }

// Eight operands of one lane of a 16-bit matrix instruction.
struct Frag {
    u32x4 v;
};
__device__ inline f32x4 mfma_bf16(const Frag &a, const Frag &b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a.v), __builtin_bit_cast(bf16x8, b.v), c, 0, 0, 0);
}
__device__ inline f32x4 mfma_f16(const Frag &a, const Frag &b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a.v), __builtin_bit_cast(f16x8, b.v), c, 0, 0, 0);
}

// Eight float32 as three bf16 parts each, hi + mid + lo == x exactly: each
// part takes the next 8 of the 24 significant bits by truncation, so nothing
// overflows and the last difference fits. A part that a value which is not
// finite would leave as inf - inf is 0, so infinities multiply as they are.
// (Parts below the least bf16 number are lost: |x| under 2^-110 keeps at
// least 8 bits.)
__device__ inline void split3(const float *x, Frag &hi, Frag &mid, Frag &lo)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float h[2], m[2], l[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float a = __builtin_canonicalizef(x[2 * i + j]);
            h[j] = bits_f32(f32_bits(a) & 0xffff0000u);
            float r = a - h[j];
            r = r == r ? r : 0.0f;
            m[j] = bits_f32(f32_bits(r) & 0xffff0000u);
            l[j] = r - m[j];
        }
        hi.v[i] = pack_hi(h[0], h[1]);
        mid.v[i] = pack_hi(m[0], m[1]);
        lo.v[i] = pack_hi(l[0], l[1]);
    }
}

}  // namespace sgemm_impl
