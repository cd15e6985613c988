// Rotary positions (sgemm_rope): pairs of components of each head turned by
// angles that grow with the row's position.
//
// The angle is formed in float64, in quarter turns; what is left of it after
// the nearest whole one lies within an eighth of a turn, where sin and cos are
// their Taylor polynomials (of degree 9 and 10: the first term left out is
// below 2^-28 and 2^-32) and a float32 argument costs at most 2^-25. All heads
// of a row turn by the same angles: a work-group forms those of its rows once,
// in LDS, and then walks over the rows' heads in pieces of eight pairs.
//
// Bound by memory: 4 prompts of up to 4096 rows, 32 and 8 heads of 128 in bf16
// (240 MB), take 49 us in a graph, 4.9 TB/s, with inputs and outputs kept out of
// the caches, 53 without; 2 of up to 1021 rows of 96 components, float32 to bf16 (42 MB), 10.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "gemm.hpp"
#include "step.hpp"

namespace sgemm_impl {
namespace {

constexpr int kThreads = 256, kAngles = 512;  // angles that a work-group holds: one row of the largest heads

struct Turn {
    float c, s;
};

__device__ inline Turn turn_of(int position, double freq, float amplitude, bool inverse)
{
    constexpr double kUp = 0.63661977236758134308, kLow = -3.9357353350364972e-17;  // 2 / pi
    // Of the angle and of its product with 2 / pi what is rounded off is kept: up to 2^-24 each at 2^30 radians.
    const double t = double(position) * freq, whole = __builtin_rint(t * kUp);
    const double left = __builtin_fma(t, kUp, -whole) + __builtin_fma(t, kLow, __builtin_fma(double(position), freq, -t) * kUp);
    const float x = float(left) * 1.57079632679489661923f, y = x * x;
    const float s = x * __builtin_fmaf(y, __builtin_fmaf(y, __builtin_fmaf(y, __builtin_fmaf(y, 1.0f / 362880, -1.0f / 5040), 1.0f / 120), -1.0f / 6), 1.0f);
    const float c = __builtin_fmaf(
        y, __builtin_fmaf(y, __builtin_fmaf(y, __builtin_fmaf(y, __builtin_fmaf(y, -1.0f / 3628800, 1.0f / 40320), -1.0f / 720), 1.0f / 24), -0.5f), 1.0f);
    const int quadrant = int(whole - 4.0 * __builtin_floor(0.25 * whole));
    const float cs = quadrant & 1 ? s : c, sn = quadrant & 1 ? c : s;
    const float cosine = quadrant == 1 || quadrant == 2 ? -cs : cs, sine = quadrant >= 2 ? -sn : sn;
    return {amplitude * cosine, amplitude * (inverse ? -sine : sine)};
}

template <class T, int N> struct Elems {
    typename T::elem x[N];
};

// Side: pairs side by side, not apart (i and i + rot / 2). Stream: outputs of 16
// bits, pairs apart, that are kept out of the caches.
template <class T, class U, bool Side, bool Stream> __global__ __launch_bounds__(kThreads) void rope_kernel(RopeProblem p, int rows_at_once)
{
    typedef typename T::elem in;
    typedef typename U::elem out;
    __shared__ Turn turns[kAngles];
    const int pairs = p.rot / 2, rest = p.dim - p.rot;
    const unsigned heads = unsigned(p.x[0].heads + p.x[1].heads), turned = unsigned(pairs + 7) / 8, copied = unsigned(rest + 15) / 16;
    const unsigned pieces = turned + copied, per_row = heads * pieces;
    for (std::int64_t row0 = std::int64_t(blockIdx.x) * rows_at_once; row0 < p.rows; row0 += std::int64_t(gridDim.x) * rows_at_once) {
        const int rows = int(p.rows - row0 < rows_at_once ? p.rows - row0 : rows_at_once);
        __syncthreads();  // the angles of the rows before are no longer read
        for (int i = threadIdx.x; i < rows * pairs; i += kThreads)
            turns[i] = turn_of(p.positions[row0 + i / pairs], p.freqs[i % pairs], p.amplitude, p.inverse != 0);
        __syncthreads();
        const unsigned all = unsigned(rows) * per_row;
        for (unsigned id = threadIdx.x; id < all; id += kThreads) {
            const unsigned r = id / per_row, in_row = id - r * per_row;
            const unsigned head = in_row / pieces, piece = in_row - head * pieces;
            const int which = head >= unsigned(p.x[0].heads) ? 1 : 0;
            const sgemm_rope_rows &o = p.x[which];
            const std::int64_t h = std::int64_t(head) - (which ? p.x[0].heads : 0), row = row0 + r;
            const in *x = static_cast<const in *>(o.X) + row * o.ldx + h * o.hsx;
            out *y = static_cast<out *>(o.Y) + row * o.ldy + h * o.hsy;
            if (piece >= turned) {
                const int at = p.rot + int(piece - turned) * 16, n = p.dim - at < 16 ? p.dim - at : 16;
                if (sizeof(in) == sizeof(out) && static_cast<const void *>(x) == static_cast<const void *>(y)) continue;  // in place
                if (n == 16) {
                    const Elems<T, 16> v = load_any<Elems<T, 16>>(x + at);
                    Elems<U, 16> w;
#pragma unroll
                    for (int j = 0; j < 16; ++j) w.x[j] = from_f32<U>(to_f32<T>(v.x[j]));
                    __builtin_memcpy(y + at, &w, sizeof(w));
                } else {
                    for (int j = 0; j < n; ++j) y[at + j] = from_f32<U>(to_f32<T>(x[at + j]));
                }
                continue;
            }
            const int i0 = int(piece) * 8, n = pairs - i0 < 8 ? pairs - i0 : 8;
            const Turn *t = turns + int(r) * pairs + i0;
            if (n == 8) {
                Elems<T, 16> v;
                if (Side) {
                    v = load_any<Elems<T, 16>>(x + 2 * i0);
                } else {
                    Elems<T, 8> a, b;
                    if constexpr (Stream && sizeof(in) == 2) {
                        a = __builtin_bit_cast(Elems<T, 8>, stream_load(x + i0)), b = __builtin_bit_cast(Elems<T, 8>, stream_load(x + pairs + i0));
                    } else {
                        a = load_any<Elems<T, 8>>(x + i0), b = load_any<Elems<T, 8>>(x + pairs + i0);
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) v.x[2 * j] = a.x[j], v.x[2 * j + 1] = b.x[j];
                }
                Elems<U, 8> a, b;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float xa = to_f32<T>(v.x[2 * j]), xb = to_f32<T>(v.x[2 * j + 1]);
                    const Turn u = t[j];
                    a.x[j] = from_f32<U>(__builtin_fmaf(xa, u.c, -(xb * u.s)));
                    b.x[j] = from_f32<U>(__builtin_fmaf(xb, u.c, xa * u.s));
                }
                if (Side) {
                    Elems<U, 16> w;
#pragma unroll
                    for (int j = 0; j < 8; ++j) w.x[2 * j] = a.x[j], w.x[2 * j + 1] = b.x[j];
                    __builtin_memcpy(y + 2 * i0, &w, sizeof(w));
                } else {
                    if constexpr (Stream) {
                        stream_store(y + i0, __builtin_bit_cast(u32x4, a));
                        stream_store(y + pairs + i0, __builtin_bit_cast(u32x4, b));
                    } else {
                        __builtin_memcpy(y + i0, &a, sizeof(a));
                        __builtin_memcpy(y + pairs + i0, &b, sizeof(b));
                    }
                }
            } else {
                for (int j = 0; j < n; ++j) {
                    const int ia = Side ? 2 * (i0 + j) : i0 + j, ib = Side ? ia + 1 : ia + pairs;
                    const float xa = to_f32<T>(x[ia]), xb = to_f32<T>(x[ib]);
                    y[ia] = from_f32<U>(__builtin_fmaf(xa, t[j].c, -(xb * t[j].s)));
                    y[ib] = from_f32<U>(__builtin_fmaf(xb, t[j].c, xa * t[j].s));
                }
            }
        }
    }
}

template <class T, class U> const void *rope_kernel_of(bool side, bool stream)
{
    if (side) return reinterpret_cast<const void *>(&rope_kernel<T, U, true, false>);
    if constexpr (sizeof(typename U::elem) == 2)
        if (stream) return reinterpret_cast<const void *>(&rope_kernel<T, U, false, true>);
    return reinterpret_cast<const void *>(&rope_kernel<T, U, false, false>);
}

template <class T> const void *rope_kernel_of(int otype, bool side, bool stream)
{
    return otype == SGEMM_F32       ? rope_kernel_of<T, F32>(side, stream)
           : otype == SGEMM_LP_BF16 ? rope_kernel_of<T, BF16>(side, stream)
                                    : rope_kernel_of<T, F16>(side, stream);
}

}  // namespace

hipError_t launch_rope(const RopeProblem &p, int cus, hipStream_t stream)
{
    const bool side = p.interleaved != 0, large = p.stream();
    const void *kernel = p.dtype == SGEMM_F32       ? rope_kernel_of<F32>(p.otype, side, large)
                         : p.dtype == SGEMM_LP_BF16 ? rope_kernel_of<BF16>(p.otype, side, large)
                                                    : rope_kernel_of<F16>(p.otype, side, large);
    // As many rows as give each thread an angle, but no more than leave every
    // compute unit a few work-groups.
    int rows_at_once = p.rot / 2 > 0 ? kThreads / (p.rot / 2) : 16;
    const int most = p.rows / (4 * cus);
    if (rows_at_once > most) rows_at_once = most;
    if (rows_at_once > 16) rows_at_once = 16;
    if (rows_at_once < 1) rows_at_once = 1;
    const std::int64_t groups = (std::int64_t(p.rows) + rows_at_once - 1) / rows_at_once;
    RopeProblem q = p;
    void *args[] = {&q, &rows_at_once};
    return hipLaunchKernel(kernel, dim3(unsigned(groups < (1 << 22) ? groups : 1 << 22)), dim3(kThreads), args, 0, stream);
}

}  // namespace sgemm_impl
