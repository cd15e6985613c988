// Softmax attention over the 8-bit cache (sgemm_kv8_attend): each type of Q
// is its own translation unit (kv8_attend_f32.hip, _bf16.hip, _f16.hip).
//
// For a sequence and a head of the cache, the rows of all query heads that
// read it (new row i, query head h of the group: row i * R + h, R heads a
// group) are the columns of two products on the 16-bit matrix cores
// (v_mfma_f32_16x16x32), walked 32 tokens at a time with the running maximum
// m and sum l of the softmax in float32:
//
//     S^T = K Q^T        z = S * (scale * log2(e) * K's scale)
//     p   = 2^(z - m)    l += p
//     O^T += V^T (p * V's scale)
//
// * S^T rather than S: the matrix instruction leaves lane 16 q + c with rows
//   (tokens) 4 q .. 4 q + 3 of column (query row) c, and takes its second
//   operand with eight k of column c in the same lane. As the order of k is
//   free as long as both operands agree, the p of two 16-token halves are the
//   second product's operand as they stand, k = 4 q + r of either half: no
//   exchange between lanes, no LDS. V's rows are read in that order.
// * Codes become bf16 (K: Q's type) by v_cvt_scalef32_pk, two a conversion,
//   exactly; the scales multiply S and p in float32. V's bytes lie along a
//   token's components, the operand along tokens: v_perm pairs the bytes of
//   two tokens first.
// * Q in bf16 and f16 enters as it is, float32 as three bf16 parts (split3).
//   p * V's scale enters as three bf16 parts as well, so that the float32
//   result carries no rounding of p to fewer bits.
#pragma once

#include <hip/hip_runtime.h>

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

__device__ inline std::uint32_t codes_bf16(std::uint32_t codes, bool upper)
{
    return upper ? __builtin_bit_cast(std::uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, 1.0f, true))
                 : __builtin_bit_cast(std::uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, 1.0f, false));
}
__device__ inline std::uint32_t codes_f16(std::uint32_t codes, bool upper)
{
    return upper ? __builtin_bit_cast(std::uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes, 1.0f, true))
                 : __builtin_bit_cast(std::uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes, 1.0f, false));
}

// Eight components of one query row as the second operand of K Q^T.
template <class T> struct QOperand;
template <> struct QOperand<BF16> {
    Frag f;
    __device__ void load(const std::uint16_t *q, bool there)
    {
        f.v = u32x4{0, 0, 0, 0};
        if (there) f.v = load_any<u32x4>(q);
    }
    __device__ f32x4 scores(u32x2 k, f32x4 acc) const
    {
        const Frag a{{codes_bf16(k[0], false), codes_bf16(k[0], true), codes_bf16(k[1], false), codes_bf16(k[1], true)}};
        return mfma_bf16(a, f, acc);
    }
};
template <> struct QOperand<F16> {
    Frag f;
    __device__ void load(const std::uint16_t *q, bool there)
    {
        f.v = u32x4{0, 0, 0, 0};
        if (there) f.v = load_any<u32x4>(q);
    }
    __device__ f32x4 scores(u32x2 k, f32x4 acc) const
    {
        const Frag a{{codes_f16(k[0], false), codes_f16(k[0], true), codes_f16(k[1], false), codes_f16(k[1], true)}};
        return mfma_f16(a, f, acc);
    }
};
template <> struct QOperand<F32> {
    Frag hi, mid, lo;
    __device__ void load(const float *q, bool there)
    {
        struct Raw {
            float x[8];
        } r;
        __builtin_memset(&r, 0, sizeof(r));
        if (there) r = load_any<Raw>(q);
        split3(r.x, hi, mid, lo);
    }
    __device__ f32x4 scores(u32x2 k, f32x4 acc) const
    {
        const Frag a{{codes_bf16(k[0], false), codes_bf16(k[0], true), codes_bf16(k[1], false), codes_bf16(k[1], true)}};
        return mfma_bf16(a, hi, mfma_bf16(a, mid, mfma_bf16(a, lo, acc)));
    }
};

// The bytes of a word that are e4m3 NaN, as 0x80 in each such byte.
__device__ inline std::uint32_t nan_codes(std::uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

// DC: a head of up to 32 DC components; MT: groups of 16 rows a wave holds.
// A work-group's four waves take the tokens of one row tile in turns of 32
// and add their sums through LDS in the waves' order.
template <class T, int DC, int MT>
__global__ __launch_bounds__(64 * kAttendWaves) void kv8_attend_kernel(Kv8AttendProblem p)
{
    constexpr int PD = 32 * DC, kRows = 16 * MT, kDTiles = 2 * DC, kLd = PD + 4;
    __shared__ float sm_m[kAttendWaves][kRows], sm_l[kAttendWaves][kRows];
    __shared__ __align__(16) float sm_o[kRows * kLd];
    typedef typename T::elem elem;
    const int lane = threadIdx.x & 63, c = lane & 15, kq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int dim = p.c.dim, block = p.c.block, R = p.heads_q / p.c.heads;

    unsigned id = blockIdx.x;
    const int tile0 = int(id % unsigned(p.plan.tiles));
    id /= unsigned(p.plan.tiles);
    const int head = int(id % unsigned(p.c.heads));
    for (unsigned seq = id / unsigned(p.c.heads); seq < unsigned(p.b.seqs); seq += gridDim.x / (unsigned(p.plan.tiles) * unsigned(p.c.heads))) {
        const Kv8Sequence s = kv8_sequence(p.b, int(seq));
        const std::int64_t all_rows = s.n * R;
        // Tokens the table cannot name: every row of the sequence is NaN.
        const std::int64_t nameable = std::int64_t(p.b.table_ld) * block;
        const bool short_table = s.len > nameable;
        for (std::int64_t row0 = std::int64_t(tile0) * kRows; row0 < all_rows; row0 += std::int64_t(p.plan.tiles) * kRows) {
            // Each lane's rows: what they see, and their operands. Rows past
            // the last repeat it; what they give is not stored.
            int lo_t[MT], n_t[MT];  // first token seen, tokens seen
            QOperand<T> q[MT][DC];
            auto seen = [&](std::int64_t row, int &from, int &count) {
                const std::int64_t pos = s.len - s.n + row / R;
                std::int64_t hi = p.causal ? pos + 1 : s.len, lo = p.window > 0 ? pos + 1 - p.window : 0;
                if (hi > nameable) hi = nameable;
                lo = lo < 0 ? 0 : lo;
                hi = hi < lo ? lo : hi;
                from = int(lo);
                count = int(hi - lo);
            };
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                std::int64_t row = row0 + 16 * t + c;
                row = row < all_rows ? row : all_rows - 1;
                seen(row, lo_t[t], n_t[t]);
                const elem *src = static_cast<const elem *>(p.Q) + (s.row0 + row / R) * p.ldq + (head * R + row % R) * p.hsq;
#pragma unroll
                for (int i = 0; i < DC; ++i) q[t][i].load(src + (kq * DC + i) * 8, (kq * DC + i) * 8 < dim);
            }
            int first_lo, first_n, last_lo, last_n;
            const std::int64_t last = row0 + kRows < all_rows ? row0 + kRows - 1 : all_rows - 1;
            seen(row0, first_lo, first_n);
            seen(last, last_lo, last_n);
            const int begin = first_lo & ~31, end = last_lo + last_n;   // tokens some row sees
            const int open = last_lo, close = first_lo + first_n;       // tokens every row sees

            f32x4 o[MT][kDTiles] = {};
            float m[MT], l[MT];
#pragma unroll
            for (int t = 0; t < MT; ++t) m[t] = -__builtin_inff(), l[t] = 0.0f;

            for (int t0 = begin + 32 * wave; t0 < end; t0 += 32 * kAttendWaves) {
                u32x2 k[2][DC];
                std::uint32_t v[8][DC / 2];
                float ks[2], vs[2];
                const std::uint8_t *vrow[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int t = t0 + 16 * h;
                    std::int64_t page = -1;
                    if (t < end) page = kv8_page(p.c, p.b, int(seq), t / block);
                    ks[h] = vs[h] = t < end ? __builtin_nanf("") : 0.0f;
                    const std::int64_t at = (page < 0 ? 0 : page) * p.c.heads + head;
                    const std::int64_t byte0 = (at * block + (t & (block - 1))) * dim;
                    if (page >= 0) ks[h] = p.c.Ks[at], vs[h] = p.c.Vs[at];
                    const std::uint8_t *kr = static_cast<const std::uint8_t *>(p.c.K) + byte0 + c * dim + kq * 8 * DC;
                    vrow[h] = page < 0 ? nullptr : static_cast<const std::uint8_t *>(p.c.V) + byte0;
                    const std::uint8_t *vr = static_cast<const std::uint8_t *>(p.c.V) + byte0 + 4 * kq * dim + c * 2 * DC;
#pragma unroll
                    for (int i = 0; i < DC; ++i) {
                        k[h][i] = u32x2{0, 0};
                        if (page >= 0 && (kq * DC + i) * 8 < dim) k[h][i] = *reinterpret_cast<const u32x2 *>(kr + 8 * i);
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
#pragma unroll
                        for (int i = 0; i < DC / 2; ++i) v[4 * h + r][i] = 0;
                        if (page >= 0 && c * 2 * DC < dim) __builtin_memcpy(v[4 * h + r], vr + r * dim, 2 * DC);
                    }
                }
                const bool cut = t0 < open || t0 + 32 > close;  // some row does not see all 32
                bool poisoned = false;
                if (cut) {
                    // NaN codes must not reach rows that do not see them (0 * NaN):
                    // they leave the product and are put back below.
                    std::uint32_t any = 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
#pragma unroll
                        for (int i = 0; i < DC / 2; ++i) {
                            const std::uint32_t n = nan_codes(v[e][i]);
                            any |= n;
                            v[e][i] &= ~((n >> 7) * 0xffu);
                        }
                    poisoned = __ballot(any != 0) != 0;
                }

                Frag ph[MT], pm[MT], pl[MT];
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    float z[8];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        f32x4 acc = {};
#pragma unroll
                        for (int i = 0; i < DC; ++i) acc = q[t][i].scores(k[h][i], acc);
                        const float f = ks[h] * (p.scale * kLog2e);
#pragma unroll
                        for (int r = 0; r < 4; ++r) z[4 * h + r] = acc[r] * f;
                    }
                    if (cut) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const unsigned j = unsigned(t0 + 16 * (e / 4) + 4 * kq + e % 4 - lo_t[t]);
                            z[e] = j < unsigned(n_t[t]) ? z[e] : -__builtin_inff();
                        }
                    }
                    float top = z[0];
#pragma unroll
                    for (int e = 1; e < 8; ++e) top = __builtin_fmaxf(top, z[e]);
                    top = column_max(top);
                    if (__ballot(top > m[t]) != 0) {
                        const float risen = __builtin_fmaxf(m[t], top);
                        const float a = m[t] == risen ? 1.0f : __builtin_amdgcn_exp2f(m[t] - risen);
                        m[t] = risen;
                        l[t] *= a;
#pragma unroll
                        for (int j = 0; j < kDTiles; ++j) o[t][j] *= a;
                    }
                    const float base = m[t] == -__builtin_inff() ? 0.0f : m[t];
                    float w[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float pe = __builtin_amdgcn_exp2f(z[e] - base);
                        l[t] += pe;
                        w[e] = pe * vs[e / 4];
                        if (cut) w[e] = z[e] == -__builtin_inff() ? 0.0f : w[e];
                    }
                    split3(w, ph[t], pm[t], pl[t]);
                }
#pragma unroll
                for (int i = 0; i < DC / 2; ++i) {
                    Frag f[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const std::uint32_t a = __builtin_amdgcn_perm(v[2 * e + 1][i], v[2 * e][i], 0x05010400u);
                        const std::uint32_t b = __builtin_amdgcn_perm(v[2 * e + 1][i], v[2 * e][i], 0x07030602u);
                        f[0].v[e] = codes_bf16(a, false);
                        f[1].v[e] = codes_bf16(a, true);
                        f[2].v[e] = codes_bf16(b, false);
                        f[3].v[e] = codes_bf16(b, true);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int t = 0; t < MT; ++t)
                            o[t][4 * i + j] = mfma_bf16(f[j], ph[t], mfma_bf16(f[j], pm[t], mfma_bf16(f[j], pl[t], o[t][4 * i + j])));
                }
                if (poisoned) {
                    for (int u = 0; u < 32; ++u) {
                        const std::uint8_t *row = vrow[u / 16];
                        if (row == nullptr) continue;
#pragma unroll
                        for (int x = 0; x < 4 * kDTiles; ++x) {
                            const int d = kq * 8 * DC + x;  // component of register x / kDTiles of d-tile x % kDTiles
                            if (d >= dim || (row[(u % 16) * dim + d] & 0x7f) != 0x7f) continue;
#pragma unroll
                            for (int t = 0; t < MT; ++t)
                                if (unsigned(t0 + u - lo_t[t]) < unsigned(n_t[t])) o[t][x % kDTiles][x / kDTiles] = __builtin_nanf("");
                        }
                    }
                }
            }

            // The waves' sums: all onto the largest maximum.
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                l[t] = column_sum(l[t]);
                if (kq == 0) sm_m[wave][16 * t + c] = m[t], sm_l[wave][16 * t + c] = l[t];
            }
            __syncthreads();
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                float top = sm_m[0][16 * t + c];
#pragma unroll
                for (int w = 1; w < kAttendWaves; ++w) top = __builtin_fmaxf(top, sm_m[w][16 * t + c]);
                const float a = m[t] == top ? 1.0f : __builtin_amdgcn_exp2f(m[t] - top);
#pragma unroll
                for (int j = 0; j < kDTiles; ++j) o[t][j] *= a;
            }
            for (int w = 0; w < kAttendWaves; ++w) {
                if (w == wave) {
#pragma unroll
                    for (int t = 0; t < MT; ++t)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
#pragma unroll
                            for (int j = 0; j < kDTiles; j += 4) {
                                f32x4 *at = reinterpret_cast<f32x4 *>(&sm_o[(16 * t + c) * kLd + (4 * kq + r) * kDTiles + j]);
                                const f32x4 x = {o[t][j][r], o[t][j + 1][r], o[t][j + 2][r], o[t][j + 3][r]};
                                *at = w == 0 ? x : *at + x;
                            }
                }
                __syncthreads();
            }
            const std::int64_t rows = all_rows - row0 < kRows ? all_rows - row0 : kRows;
            for (int e = threadIdx.x; e < int(rows) * dim; e += 64 * kAttendWaves) {
                const int i = e / dim, d = e % dim;
                float top = sm_m[0][i], sum = 0.0f;
#pragma unroll
                for (int w = 1; w < kAttendWaves; ++w) top = __builtin_fmaxf(top, sm_m[w][i]);
#pragma unroll
                for (int w = 0; w < kAttendWaves; ++w)
                    sum += sm_l[w][i] * (sm_m[w][i] == top ? 1.0f : __builtin_amdgcn_exp2f(sm_m[w][i] - top));
                float x = sm_o[i * kLd + d];
                x = sum == 0.0f ? 0.0f : x / sum;
                if (short_table) x = __builtin_nanf("");
                const std::int64_t row = row0 + i;
                p.O[(s.row0 + row / R) * p.ldo + (head * R + row % R) * p.hso + d] = x;
            }
            __syncthreads();
        }
    }
}

template <class T, int DC, int MT> hipError_t launch_attend_shape(const Kv8AttendProblem &p, hipStream_t stream)
{
    const std::int64_t per_seq = std::int64_t(p.plan.tiles) * p.c.heads;
    std::int64_t seqs = (std::int64_t(1) << 23) / per_seq;
    seqs = seqs < 1 ? 1 : seqs < p.b.seqs ? seqs : p.b.seqs;
    Kv8AttendProblem q = p;
    void *args[] = {&q};
    return hipLaunchKernel(reinterpret_cast<const void *>(&kv8_attend_kernel<T, DC, MT>), dim3(unsigned(per_seq * seqs)),
                           dim3(64 * kAttendWaves), args, 0, stream);
}

template <class T> hipError_t launch_attend(const Kv8AttendProblem &p, hipStream_t stream)
{
    if (p.c.dim <= 64) return launch_attend_shape<T, 2, 1>(p, stream);
    if (p.c.dim <= 128) return launch_attend_shape<T, 4, 1>(p, stream);
    return launch_attend_shape<T, 8, 1>(p, stream);
}

}  // namespace
}  // namespace sgemm_impl
