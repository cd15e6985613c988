// Softmax attention over the 4-bit cache (sgemm_kv4_attend): each type of Q is
// its own translation unit (kv4_attend_f32.hip, _bf16.hip, _f16.hip).
//
// As over the 8-bit cache (kv8_attend.hpp): S^T = K Q^T and O^T += V^T P^T on
// the 16-bit matrix cores, 32 tokens a turn, the running maximum and sum of the
// softmax in float32, the weights as they stand in registers the second
// product's operand. What differs is what the codes ask for:
//
// * A token has a scale of its own, K's multiplied into its scores and V's
//   into its weight, both in float32.
// * Codes become bf16 (K: Q's type) by v_cvt_scalef32_pk_*_fp4, the two of a
//   byte in one conversion. K's bytes lie along the components as the operand
//   wants them. V's operand wants two tokens of one component in a pair: the
//   halves of the bytes of two tokens are exchanged before the conversion, four
//   instructions for sixteen codes.
// * A code is always a finite number, so tokens that a row does not see need
//   no care beyond a weight of zero.
//
// Codes are exact in f16, so the weights may be held in two parts of f16, 22
// bits, where bf16 would need three for as many, and a matrix instruction of
// four is saved (prompts 259 -> 228 us). f16's range is made enough by a
// common power of two for each row: the running maximum m is that of z +
// exponent(V's scale) over the tokens seen, and weights are 2^(z - m + 14), so
// that the largest product of a weight and a scale lies between 2^14 and 2^15
// whatever the scales are. The sum l counts weights of the same factor, which
// the quotient drops. A product is held to 2^-22 of itself, or to 2^-39 of the
// row's largest where that is more. Tokens that a row does not see take no part
// in its maximum, so their scales do not cost it precision.
//
// While a wave feeds the matrix cores in a prompt its priority is raised: the
// other wave of the SIMD then finds its vector instructions' turn while those
// run (228 -> 216 us).
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "attend.hpp"
#include "kv8.hpp"
#include "step.hpp"

namespace sgemm_impl {
namespace {

// The two codes of byte `at` of a word as a pair of bf16 or f16.
template <int At> __device__ inline std::uint32_t fp4_bf16(std::uint32_t codes)
{
    return __builtin_bit_cast(std::uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, 1.0f, At));
}
template <int At> __device__ inline std::uint32_t fp4_f16(std::uint32_t codes)
{
    return __builtin_bit_cast(std::uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, At));
}

// Eight components of one query row as the second operand of K Q^T, by eight
// codes of a token.
template <class T> struct QOperand4;
template <> struct QOperand4<BF16> {
    Frag f;
    __device__ void load(const std::uint16_t *q, bool there)
    {
        f.v = u32x4{0, 0, 0, 0};
        if (there) f.v = load_any<u32x4>(q);
    }
    __device__ f32x4 scores(std::uint32_t k, f32x4 acc) const
    {
        const Frag a{{fp4_bf16<0>(k), fp4_bf16<1>(k), fp4_bf16<2>(k), fp4_bf16<3>(k)}};
        return mfma_bf16(a, f, acc);
    }
};
template <> struct QOperand4<F16> {
    Frag f;
    __device__ void load(const std::uint16_t *q, bool there)
    {
        f.v = u32x4{0, 0, 0, 0};
        if (there) f.v = load_any<u32x4>(q);
    }
    __device__ f32x4 scores(std::uint32_t k, f32x4 acc) const
    {
        const Frag a{{fp4_f16<0>(k), fp4_f16<1>(k), fp4_f16<2>(k), fp4_f16<3>(k)}};
        return mfma_f16(a, f, acc);
    }
};
template <> struct QOperand4<F32> {
    Frag hi, lo;
    __device__ f32x4 scores(std::uint32_t k, f32x4 acc) const
    {
        const Frag a{{fp4_f16<0>(k), fp4_f16<1>(k), fp4_f16<2>(k), fp4_f16<3>(k)}};
        return mfma_f16(a, hi, mfma_f16(a, lo, acc));
    }
};

// Two float32 as two parts of f16, hi + lo, each rounded to nearest: 22 bits
// and the sign, or down to 2^-24 for what lies below f16's normal numbers.
__device__ inline void split2(float a, float b, std::uint32_t &hi, std::uint32_t &lo)
{
    hi = __builtin_bit_cast(std::uint32_t, f16x2{_Float16(a), _Float16(b)});
    float ra, rb;  // a - hi, b - hi: exact
    asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel_hi:[1,0,0]" : "=v"(ra) : "v"(hi), "v"(a));
    asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "=v"(rb) : "v"(hi), "v"(b));
    lo = __builtin_bit_cast(std::uint32_t, f16x2{_Float16(ra), _Float16(rb)});
}

// A lane's pieces of one query row (eight components each, of those that are
// `there`), and the factor that its scores are to be multiplied by. float32
// rows are brought to a largest component of 2^14 to 2^15 by a power of two,
// so that their parts hold each component to 2^-22 of itself or 2^-39 of the
// largest. (A row with a component that is not finite has no finite score.)
template <class T, int DC, class There> __device__ inline float load_query(QOperand4<T> (&q)[DC], const typename T::elem *src, There &&there)
{
    if constexpr (sizeof(typename T::elem) == 2) {
#pragma unroll
        for (int i = 0; i < DC; ++i) q[i].load(src + 8 * i, there(i));
        return 1.0f;
    } else {
        struct Raw {
            float x[8];
        } r[DC];
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < DC; ++i) {
            __builtin_memset(&r[i], 0, sizeof(Raw));
            if (there(i)) r[i] = load_any<Raw>(src + 8 * i);
#pragma unroll
            for (int j = 0; j < 8; ++j) top = __builtin_fmaxf(top, __builtin_fabsf(r[i].x[j]));
        }
        top = column_max(top);
        int field = 127 + 14 + 127 - int(f32_bits(top) >> 23);
        field = field > 253 ? 253 : field;
        const float up = bits_f32(std::uint32_t(field) << 23);
#pragma unroll
        for (int i = 0; i < DC; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                std::uint32_t hi, lo;
                split2(r[i].x[2 * j] * up, r[i].x[2 * j + 1] * up, hi, lo);
                q[i].hi.v[j] = hi;
                q[i].lo.v[j] = lo;
            }
        return bits_f32(std::uint32_t(254 - field) << 23);
    }
}

// Four bfloat16 scales of adjacent tokens.
__device__ inline float scale_of(u32x2 s, int r)
{
    return bits_f32(r & 1 ? s[r / 2] & 0xffff0000u : s[r / 2] << 16);
}

// The exponents of the sizes of two scales (the lower half's and the upper
// one's), in float32 and 127 too large. Scales below 2^-90 (and zeros) count as
// 2^-90, so that a weight that such a scale is to bring back into range does
// not overflow.
__device__ inline void exponents_of(std::uint32_t s, float &lower, float &upper)
{
    typedef __attribute__((ext_vector_type(2))) std::uint16_t u16x2;
    const u16x2 v = __builtin_elementwise_max(__builtin_bit_cast(u16x2, s << 1), u16x2{(127 - 90) << 8, (127 - 90) << 8});
    const std::uint32_t u = __builtin_bit_cast(std::uint32_t, v);
    lower = float((u >> 8) & 0xffu);
    upper = float(u >> 24);
}

template <class T, int DC, bool Full, int MT, bool Rows>
__global__ __launch_bounds__(64 * kAttendWaves, 2) void kv4_attend_kernel(Kv4AttendProblem p)
{
    constexpr int PD = 32 * DC, kRows = 16 * MT, kDTiles = 2 * DC, kLd = PD + 4, kVWords = (DC + 3) / 4;
    __shared__ float sm_m[kAttendWaves][kRows], sm_l[kAttendWaves][kRows];
    __shared__ __align__(16) float sm_o[Rows ? 4 : kRows * kLd];
    typedef typename T::elem elem;
    const int lane = threadIdx.x & 63, c = lane & 15, kq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int dim = Full ? PD : p.c.dim, R = p.heads_q / p.c.heads;
    const int shift = 31 - __builtin_clz(unsigned(p.c.block)), block = 1 << shift;

    unsigned id = blockIdx.x;
    const int split = int(id % unsigned(p.plan.splits));
    id /= unsigned(p.plan.splits);
    const int tile0 = int(id % unsigned(p.plan.tiles));
    id /= unsigned(p.plan.tiles);
    const int head = int(id % unsigned(p.c.heads));
    const unsigned seqs_at_once = gridDim.x / (unsigned(p.plan.splits) * unsigned(p.plan.tiles) * unsigned(p.c.heads));
    const float factor = p.scale * kLog2e;
    const std::uint8_t *const codes_k = static_cast<const std::uint8_t *>(p.c.K), *const codes_v = static_cast<const std::uint8_t *>(p.c.V);
    const std::uint16_t *const scales_k = static_cast<const std::uint16_t *>(p.c.Ks), *const scales_v = static_cast<const std::uint16_t *>(p.c.Vs);
    // Lanes past the head's components read its first ones: keys are then
    // zeroed, values give components that are not stored.
    const int k_at = c * (dim / 2), v_at = 4 * kq * (dim / 2) + (Full || c * 2 * DC < dim ? c * DC : 0);

    for (unsigned seq = id / unsigned(p.c.heads); seq < unsigned(p.b.seqs); seq += seqs_at_once) {
        const Kv8Sequence s = kv8_sequence(p.b, int(seq));
        const std::int64_t all_rows = s.n * R;
        const KvSeen seen{s.len - s.n, s.len, std::int64_t(p.b.table_ld) << shift, R, p.causal, p.window};
        const int *const table = p.b.table + std::int64_t(seq) * p.b.table_ld;
        for (std::int64_t tile = tile0;; tile += p.plan.tiles) {
            const std::int64_t row0 = Rows ? (tile * kAttendWaves + wave) * kRows : tile * kRows;
            if ((Rows ? tile * kAttendWaves * kRows : row0) >= all_rows) break;
            // Tiles beyond those the grid (and the workspace) was laid out for are not split.
            const bool whole = p.plan.splits == 1 || tile >= p.plan.tiles;
            if (whole && split > 0) break;
            if (Rows && row0 >= all_rows) continue;  // no barrier below when Rows

            // Each lane's rows: what they see, and their operands. Rows past
            // the last repeat it; what they give is not stored.
            int lo_t[MT], n_t[MT];  // first token seen, tokens seen
            QOperand4<T> q[MT][DC];
            float row_factor[MT];
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                std::int64_t row = row0 + 16 * t + c;
                row = row < all_rows ? row : all_rows - 1;
                seen(row, lo_t[t], n_t[t]);
                const elem *src = static_cast<const elem *>(p.Q) + (s.row0 + row / R) * p.ldq + (head * R + row % R) * p.hsq;
                row_factor[t] = load_query<T, DC>(q[t], src + kq * DC * 8, [&](int i) { return Full || (kq * DC + i) * 8 < dim; });
            }
            int first_lo, first_n, last_lo, last_n;
            seen(row0, first_lo, first_n);
            seen(row0 + kRows < all_rows ? row0 + kRows - 1 : all_rows - 1, last_lo, last_n);
            // Turns of 32 tokens: begin .. end sees some row; inner .. outer every row in full.
            // (Positions reach 2^31 - 1, so that rounding up needs the sign bit.)
            const int limit = last_lo + last_n;
            int begin = first_lo >> 5, end = int((unsigned(limit) + 31u) >> 5);
            const int inner = int((unsigned(last_lo) + 31u) >> 5), outer = (first_lo + first_n) >> 5;
            if (!whole) {
                const int turns = end - begin, b = begin;
                begin = b + int(std::int64_t(turns) * split / p.plan.splits);
                end = b + int(std::int64_t(turns) * (split + 1) / p.plan.splits);
            }

            f32x4 o[MT][kDTiles] = {};
            float m[MT], l[MT];
#pragma unroll
            for (int t = 0; t < MT; ++t) m[t] = -__builtin_inff(), l[t] = 0.0f;

            // The page of a half turn, and where its first token lies; `good`: it may be read.
            struct Half {
                std::int64_t token;
                bool good;
            };
            auto half_at = [&](int t) {
                // Past the tokens seen (limit <= nameable) any page of the table will do; none is named by an empty one.
                const int page = uniform_load(table, (t < limit ? t : limit - 1) >> shift);
                const bool good = unsigned(page) < unsigned(p.c.pages);
                return Half{(((std::int64_t(good ? page : 0) * p.c.heads + head) << shift) + (t & (block - 1))), good};
            };
            std::uint32_t k[2][DC], v[8][kVWords];
            u32x2 ks[2], vs[2];
            auto load_keys = [&](const Half (&h)[2]) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const std::uint8_t *const at = codes_k + h[x].token * (dim / 2) + k_at;
                    if (Full) {
                        __builtin_memcpy(k[x], at + kq * 4 * DC, 4 * DC);
                    } else {
#pragma unroll
                        for (int i = 0; i < DC; i += 2) {
                            const bool there = (kq * DC + i) * 8 < dim;
                            __builtin_memcpy(&k[x][i], at + (there ? (kq * DC + i) * 4 : 0), 8);
                            k[x][i] = there ? k[x][i] : 0;
                            k[x][i + 1] = there ? k[x][i + 1] : 0;
                        }
                    }
                    ks[x] = *reinterpret_cast<const u32x2 *>(scales_k + h[x].token + 4 * kq);
                    if (!h[x].good) ks[x] = u32x2{~0u, ~0u};  // NaN
                }
            };
            auto load_values = [&](const Half (&h)[2]) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const std::uint8_t *const at = codes_v + h[x].token * (dim / 2) + v_at;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if constexpr (DC == 2) v[4 * x + e][0] = load_any<std::uint16_t>(at + e * (dim / 2));
                        else __builtin_memcpy(v[4 * x + e], at + e * (dim / 2), DC);
                    }
                    vs[x] = *reinterpret_cast<const u32x2 *>(scales_v + h[x].token + 4 * kq);
                }
            };

            // Turns from .. to, this wave's among them; Cut: some row does not see all of a turn.
            auto turns = [&](int from, int to, auto cut_) {
                constexpr bool Cut = decltype(cut_)::value;
                constexpr int kStride = Rows ? 1 : kAttendWaves;
                int turn = from + (Rows ? 0 : (wave - from) & (kAttendWaves - 1));
                if (turn >= to) return;
                {
                    const Half first[2] = {half_at(32 * turn), half_at(32 * turn + 16)};
                    load_keys(first);
                    load_values(first);
                }
                for (; turn < to; turn += kStride) {
                    const int t0 = 32 * turn, tn = turn + kStride < to ? 32 * (turn + kStride) : t0;
                    const Half next[2] = {half_at(tn), half_at(tn + 16)};
                    f32x4 acc[2][MT];
                    float g[8], ev[8];
                    if (Rows) __builtin_amdgcn_s_setprio(1);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
#pragma unroll
                        for (int t = 0; t < MT; ++t) {
                            acc[x][t] = f32x4{0, 0, 0, 0};
#pragma unroll
                            for (int i = 0; i < DC; ++i) acc[x][t] = q[t][i].scores(k[x][i], acc[x][t]);
                            if (sizeof(elem) == 4) acc[x][t] *= row_factor[t];
                        }
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            // x * 0 + x: a scale that is not finite becomes NaN.
                            const float f = scale_of(ks[x], r);
                            g[4 * x + r] = __builtin_fmaf(f, 0.0f, f) * factor;
                        }
#pragma unroll
                        for (int r = 0; r < 2; ++r) exponents_of(vs[x][r], ev[4 * x + 2 * r], ev[4 * x + 2 * r + 1]);
                    }
                    if (Rows) __builtin_amdgcn_s_setprio(0);
                    load_keys(next);
                    Frag ph[MT], pl[MT];
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        unsigned seen = 0;  // bits of the tokens that the row sees
                        float top = -__builtin_inff();
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            float y = __builtin_fmaf(acc[e / 4][t][e % 4], g[e], ev[e]);
                            if (Cut) {
                                const unsigned j = unsigned(t0 + 16 * (e / 4) + 4 * kq + e % 4 - lo_t[t]);
                                const bool sees = j < unsigned(n_t[t]);
                                y = sees ? y : -__builtin_inff();
                                seen |= sees ? 1u << e : 0u;
                            }
                            top = __builtin_fmaxf(top, y);
                        }
                        top = column_max(top);
                        if (__ballot(top > m[t]) != 0) {
                            const float risen = __builtin_fmaxf(m[t], top), a = rescale(m[t], risen);
                            m[t] = risen;
                            l[t] *= a;
#pragma unroll
                            for (int j = 0; j < kDTiles; ++j) o[t][j] *= a;
                        }
                        const float base = m[t] == -__builtin_inff() ? 0.0f : m[t] - (127.0f + 14.0f);
                        float w[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            float pe = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[e / 4][t][e % 4], g[e], -base));
                            // A scale that is not finite makes the whole row NaN, by w or by its parts.
                            w[e] = pe * scale_of(vs[e / 4], e % 4);
                            if (Cut && !(seen >> e & 1)) pe = w[e] = 0.0f;
                            l[t] += pe;
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            std::uint32_t hi, lo;
                            split2(w[2 * e], w[2 * e + 1], hi, lo);
                            ph[t].v[e] = hi;
                            pl[t].v[e] = lo;
                        }
                    }
                    if (Rows) __builtin_amdgcn_s_setprio(1);
#pragma unroll
                    for (int i = 0; i < kVWords; ++i) {
                        // Byte x of even (odd): component 2 x (2 x + 1) of the word, of tokens 2 e and 2 e + 1.
                        std::uint32_t even[4], odd[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const std::uint32_t a = v[2 * e][i], b = v[2 * e + 1][i];
                            even[e] = (a & 0x0f0f0f0fu) | ((b << 4) & 0xf0f0f0f0u);
                            odd[e] = ((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u);
                        }
                        auto byte = [&](auto at_) {
                            constexpr int At = decltype(at_)::value;
                            Frag f[2];
#pragma unroll
                            for (int e = 0; e < 4; ++e) f[0].v[e] = fp4_f16<At>(even[e]), f[1].v[e] = fp4_f16<At>(odd[e]);
#pragma unroll
                            for (int t = 0; t < MT; ++t)
#pragma unroll
                                for (int j = 0; j < 2; ++j) {
                                    f32x4 &sum = o[t][8 * i + 2 * At + j];
                                    sum = mfma_f16(f[j], ph[t], mfma_f16(f[j], pl[t], sum));
                                }
                        };
                        byte(std::integral_constant<int, 0>{});
                        byte(std::integral_constant<int, 1>{});
                        if constexpr (DC > 2) {
                            byte(std::integral_constant<int, 2>{});
                            byte(std::integral_constant<int, 3>{});
                        }
                    }
                    if (Rows) __builtin_amdgcn_s_setprio(0);
                    load_values(next);
                }
            };
            if (inner < outer) {
                const int a = inner < end ? (inner > begin ? inner : begin) : end, b = outer < end ? (outer > a ? outer : a) : end;
                turns(begin, a, std::true_type{});
                turns(a, b, std::false_type{});
                turns(b, end, std::true_type{});
            } else {
                turns(begin, end, std::true_type{});
            }
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                // A row that sees no token is 0 / 1; one whose scores are all -inf is 0 / 0.
                const float sum = column_sum(l[t]);
                l[t] = n_t[t] == 0 ? 1.0f : sum;
            }

            if constexpr (Rows) {
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    const std::int64_t row = row0 + 16 * t + c;
                    if (row >= all_rows) continue;
                    float inverse = 1.0f / l[t];
                    if (seen.beyond(row)) inverse = __builtin_nanf("");
                    float *dst = p.O + (s.row0 + row / R) * p.ldo + (head * R + row % R) * p.hso + kq * 8 * DC;
#pragma unroll
                    for (int x = 0; x < 4 * kDTiles; x += 4) {
                        if (!Full && kq * 8 * DC + x >= dim) continue;
                        f32x4 y;
#pragma unroll
                        for (int j = 0; j < 4; ++j) y[j] = o[t][(x + j) % kDTiles][x / kDTiles] * inverse;
                        __builtin_memcpy(dst + x, &y, sizeof(y));
                    }
                }
                continue;
            }

            // The waves' sums: all onto the largest maximum.
#pragma unroll
            for (int t = 0; t < MT; ++t)
                if (kq == 0) sm_m[wave][16 * t + c] = m[t], sm_l[wave][16 * t + c] = l[t];
            __syncthreads();
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                float top = sm_m[0][16 * t + c];
#pragma unroll
                for (int w = 1; w < kAttendWaves; ++w) top = __builtin_fmaxf(top, sm_m[w][16 * t + c]);
                const float a = rescale(m[t], top);
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
            const int rows = int(all_rows - row0 < kRows ? all_rows - row0 : kRows);
            // A thread keeps one component quad of every 4 * 64 / (PD / 4)-th row.
            constexpr int kQuads = PD / 4, kStep = 64 * kAttendWaves / kQuads;
            const int d = int(threadIdx.x) % kQuads * 4;
            for (int i = threadIdx.x / kQuads; i < rows; i += kStep) {
                float top = sm_m[0][i], sum = 0.0f;
#pragma unroll
                for (int w = 1; w < kAttendWaves; ++w) top = __builtin_fmaxf(top, sm_m[w][i]);
#pragma unroll
                for (int w = 0; w < kAttendWaves; ++w) sum += sm_l[w][i] * rescale(sm_m[w][i], top);
                if (!Full && d >= dim) continue;
                f32x4 x = *reinterpret_cast<const f32x4 *>(&sm_o[i * kLd + d]);
                if (whole) {
                    const std::int64_t row = row0 + i;
                    x = x / sum;
                    if (seen.beyond(row)) x = x * __builtin_nanf("");
                    __builtin_memcpy(p.O + (s.row0 + row / R) * p.ldo + (head * R + row % R) * p.hso + d, &x, sizeof(x));
                } else {
                    const std::int64_t at = (((std::int64_t(seq) * p.c.heads + head) * p.plan.tiles + tile) * p.plan.splits + split) * kRows + i;
                    *reinterpret_cast<f32x4 *>(p.ws + at * (dim + 4) + d) = x;
                    if (d == 0) p.ws[at * (dim + 4) + dim] = top, p.ws[at * (dim + 4) + dim + 1] = sum;
                }
            }
            __syncthreads();
        }
    }
}

template <class T, int DC, bool Full, int MT, bool Rows> hipError_t launch_kv4_kernel(const Kv4AttendProblem &p, hipStream_t stream)
{
    const std::int64_t per_seq = std::int64_t(p.plan.tiles) * p.c.heads * p.plan.splits;
    std::int64_t seqs = (std::int64_t(1) << 23) / per_seq;  // splits > 1: all of them (plan_kv4_attend)
    seqs = seqs < 1 ? 1 : seqs < p.b.seqs ? seqs : p.b.seqs;
    Kv4AttendProblem q = p;
    void *args[] = {&q};
    hipError_t e = hipLaunchKernel(reinterpret_cast<const void *>(&kv4_attend_kernel<T, DC, Full, MT, Rows>), dim3(unsigned(per_seq * seqs)),
                                   dim3(64 * kAttendWaves), args, 0, stream);
    if (e != hipSuccess || p.plan.splits == 1) return e;
    const unsigned units = unsigned(p.plan.tiles) * unsigned(p.c.heads) * unsigned(p.b.seqs);
    return hipLaunchKernel(reinterpret_cast<const void *>(&kv_join_kernel<Kv4AttendProblem, MT>), dim3(units * (4 * MT)), dim3(256), args, 0, stream);
}

template <class T, int DC, bool Full> hipError_t launch_kv4_shape(const Kv4AttendProblem &p, hipStream_t stream)
{
    constexpr int kMost = DC > 4 ? 1 : 2;  // plan_kv4_attend gives no more
    if (p.plan.rows) return launch_kv4_kernel<T, DC, Full, kMost, true>(p, stream);
    return p.plan.mt == 1 ? launch_kv4_kernel<T, DC, Full, 1, false>(p, stream) : launch_kv4_kernel<T, DC, Full, kMost, false>(p, stream);
}

template <class T> hipError_t launch_kv4(const Kv4AttendProblem &p, hipStream_t stream)
{
    switch (p.c.dim) {
    case 64: return launch_kv4_shape<T, 2, true>(p, stream);
    case 128: return launch_kv4_shape<T, 4, true>(p, stream);
    case 256: return launch_kv4_shape<T, 8, true>(p, stream);
    }
    if (p.c.dim < 64) return launch_kv4_shape<T, 2, false>(p, stream);
    return p.c.dim < 128 ? launch_kv4_shape<T, 4, false>(p, stream) : launch_kv4_shape<T, 8, false>(p, stream);
}

}  // namespace
}  // namespace sgemm_impl
