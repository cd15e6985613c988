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

#include <type_traits>

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

// An element that all lanes read, of an array that no kernel writes meanwhile:
// through the constant address space it becomes a scalar load, which no wait
// for a vector load holds up.
template <class V> __device__ inline V uniform_load(const V *p, std::int64_t i)
{
    return reinterpret_cast<const __attribute__((address_space(4))) V *>(reinterpret_cast<std::uintptr_t>(p))[i];
}

// The bytes of a word that are e4m3 NaN, as 0x80 in each such byte.
__device__ inline std::uint32_t nan_codes(std::uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

__device__ inline bool finite(float x) { return (f32_bits(x) & 0x7f800000u) != 0x7f800000u; }

// Eight weights p * scale, p >= 0, as three bf16 parts that add up to them
// exactly (split3 without its care for infinities: a weight that is not
// finite makes its whole row NaN in any case).
__device__ inline void split_weights(const float *w, Frag &hi, Frag &mid, Frag &lo)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float h[2], m[2], l[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float x = w[2 * i + j];
            h[j] = bits_f32(f32_bits(x) & 0xffff0000u);
            const float r = x - h[j];
            m[j] = bits_f32(f32_bits(r) & 0xffff0000u);
            l[j] = r - m[j];
        }
        hi.v[i] = pack_hi(h[0], h[1]);
        mid.v[i] = pack_hi(m[0], m[1]);
        lo.v[i] = pack_hi(l[0], l[1]);
    }
}

// The factor that brings a sum with maximum m to maximum top.
__device__ inline float rescale(float m, float top) { return m == top ? 1.0f : __builtin_amdgcn_exp2f(m - top); }

// What the rows of one tile see: row `row` of a sequence (row / R th new row,
// query head row % R of the group) sees `count` tokens from `from` on, of
// those that the table can name (from + count <= nameable).
struct Kv8Seen {
    std::int64_t first, len, nameable;  // position of new row 0, tokens, tokens that the table can name
    int R, causal, window;
    __device__ std::int64_t behind(std::int64_t row) const { return causal ? first + row / R + 1 : len; }
    __device__ void operator()(std::int64_t row, int &from, int &count) const
    {
        const std::int64_t end = behind(row), begin = window > 0 ? end - window : 0;
        const std::int64_t hi = end < 0 ? 0 : end < nameable ? end : nameable, lo = begin < 0 ? 0 : begin < hi ? begin : hi;
        from = int(lo);
        count = int(hi - lo);
    }
    // The last token seen lies behind the table's last column: the row is NaN.
    __device__ bool beyond(std::int64_t row) const { return behind(row) > nameable; }
};

// Waves a SIMD has registers for: two, but for the longest heads and for two
// groups of float32 rows (three parts of Q each).
template <class T> constexpr int kv8_waves_per_simd(int DC, int MT) { return DC > 4 || (DC == 4 && MT == 2 && sizeof(typename T::elem) == 4) ? 1 : 2; }

// DC: a head of up to 32 DC components; Full: of exactly that many. MT: groups
// of 16 rows a wave holds. Rows: the four waves of a work-group take row tiles
// of their own (prompts: the same keys and values pass through the compute
// unit's cache for all four). Otherwise they take the tokens of one row tile
// in turns of 32 and add their sums through LDS in the waves' order, and
// `splits` work-groups share the tile's tokens: each leaves its sums in the
// workspace and kv8_join_kernel adds them.
//
// Keys of the next 32 tokens are loaded into the registers of the last ones
// as soon as their scores are formed, values likewise after their product:
// each has half a turn to arrive. No load is conditional (that would make the
// compiler wait for all of them): pages that may not be read are replaced by
// page 0 and their scores by NaN.
//
// 32 sequences of up to 8192 tokens, 8 heads of 128 with 4 query heads each
// (0.41 GB): 82.6 us, 4.9 TB/s, bound by memory. 2 prompts of 1024 rows behind
// 4096 tokens in f16: 260 us, 460 TFLOP/s, bound by the SIMDs: matrix
// instructions take 43% of the cycles a compute unit is busy, the softmax and
// the conversion of codes 55%. No vector register is spilled; the table,
// scales and addresses take more scalar registers than there are (29 to 284 go
// to vector registers; for padded heads of 144 to 240 components 48 bytes a
// lane go to scratch).
template <class T, int DC, bool Full, int MT, bool Rows>
__global__ __launch_bounds__(64 * kAttendWaves, kv8_waves_per_simd<T>(DC, MT)) void kv8_attend_kernel(Kv8AttendProblem p)
{
    constexpr int PD = 32 * DC, kRows = 16 * MT, kDTiles = 2 * DC, kLd = PD + 4;
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
    // Lanes past the head's components read its first ones: keys are then
    // zeroed, values give components that are not stored.
    const int k_at = c * dim, v_at = 4 * kq * dim + (Full || c * 2 * DC < dim ? c * 2 * DC : 0);

    for (unsigned seq = id / unsigned(p.c.heads); seq < unsigned(p.b.seqs); seq += seqs_at_once) {
        const Kv8Sequence s = kv8_sequence(p.b, int(seq));
        const std::int64_t all_rows = s.n * R;
        const Kv8Seen seen{s.len - s.n, s.len, std::int64_t(p.b.table_ld) << shift, R, p.causal, p.window};
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
            QOperand<T> q[MT][DC];
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                std::int64_t row = row0 + 16 * t + c;
                row = row < all_rows ? row : all_rows - 1;
                seen(row, lo_t[t], n_t[t]);
                const elem *src = static_cast<const elem *>(p.Q) + (s.row0 + row / R) * p.ldq + (head * R + row % R) * p.hsq;
#pragma unroll
                for (int i = 0; i < DC; ++i) q[t][i].load(src + (kq * DC + i) * 8, Full || (kq * DC + i) * 8 < dim);
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

            // The page of a half turn, and its offset in codes; NaN scales where it may not be read.
            struct Half {
                const std::uint8_t *k, *v;
                float ks, vs;
            };
            auto half_at = [&](int t) {
                // Past the tokens seen (limit <= nameable) any page of the table will do; none is named by an empty one.
                const int page = uniform_load(table, (t < limit ? t : limit - 1) >> shift);
                const bool good = unsigned(page) < unsigned(p.c.pages);
                const std::int64_t at = std::int64_t(good ? page : 0) * p.c.heads + head;
                const std::int64_t byte0 = ((at << shift) + (t & (block - 1))) * dim;
                Half h{codes_k + byte0, codes_v + byte0, uniform_load(p.c.Ks, at), uniform_load(p.c.Vs, at)};
                if (!good) h.ks = h.vs = __builtin_nanf("");
                return h;
            };
            u32x2 k[2][DC];
            std::uint32_t v[8][DC / 2];
            auto load_keys = [&](const Half (&h)[2]) {
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int i = 0; i < DC; ++i) {
                        const int d = (kq * DC + i) * 8;
                        const bool there = Full || d < dim;
                        k[x][i] = *reinterpret_cast<const u32x2 *>(h[x].k + k_at + (there ? d : 0));
                        if (!Full) k[x][i] = there ? k[x][i] : u32x2{0, 0};
                    }
            };
            auto load_values = [&](const Half (&h)[2]) {
#pragma unroll
                for (int e = 0; e < 8; ++e) __builtin_memcpy(v[e], h[e / 4].v + v_at + (e % 4) * dim, 2 * DC);
            };

            // Turns from .. to, this wave's among them; Cut: some row does not see all of a turn.
            auto turns = [&](int from, int to, auto cut_) {
                constexpr bool Cut = decltype(cut_)::value;
                constexpr int kStride = Rows ? 1 : kAttendWaves;
                int turn = from + (Rows ? 0 : (wave - from) & (kAttendWaves - 1));
                if (turn >= to) return;
                // A scale of V that is not finite makes every row that sees the page NaN, whatever its weights: by
                // the scores, of which a row takes those that it sees.
                auto checked = [](Half h) {
                    if (!finite(h.vs)) h.ks = __builtin_nanf("");
                    return h;
                };
                Half now[2] = {checked(half_at(32 * turn)), checked(half_at(32 * turn + 16))};
                load_keys(now);
                load_values(now);
                for (; turn < to; turn += kStride) {
                    const int t0 = 32 * turn, tn = turn + kStride < to ? 32 * (turn + kStride) : t0;
                    const Half next[2] = {half_at(tn), half_at(tn + 16)};
                    float z[MT][8];
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int t = 0; t < MT; ++t) {
                            f32x4 acc = {0, 0, 0, 0};
#pragma unroll
                            for (int i = 0; i < DC; ++i) acc = q[t][i].scores(k[x][i], acc);
#pragma unroll
                            for (int r = 0; r < 4; ++r) z[t][4 * x + r] = acc[r] * (now[x].ks * factor);
                        }
                    load_keys(next);
                    bool poisoned = false;
                    if (Cut) {
                        // NaN codes must not reach rows that do not see them (0 * NaN):
                        // they leave the product and are put back below.
                        std::uint32_t any = 0;
#pragma unroll
                        for (int e = 0; e < 8; ++e)
#pragma unroll
                            for (int i = 0; i < DC / 2; ++i) {
                                const std::uint32_t nan = nan_codes(v[e][i]);
                                any |= nan;
                                v[e][i] &= ~((nan >> 7) * 0xffu);
                            }
                        poisoned = __ballot(any != 0) != 0;
                    }
                    Frag ph[MT], pm[MT], pl[MT];
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        if (Cut) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const unsigned j = unsigned(t0 + 16 * (e / 4) + 4 * kq + e % 4 - lo_t[t]);
                                z[t][e] = j < unsigned(n_t[t]) ? z[t][e] : -__builtin_inff();
                            }
                        }
                        float top = __builtin_fmaxf(z[t][0], z[t][1]);
#pragma unroll
                        for (int e = 2; e < 8; ++e) top = __builtin_fmaxf(top, z[t][e]);
                        top = column_max(top);
                        if (__ballot(top > m[t]) != 0) {
                            const float risen = __builtin_fmaxf(m[t], top), a = rescale(m[t], risen);
                            m[t] = risen;
                            l[t] *= a;
#pragma unroll
                            for (int j = 0; j < kDTiles; ++j) o[t][j] *= a;
                        }
                        const float base = m[t] == -__builtin_inff() ? 0.0f : m[t];
                        float w[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float pe = __builtin_amdgcn_exp2f(z[t][e] - base);
                            l[t] += pe;
                            w[e] = pe * now[e / 4].vs;
                            if (Cut) w[e] = z[t][e] == -__builtin_inff() ? 0.0f : w[e];
                        }
                        split_weights(w, ph[t], pm[t], pl[t]);
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
                        for (int t = 0; t < MT; ++t)
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                f32x4 &acc = o[t][4 * i + j];
                                acc = mfma_bf16(f[j], ph[t], mfma_bf16(f[j], pm[t], mfma_bf16(f[j], pl[t], acc)));
                            }
                    }
                    if (Cut && poisoned) {
                        for (int u = 0; u < 32; ++u) {
                            const float vs = u < 16 ? now[0].vs : now[1].vs;
                            if (vs != vs) continue;  // NaN already
                            const std::uint8_t *row = (u < 16 ? now[0].v : now[1].v) + (u % 16) * dim;
#pragma unroll
                            for (int x = 0; x < 4 * kDTiles; ++x) {
                                const int d = kq * 8 * DC + x;  // component of register x / kDTiles of d-tile x % kDTiles
                                if (d >= dim || (row[d] & 0x7f) != 0x7f) continue;
#pragma unroll
                                for (int t = 0; t < MT; ++t)
                                    if (unsigned(t0 + u - lo_t[t]) < unsigned(n_t[t])) o[t][x % kDTiles][x / kDTiles] = __builtin_nanf("");
                            }
                        }
                    }
                    load_values(next);
                    now[0] = checked(next[0]);
                    now[1] = checked(next[1]);
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

// Adds the sums that the splits of a row tile left in the workspace, in their
// order: one wave for each row (32 sequences of 8192 tokens in 3 splits: 5 us,
// most of it the launch).
template <int MT> __global__ __launch_bounds__(256) void kv8_join_kernel(Kv8AttendProblem p)
{
    constexpr int kRows = 16 * MT;
    const int lane = threadIdx.x & 63, R = p.heads_q / p.c.heads, dim = p.c.dim, splits = p.plan.splits;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const unsigned unit = blockIdx.x / (kRows / 4), i = blockIdx.x % (kRows / 4) * 4 + unsigned(wave);
    const int tile = int(unit % unsigned(p.plan.tiles)), head = int(unit / unsigned(p.plan.tiles) % unsigned(p.c.heads));
    const int seq = int(unit / unsigned(p.plan.tiles) / unsigned(p.c.heads));
    const Kv8Sequence s = kv8_sequence(p.b, seq);
    const std::int64_t row = std::int64_t(tile) * kRows + i;
    if (row >= s.n * R) return;
    const float *const part = p.ws + (std::int64_t(unit) * splits * kRows + i) * (dim + 4);
    const std::int64_t pitch = std::int64_t(kRows) * (dim + 4);
    // Lane x: split x's maximum and sum (at most 64 splits).
    float m = -__builtin_inff(), l = 0.0f;
    if (lane < splits) m = part[lane * pitch + dim], l = part[lane * pitch + dim + 1];
    float top = m;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, d));
    // A split that saw nothing of its row weighs nothing, and its components were left as sums of nothing: zeros.
    const float a = l == 0.0f ? 0.0f : rescale(m, top);
    float sum = l * a;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
    f32x4 y = {0, 0, 0, 0};
    const float *const at = part + (4 * lane < dim ? 4 * lane : 0);
    int x = 0;
    for (; x + 4 <= splits; x += 4) {
        f32x4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const f32x4 *>(at + (x + i) * pitch);
#pragma unroll
        for (int i = 0; i < 4; ++i) y += v[i] * __shfl(a, x + i);
    }
    for (; x < splits; ++x) y += *reinterpret_cast<const f32x4 *>(at + x * pitch) * __shfl(a, x);
    if (4 * lane >= dim) return;
    y = y / sum;
    const Kv8Seen seen{s.len - s.n, s.len, std::int64_t(p.b.table_ld) * p.c.block, R, p.causal, p.window};
    if (seen.beyond(row)) y = y * __builtin_nanf("");
    __builtin_memcpy(p.O + (s.row0 + row / R) * p.ldo + (head * R + row % R) * p.hso + 4 * lane, &y, sizeof(y));
}

template <class T, int DC, bool Full, int MT, bool Rows> hipError_t launch_attend_kernel(const Kv8AttendProblem &p, hipStream_t stream)
{
    const std::int64_t per_seq = std::int64_t(p.plan.tiles) * p.c.heads * p.plan.splits;
    std::int64_t seqs = (std::int64_t(1) << 23) / per_seq;  // splits > 1: all of them (plan_kv8_attend)
    seqs = seqs < 1 ? 1 : seqs < p.b.seqs ? seqs : p.b.seqs;
    Kv8AttendProblem q = p;
    void *args[] = {&q};
    hipError_t e = hipLaunchKernel(reinterpret_cast<const void *>(&kv8_attend_kernel<T, DC, Full, MT, Rows>), dim3(unsigned(per_seq * seqs)),
                                   dim3(64 * kAttendWaves), args, 0, stream);
    if (e != hipSuccess || p.plan.splits == 1) return e;
    const unsigned units = unsigned(p.plan.tiles) * unsigned(p.c.heads) * unsigned(p.b.seqs);
    return hipLaunchKernel(reinterpret_cast<const void *>(&kv8_join_kernel<MT>), dim3(units * (4 * MT)), dim3(256), args, 0, stream);
}

template <class T, int DC, bool Full> hipError_t launch_attend_shape(const Kv8AttendProblem &p, hipStream_t stream)
{
    constexpr int kMost = DC > 4 ? 1 : 2;  // plan_kv8_attend gives no more
    if (p.plan.rows) return launch_attend_kernel<T, DC, Full, kMost, true>(p, stream);
    return p.plan.mt == 1 ? launch_attend_kernel<T, DC, Full, 1, false>(p, stream) : launch_attend_kernel<T, DC, Full, kMost, false>(p, stream);
}

template <class T> hipError_t launch_attend(const Kv8AttendProblem &p, hipStream_t stream)
{
    switch (p.c.dim) {
    case 64: return launch_attend_shape<T, 2, true>(p, stream);
    case 128: return launch_attend_shape<T, 4, true>(p, stream);
    case 256: return launch_attend_shape<T, 8, true>(p, stream);
    }
    if (p.c.dim < 64) return launch_attend_shape<T, 2, false>(p, stream);
    return p.c.dim < 128 ? launch_attend_shape<T, 4, false>(p, stream) : launch_attend_shape<T, 8, false>(p, stream);
}

}  // namespace
}  // namespace sgemm_impl
