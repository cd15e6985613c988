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
// A weight is 2^(x - m), x the score and m a little above the row's largest so
// far, so that the exponents of weights that count are small and float32 holds
// them well, whatever the values' scales. Codes are exact in f16, so a weight's
// product with its value's scale may be held in two parts of f16, 22 bits, where
// bf16 would need three for as many, and a matrix instruction of four is saved.
// f16's range is made enough by a power of two for each row, which the products
// are multiplied by (unit_of). A product is held to 2^-22 of itself, or to 2^-38
// of the row's largest where that is more. Tokens that a row does not see take
// no part in its largest, so their scales do not cost it precision. (With the
// exponent of a value's scale in m no factor is needed, but the exponential's
// argument is as large as that exponent: weights at scales of 2^-80 were off by
// 52 units of 2^-24, now by 5 at any scale.)
//
// While a wave feeds the matrix cores in a prompt its priority is raised: the
// other wave of the SIMD then finds its vector instructions' turn while those
// run.
//
// Both steps when they were taken, at 2 prompts of 1024 rows behind 4096 tokens, in
// f16: three parts of bf16 259 us, two of f16 228, with the priority 216.
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
    __device__ f32x4 scores(std::uint32_t k, f32x4 acc) const
    {
        const Frag a{{fp4_bf16<0>(k), fp4_bf16<1>(k), fp4_bf16<2>(k), fp4_bf16<3>(k)}};
        return mfma_bf16(a, f, acc);
    }
};
template <> struct QOperand4<F16> {
    Frag f;
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

// Two float32 times a power of two as two parts of f16, hi + lo, each rounded to
// nearest: 22 bits and the sign, or down to 2^-24 for what lies below f16's normal
// numbers.
__device__ inline void split2(float a, float b, float power, std::uint32_t &hi, std::uint32_t &lo)
{
    a *= power, b *= power;
    hi = __builtin_bit_cast(std::uint32_t, f16x2{_Float16(a), _Float16(b)});
    float ra, rb;  // a - hi, b - hi: exact
    asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel_hi:[1,0,0]" : "=v"(ra) : "v"(hi), "v"(a));
    asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "=v"(rb) : "v"(hi), "v"(b));
    lo = __builtin_bit_cast(std::uint32_t, f16x2{_Float16(ra), _Float16(rb)});
}

// A lane's pieces of one query row, eight components each, of those that are
// `there`.
template <class T, int DC> struct QueryPieces {
    struct Piece {
        typename T::elem x[8];
    } r[DC];
    template <class There> __device__ void load(const typename T::elem *src, There &&there)
    {
#pragma unroll
        for (int i = 0; i < DC; ++i) {
            __builtin_memset(&r[i], 0, sizeof(Piece));
            if (there(i)) r[i] = load_any<Piece>(src + 8 * i);
        }
    }
};

// The same as operands, and the factor that the row's scores are to be
// multiplied by. float32 rows are brought to a largest component of 2^14 to
// 2^15 by a power of two, so that their parts hold each component to 2^-22 of
// itself or 2^-39 of the largest. (A row with a component that is not finite
// has no finite score.)
template <class T, int DC> __device__ inline float query_operands(const QueryPieces<T, DC> &raw, QOperand4<T> (&q)[DC])
{
    if constexpr (sizeof(typename T::elem) == 2) {
#pragma unroll
        for (int i = 0; i < DC; ++i) q[i].f.v = __builtin_bit_cast(u32x4, raw.r[i]);
        return 1.0f;
    } else {
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < DC; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) top = __builtin_fmaxf(top, __builtin_fabsf(raw.r[i].x[j]));
        top = column_max(top);
        int field = 127 + 14 + 127 - int(f32_bits(top) >> 23);
        field = field > 253 ? 253 : field;
        const float up = bits_f32(std::uint32_t(field) << 23);
#pragma unroll
        for (int i = 0; i < DC; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                std::uint32_t hi, lo;
                split2(raw.r[i].x[2 * j], raw.r[i].x[2 * j + 1], up, hi, lo);
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

// The largest (sum) of a value over the P copies of a column's row.
template <int N> __device__ inline float turned(float x)  // from the lane N places before, around the 16 lanes of a row
{
    const int u = __builtin_bit_cast(int, x);
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(u, 0x120 + N, 0xf, 0xf, true));
}
template <int P> __device__ inline float copies_max(float x)
{
    if constexpr (P == 4) x = __builtin_fmaxf(x, turned<4>(x));
    if constexpr (P >= 2) x = __builtin_fmaxf(x, turned<8>(x));
    return x;
}
template <int P> __device__ inline float copies_sum(float x)
{
    if constexpr (P == 4) x += turned<4>(x);
    if constexpr (P >= 2) x += turned<8>(x);
    return x;
}

// How far above a row's largest score m is put when that rises beyond m, so that
// it seldom does again. Weights are then at most 1 and that of the largest score at
// least 2^-4, whose exponent float32 holds to 2^-23. Together with products that may
// grow to twice what their unit was made for: 2 prompts of 1024 behind 4096 206 us,
// with neither 219 to 229.
constexpr float kAbove = 4.0f;

// What a row's products of a weight and a scale are multiplied by, as the
// exponent of a power of two, given the largest of them: it comes to lie between
// 2^13 and 2^14, and has not to rise beyond 2^15. (Products below 2^-100 count as
// that. One that is not finite makes its row NaN in any case.)
__device__ inline int unit_of(float top)
{
    const int e = int(f32_bits(top) >> 23);
    return 127 + 13 - (e < 27 ? 27 : e);
}
__device__ inline float power(int e) { return bits_f32(std::uint32_t(127 + e) << 23); }  // 2^e, |e| < 127

// What sums of products that have the unit of largest product `from` are multiplied
// by to have that of `to` (at least a * from), where a larger m makes them a times as
// large: at most 2. One power of two, as of two factors one may overflow.
__device__ inline float to_unit(float a, float from, float to) { return __builtin_ldexpf(a, unit_of(to) - unit_of(from)); }

// Sums of products with the unit of largest product `top`, without it.
__device__ inline f32x4 in_values(f32x4 x, float top)
{
    const int e = -unit_of(top);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = __builtin_ldexpf(x[j], e);
    return x;
}

// Pair e of the four pairs of weights of a row that its P copies hold in order,
// in the lanes of the first copy. (What the others get is another row's.)
template <int P, int N> __device__ inline std::uint32_t from_copy(const std::uint32_t (&own)[N], int e)
{
    const std::uint32_t x = own[e % N];
    if (e / N == 0) return x;
    const int u = int(x);
    if (P == 2 || e / N == 2) return std::uint32_t(__builtin_amdgcn_mov_dpp(u, 0x120 + 8, 0xf, 0xf, true));
    return std::uint32_t(e / N == 1 ? __builtin_amdgcn_mov_dpp(u, 0x120 + 12, 0xf, 0xf, true)
                                    : __builtin_amdgcn_mov_dpp(u, 0x120 + 4, 0xf, 0xf, true));
}

__device__ inline std::int64_t broadcast(std::int64_t x, int lane)
{
    const std::uint32_t lo = std::uint32_t(__builtin_amdgcn_readlane(int(std::uint32_t(x)), lane));
    const std::uint32_t hi = std::uint32_t(__builtin_amdgcn_readlane(int(std::uint32_t(std::uint64_t(x) >> 32)), lane));
    return std::int64_t(std::uint64_t(hi) << 32 | lo);
}

// a / b, by 32 bits where they are enough: a division of 64 takes over a
// hundred instructions.
__device__ inline std::int64_t divide(std::int64_t a, int b) { return a >> 31 ? a / b : std::int64_t(unsigned(a) / unsigned(b)); }

// kv8_sequence for a sequence that is the same in all lanes: by scalar loads,
// so that all that follows from it stays in scalar registers.
__device__ inline Kv8Sequence uniform_sequence(const sgemm_kv8_batch &b, int seq)
{
    auto cut = [&](int row) { return std::int64_t(row < 0 ? 0 : row < b.rows ? row : b.rows); };
    const std::int64_t row0 = cut(uniform_load(b.starts, seq)), end = cut(uniform_load(b.starts, std::int64_t(seq) + 1));
    const int len = uniform_load(b.lens, seq);
    return {seq, len > 0 ? len : 0, end > row0 ? end - row0 : 0, row0};
}

// How the turns (32 tokens each) that a tile of rows sees are shared out when
// rows are few: those of all sequences in one row, in equal parts to `slots`
// work-groups, whatever the sequences' lengths. A part may end within a
// sequence and go on in the next. Slot g takes turns g T / G .. (g + 1) T / G;
// turn x belongs to slot ((x + 1) G - 1) / T. A part of a sequence that slot g
// does has the number g + seq, which no other part of the tile has.
struct Kv4Shares {
    std::int64_t total;  // T
    int slots;           // G: every slot has a turn
    __device__ std::int64_t begin(int slot) const { return divide(total * slot, slots); }
    __device__ int slot_of(std::int64_t turn) const { return int(total >> 31 ? ((turn + 1) * slots - 1) / total : divide((turn + 1) * slots - 1, int(total))); }
};

// How a sequence's tile of rows was shared out, behind the parts in the
// workspace: the work-group that does its first part leaves this for the join.
struct Kv4Split {
    int slot, count;  // first slot; parts, or 0 if that one did all of it
};
static_assert(sizeof(Kv4Split) == kKv4SplitBytes, "the workspace has room for it");
__device__ inline Kv4Split *kv4_split(const Kv4AttendProblem &p, int tile_rows, std::int64_t unit, int seq)
{
    const std::int64_t floats = std::int64_t(p.c.heads) * p.plan.tiles * p.plan.parts * tile_rows * (p.c.dim + 4);
    return reinterpret_cast<Kv4Split *>(p.ws + floats) + unit * p.b.seqs + seq;
}

// Turns of a sequence that new rows `r_first` .. `r_last` see; one where it has
// rows but they see nothing (somebody has to say so), none without rows.
__device__ inline int kv4_turns(const Kv4AttendProblem &p, const Kv8Sequence &s, std::int64_t r_first, std::int64_t r_last, int shift)
{
    if (r_first >= s.n) return 0;
    const KvSeen seen{s.len - s.n, s.len, std::int64_t(p.b.table_ld) << shift, 1, p.causal, p.window};
    int from, count, last, more;
    seen.by_new(r_first, from, count);
    seen.by_new(r_last < s.n ? r_last : s.n - 1, last, more);
    const int turns = int((unsigned(last + more) + 31u) >> 5) - (from >> 5);
    return turns < 1 ? 1 : turns;
}

// A value of the lane that the data-parallel primitive `Ctrl` names, in the rows
// of 16 lanes of `Rows`; 0 elsewhere and past a row's first lane.
template <int Ctrl, int Rows> __device__ inline std::int64_t shifted(std::int64_t x)
{
    const std::uint32_t lo = std::uint32_t(__builtin_amdgcn_update_dpp(0, int(std::uint32_t(x)), Ctrl, Rows, 0xf, false));
    const std::uint32_t hi = std::uint32_t(__builtin_amdgcn_update_dpp(0, int(std::uint32_t(std::uint64_t(x) >> 32)), Ctrl, Rows, 0xf, false));
    return std::int64_t(std::uint64_t(hi) << 32 | lo);
}

// 64 sequences from `first` on, one a lane: the sequence (none past the last),
// its turns, and those of all sequences up to it.
struct Kv4Group {
    Kv8Sequence s;
    int turns;
    std::int64_t upto;
};
__device__ inline Kv4Group kv4_group(const Kv4AttendProblem &p, int first, std::int64_t before, std::int64_t r_first, std::int64_t r_last, int shift, int lane)
{
    Kv4Group g = {{first + lane, 0, 0, 0}, 0, 0};
    if (first + lane < p.b.seqs) {
        g.s = kv8_sequence(p.b, first + lane);
        g.turns = kv4_turns(p, g.s, r_first, r_last, shift);
    }
    // Sums over the lanes before within each 16, then the last lanes' of the 16 and of the 32 before.
    std::int64_t x = g.turns;
    x += shifted<0x111, 0xf>(x);
    x += shifted<0x112, 0xf>(x);
    x += shifted<0x114, 0xf>(x);
    x += shifted<0x118, 0xf>(x);
    x += shifted<0x142, 0xa>(x);
    x += shifted<0x143, 0xc>(x);
    g.upto = x;
    g.upto += before;
    return g;
}

// The shares, given the first group.
__device__ inline Kv4Shares kv4_shares(const Kv4AttendProblem &p, const Kv4Group &g0, std::int64_t r_first, std::int64_t r_last, int shift, int lane)
{
    std::int64_t total = broadcast(g0.upto, 63);
    for (int first = 64; first < p.b.seqs; first += 64) total = broadcast(kv4_group(p, first, total, r_first, r_last, shift, lane).upto, 63);
    const std::int64_t most = total / kKv4LeastTurns;
    return {total, int(most < 1 ? 1 : most < p.plan.slots ? most : p.plan.slots)};
}

// Few rows: the four waves of a work-group take the turns of one row tile in
// turn and add their sums through LDS, and the tile's turns over all sequences
// are shared out to `slots` work-groups (Kv4Shares): what a work-group does of
// a sequence that others work on too is left in the workspace, and
// kv4_join_kernel adds it.
//
// A tile has 16 rows, or 16 / P where there are no more: the columns of the
// matrix instruction then hold each row P times over, every copy takes a P-th of
// the tokens through the softmax, and the weights come back to the first copy
// for the second product.
//
// Codes and scales of the next turn are loaded as soon as this one's have gone
// into the first product and been regrouped, before its softmax; nothing that
// is loaded is looked at before its turn, so that no wait comes early. Pages
// that may not be read are replaced by page 0 and their scores by NaN.
//
// Where a sequence's keys are read by one tile only and one load of a wave
// covers whole lines (64 and 128 components), they are kept out of the caches. In a
// graph of three batches in turn, 32 x 8192 tokens of 128 components 50.0 us
// instead of 55.4, 64 x 4096 50.8 instead of 56.3, 32 x 4096 33.9 instead of 35.3, of 64
// components 38.6, 38.6 and 29.1 instead of 39.2, 39.9 and 28.7; up to 32 x 2000 no
// difference beyond 3% either way. One batch alone, again and again, that the chip's
// caches hold whole loses up to 3% (32 x 8192 47.9 instead of 47.3, 64 x 4096 of 64
// components 38.6 instead of 37.7). So the rule has no size in it. Values, whose lines take several
// loads, lost by it (51.7 with both when keys alone took 50.3), and so did keys of 80
// components (34.8 -> 36.1), 192 and 256.
//
// 32 sequences of up to 8192 tokens, 8 heads of 128 with 4 query heads each
// (0.21 GB): 41.8 us, 5.0 TB/s, and 4.8 for the join; with equal splits of each
// sequence instead of equal shares, and no copies, 10% more. Bound by memory.
template <class T, int DC, bool Full, int P>
__global__ __launch_bounds__(64 * kAttendWaves, DC <= (P == 1 ? 2 : 4) ? 3 : 2)  // as many a compute unit as plan_kv4_attend counts on
void kv4_few_kernel(Kv4AttendProblem p)
{
    constexpr int PD = 32 * DC, kRows = 16 / P, kDTiles = 2 * DC, kLd = PD + 4, kVWords = (DC + 3) / 4, E = 8 / P;
    __shared__ float sm_m[kAttendWaves][kRows], sm_l[kAttendWaves][kRows], sm_top[kAttendWaves][kRows];
    __shared__ __align__(16) float sm_o[kAttendWaves][kRows * kLd];
    typedef typename T::elem elem;
    const int lane = threadIdx.x & 63, c = lane & 15, kq = lane >> 4, copy = c / kRows;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int dim = Full ? PD : p.c.dim, R = p.heads_q / p.c.heads;
    const int shift = 31 - __builtin_clz(unsigned(p.c.block)), block = 1 << shift;

    unsigned id = blockIdx.x;
    const unsigned slots = p.plan.slots ? unsigned(p.plan.slots) : 1u;
    const int slot = int(id % slots);
    id /= slots;
    const int tile0 = int(id % unsigned(p.plan.tiles));
    id /= unsigned(p.plan.tiles);
    const int head = int(id % unsigned(p.c.heads));
    const unsigned seq0 = id / unsigned(p.c.heads), seqs_at_once = gridDim.x / (slots * unsigned(p.plan.tiles) * unsigned(p.c.heads));
    const float factor = p.scale * kLog2e;
    const std::uint8_t *const codes_k = static_cast<const std::uint8_t *>(p.c.K), *const codes_v = static_cast<const std::uint8_t *>(p.c.V);
    const std::uint16_t *const scales_k = static_cast<const std::uint16_t *>(p.c.Ks), *const scales_v = static_cast<const std::uint16_t *>(p.c.Vs);
    // Lanes past the head's components read its first ones: their queries are
    // zero, their values give components that are not stored.
    const int v_at = 4 * kq * (dim / 2) + (Full || c * 2 * DC < dim ? c * DC : 0);
    int k_at[(DC + 1) / 2];  // of 16 components each
#pragma unroll
    for (int i = 0; i < DC; i += 2) k_at[i / 2] = c * (dim / 2) + (Full || (kq * DC + i) * 8 < dim ? (kq * DC + i) * 4 : 0);

    // Turns `from` .. `to` of those that a sequence's rows `tile` see; `part`: the workspace's, or -1 for all of them.
    auto piece = [&](const Kv8Sequence &s, std::int64_t tile, int from, int to, int part) {
        const int seq = s.seq;
        const std::int64_t all_rows = s.n * R, row0 = tile * kRows;
        const KvSeen seen{s.len - s.n, s.len, std::int64_t(p.b.table_ld) << shift, 1, p.causal, p.window};
        const int *const table = p.b.table + std::int64_t(seq) * p.b.table_ld;
        const int rows = int(all_rows - row0 < kRows ? all_rows - row0 : kRows);
        const std::int64_t fresh0 = divide(row0, R);
        const int rest0 = int(row0 - fresh0 * R);  // row i of the tile: new row fresh0 + (rest0 + i) / R, its query head (rest0 + i) % R

        // Each lane's row: what it sees, and its operands. Rows past the last
        // repeat it; what they give is not stored.
        int lo_t, n_t;  // first token seen, tokens seen
        QueryPieces<T, DC> raw;
        const int row = rest0 + (c % kRows < rows ? c % kRows : rows - 1);
        const int fresh = int(unsigned(row) / unsigned(R));
        seen.by_new(fresh0 + fresh, lo_t, n_t);
        const elem *src = static_cast<const elem *>(p.Q) + (s.row0 + fresh0 + fresh) * p.ldq + (head * R + row - fresh * R) * p.hsq;
        raw.load(src + kq * DC * 8, [&](int i) { return Full || (kq * DC + i) * 8 < dim; });
        int first_lo, first_n, last_lo, last_n;
        seen.by_new(fresh0, first_lo, first_n);
        seen.by_new(fresh0 + unsigned(rest0 + rows - 1) / unsigned(R), last_lo, last_n);
        // Turns of 32 tokens: begin .. end sees some row; inner .. outer every row in full.
        // (Positions reach 2^31 - 1, so that rounding up needs the sign bit.)
        const int limit = last_lo + last_n, begin = first_lo >> 5, last = int((unsigned(limit) + 31u) >> 5);
        const int inner = int((unsigned(last_lo) + 31u) >> 5), outer = (first_lo + first_n) >> 5;
        const int end = to < last - begin ? begin + to : last;

        f32x4 o[kDTiles] = {};
        float m = -__builtin_inff(), l = 0.0f;            // what scores are relative to; sum of the weights
        float top_w = 0.0f, unit = power(unit_of(0.0f));  // largest product when the unit was made; what products are multiplied by

        QOperand4<T> q[DC];
        float row_factor;
        // One turn's codes and scales, and whether its halves' pages may be read.
        std::uint32_t k[2][DC], v[8][kVWords];
        struct Scales {
            std::uint32_t k[E / 2], v[E / 2];
            bool good[2];
        } scales;
        struct Place {
            std::int64_t token[2];
            bool good[2];
        };
        auto place_of = [&](int turn) {
            Place w;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                // Past the tokens seen (limit <= nameable) any page of the table will do; none is named by an empty one.
                const int t = 32 * turn + 16 * x, page = uniform_load(table, (t < limit ? t : limit - 1) >> shift);
                w.good[x] = unsigned(page) < unsigned(p.c.pages);
                w.token[x] = ((std::int64_t(w.good[x] ? page : 0) * p.c.heads + head) << shift) + (t & (block - 1));
            }
            return w;
        };
        auto load_keys = [&](const Place &w) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const std::uint8_t *const at = codes_k + w.token[x] * (dim / 2);
                if constexpr (Full && P > 1 && DC <= 4) {
                    typedef std::uint32_t words __attribute__((ext_vector_type(DC)));
                    const words w = __builtin_nontemporal_load(reinterpret_cast<const words *>(at + k_at[0]));
                    __builtin_memcpy(k[x], &w, sizeof(w));
                } else if (Full) {
                    __builtin_memcpy(k[x], at + k_at[0], 4 * DC);
                } else {
#pragma unroll
                    for (int i = 0; i < DC; i += 2) __builtin_memcpy(&k[x][i], at + k_at[i / 2], 8);
                }
            }
        };
        auto load_values = [&](const Place &w) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const std::uint8_t *const at = codes_v + w.token[x] * (dim / 2) + v_at;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (DC == 2) v[4 * x + e][0] = load_any<std::uint16_t>(at + e * (dim / 2));
                    else __builtin_memcpy(v[4 * x + e], at + e * (dim / 2), DC);
                }
            }
        };
        auto load_scales = [&](const Place &w) {
            Scales r;
            r.good[0] = w.good[0];
            r.good[1] = w.good[1];
            // Those of this lane's copy: E adjacent ones of a half, or four of both.
            if constexpr (P == 1) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    __builtin_memcpy(&r.k[2 * x], scales_k + w.token[x] + 4 * kq, 8);
                    __builtin_memcpy(&r.v[2 * x], scales_v + w.token[x] + 4 * kq, 8);
                }
            } else {
                const std::int64_t at = (copy * 2 / P ? w.token[1] : w.token[0]) + 4 * kq + copy * E % 4;
                __builtin_memcpy(r.k, scales_k + at, 2 * E);
                __builtin_memcpy(r.v, scales_v + at, 2 * E);
            }
            return r;
        };

        auto work = [&](int turn, int next) {
#pragma clang fp contract(off)  // a score is rounded before m is taken off it: equal scores are then equal to the bit, and none is above m
            const bool cut = turn < inner || turn >= outer;  // some row does not see all of the turn
            const Place then = place_of(next);
            f32x4 acc[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                acc[x] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < DC; ++i) acc[x] = q[i].scores(k[x][i], acc[x]);
            }
            load_keys(then);
            // Byte x of even (odd): component 2 x (2 x + 1) of the word, of tokens 2 e and 2 e + 1.
            std::uint32_t even[kVWords][4], odd[kVWords][4];
#pragma unroll
            for (int i = 0; i < kVWords; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const std::uint32_t a = v[2 * e][i], b = v[2 * e + 1][i];
                    even[i][e] = (a & 0x0f0f0f0fu) | ((b << 4) & 0xf0f0f0f0u);
                    odd[i][e] = ((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u);
                }
            load_values(then);
            const Scales own = scales;
            scales = load_scales(then);
            // Token i of this lane: number 16 * half + 4 kq + i % 4 of the turn.
            float g[E];
#pragma unroll
            for (int i = 0; i < E; ++i) {
                // x * 0 + x: a scale that is not finite becomes NaN.
                const float f = bits_f32(i & 1 ? own.k[i / 2] & 0xffff0000u : own.k[i / 2] << 16);
                g[i] = __builtin_fmaf(f, 0.0f, f) * factor;
            }
            if (!(own.good[0] && own.good[1])) {
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const bool good = P == 1 ? own.good[i / 4] : copy * 2 / P ? own.good[1] : own.good[0];
                    if (!good) g[i] = __builtin_nanf("");
                }
            }
            Frag ph, pl;
            float z[E];
#pragma unroll
            for (int i = 0; i < E; ++i) {
                if constexpr (P == 1) z[i] = acc[i / 4][i % 4];
                else if constexpr (P == 2) z[i] = copy ? acc[1][i] : acc[0][i];
                else {
                    const float a = copy & 1 ? acc[0][2 + i] : acc[0][i], b = copy & 1 ? acc[1][2 + i] : acc[1][i];
                    z[i] = copy & 2 ? b : a;
                }
                if (sizeof(elem) == 4) z[i] *= row_factor;
            }
            unsigned sees = ~0u;  // bits of the tokens that the row sees
#pragma unroll
            for (int i = 0; i < E; ++i) z[i] *= g[i];
            if (cut) {
                sees = 0;
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const int half = P == 1 ? i / 4 : copy * 2 / P, at = P == 1 ? i % 4 : copy * E % 4 + i;
                    const bool yes = unsigned(32 * turn + 16 * half + 4 * kq + at - lo_t) < unsigned(n_t);
                    z[i] = yes ? z[i] : -__builtin_inff();
                    sees |= yes ? 1u << i : 0u;
                }
            }
            float w[E], top = z[0], a = 1.0f;
#pragma unroll
            for (int i = 1; i < E; ++i) top = __builtin_fmaxf(top, z[i]);
            const bool risen = __ballot(top > m) != 0;
            if (risen) {
                top = column_max(copies_max<P>(top));
                const float to = top > m ? top + kAbove : m;
                a = rescale(m, to);
                m = to;
                l *= a;
            }
            const float base = __builtin_fmaxf(m, -3.402823466e38f);  // finite where a row has seen nothing
            float largest = 0.0f;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                float pe = __builtin_amdgcn_exp2f(z[i] - base);
                // A scale that is not finite makes the whole row NaN, by w or by its parts.
                w[i] = pe * bits_f32(i & 1 ? own.v[i / 2] & 0xffff0000u : own.v[i / 2] << 16);
                if (cut && !(sees >> i & 1)) pe = w[i] = 0.0f;
                l += pe;
                largest = __builtin_fmaxf(largest, __builtin_fabsf(w[i]));
            }
            if (risen || __ballot(0.5f * largest > top_w) != 0) {
                const float to = __builtin_fmaxf(top_w * a, column_max(copies_max<P>(largest)));
                const float b = to_unit(a, top_w, to);
#pragma unroll
                for (int j = 0; j < kDTiles; ++j) o[j] *= b;
                top_w = to;
                unit = power(unit_of(to));
            }
            std::uint32_t hi[E / 2], lo[E / 2];
#pragma unroll
            for (int i = 0; i < E / 2; ++i) split2(w[2 * i], w[2 * i + 1], unit, hi[i], lo[i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                ph.v[e] = from_copy<P>(hi, e);
                pl.v[e] = from_copy<P>(lo, e);
            }
#pragma unroll
            for (int i = 0; i < kVWords; ++i) {
                auto byte = [&](auto at_) {
                    constexpr int At = decltype(at_)::value;
                    Frag f[2];
#pragma unroll
                    for (int e = 0; e < 4; ++e) f[0].v[e] = fp4_f16<At>(even[i][e]), f[1].v[e] = fp4_f16<At>(odd[i][e]);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        f32x4 &sum = o[8 * i + 2 * At + j];
                        sum = mfma_f16(f[j], ph, mfma_f16(f[j], pl, sum));
                    }
                };
                byte(std::integral_constant<int, 0>{});
                byte(std::integral_constant<int, 1>{});
                if constexpr (DC > 2) {
                    byte(std::integral_constant<int, 2>{});
                    byte(std::integral_constant<int, 3>{});
                }
            }
        };
        int turn = begin + from + wave;
        if (turn < end) {
            // The first turn's codes are on their way before the queries, which came with the table, are looked at.
            const Place first = place_of(turn);
            load_keys(first);
            load_values(first);
            scales = load_scales(first);
            row_factor = query_operands<T, DC>(raw, q);
            for (; turn < end; turn += kAttendWaves) {
                const int next = turn + kAttendWaves < end ? turn + kAttendWaves : turn;
                work(turn, next);
            }
        }

        // The waves' sums, in LDS; then all onto the largest maximum.
        // A row that sees no token is 0 / 1; one whose scores are all -inf is 0 / 0.
        const float sum = column_sum(copies_sum<P>(l));
        if (c < kRows) {
            if (kq == 0) sm_m[wave][c] = m, sm_top[wave][c] = top_w, sm_l[wave][c] = n_t == 0 ? 1.0f : sum;
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int j = 0; j < kDTiles; j += 4)
                    *reinterpret_cast<f32x4 *>(&sm_o[wave][c * kLd + (4 * kq + r) * kDTiles + j]) =
                        f32x4{o[j][r], o[j + 1][r], o[j + 2][r], o[j + 3][r]};
        }
        __syncthreads();
        // A thread keeps one component quad of every 4 * 64 / (PD / 4)-th row.
        constexpr int kQuads = PD / 4, kStep = 64 * kAttendWaves / kQuads;
        const int d = int(threadIdx.x) % kQuads * 4;
        for (int i = int(threadIdx.x) / kQuads; i < rows; i += kStep) {
            float m = sm_m[0][i], top = 0.0f, sum = 0.0f;
#pragma unroll
            for (int w = 1; w < kAttendWaves; ++w) m = __builtin_fmaxf(m, sm_m[w][i]);
#pragma unroll
            for (int w = 0; w < kAttendWaves; ++w) top = __builtin_fmaxf(top, sm_top[w][i] * rescale(sm_m[w][i], m));
            f32x4 x = {0, 0, 0, 0};
#pragma unroll
            for (int w = 0; w < kAttendWaves; ++w) {
                const float a = rescale(sm_m[w][i], m);
                sum += sm_l[w][i] * a;
                x += *reinterpret_cast<const f32x4 *>(&sm_o[w][i * kLd + d]) * to_unit(a, sm_top[w][i], top);
            }
            if (!Full && d >= dim) continue;
            if (part < 0) {
                const int fresh = int(unsigned(rest0 + i) / unsigned(R));
                x = in_values(x / sum, top);
                if (seen.beyond_new(fresh0 + fresh)) x = x * __builtin_nanf("");
                __builtin_memcpy(p.O + (s.row0 + fresh0 + fresh) * p.ldo + (head * R + rest0 + i - fresh * R) * p.hso + d, &x, sizeof(x));
            } else {
                const std::int64_t at = ((std::int64_t(head) * p.plan.tiles + tile) * p.plan.parts + part) * kRows + i;
                *reinterpret_cast<f32x4 *>(p.ws + at * (dim + 4) + d) = x;
                if (d == 0) p.ws[at * (dim + 4) + dim] = m, p.ws[at * (dim + 4) + dim + 1] = sum, p.ws[at * (dim + 4) + dim + 2] = top;
            }
        }
        __syncthreads();
    };

    // Which pieces: first this work-group's share of the turns of tile `tile0`
    // of all sequences, then whole tiles: all of them without shares, those
    // beyond what the grid and the workspace were laid out for with them.
    constexpr int kAll = 1 << 30;
    const bool shared = p.plan.slots > 0;
    const std::int64_t r_first = divide(std::int64_t(tile0) * kRows, R), r_last = divide(std::int64_t(tile0) * kRows + kRows - 1, R);
    std::int64_t lo = 0, hi = 0, tile = tile0;
    Kv4Group g = {};
    std::uint64_t mine = 0;  // sequences of the 64 from `first` on that the share meets
    int first = 0;
    Kv4Shares shares = {};
    if (shared) {
        g = kv4_group(p, 0, 0, r_first, r_last, shift, lane);
        shares = kv4_shares(p, g, r_first, r_last, shift, lane);
        if (slot < shares.slots) lo = shares.begin(slot), hi = shares.begin(slot + 1);
        mine = __ballot(g.turns > 0 && g.upto > lo && g.upto - g.turns < hi);
    }
    bool whole = !shared;
    int seq = shared ? slot : int(seq0);
    const int step = shared ? p.plan.slots : int(seqs_at_once);
    if (shared) tile += p.plan.tiles;
    for (;;) {
        int from = 0, to = kAll, part = -1;
        Kv8Sequence s;
        std::int64_t at = tile0;
        if (!whole) {
            while (mine == 0) {
                const std::int64_t before = broadcast(g.upto, 63);
                first += 64;
                if (first >= p.b.seqs || before >= hi) {
                    whole = true;
                    break;
                }
                g = kv4_group(p, first, before, r_first, r_last, shift, lane);
                mine = __ballot(g.turns > 0 && g.upto > lo && g.upto - g.turns < hi);
            }
        }
        if (!whole) {
            const int b = __builtin_ctzll(mine);
            mine &= mine - 1;
            const int count = __builtin_amdgcn_readlane(g.turns, b);
            const std::int64_t start = broadcast(g.upto, b) - count;
            from = int(start < lo ? lo - start : 0);
            to = int(start + count > hi ? hi - start : count);
            part = from == 0 && to == count ? -1 : slot + first + b;
            s = {first + b, broadcast(g.s.len, b), broadcast(g.s.n, b), broadcast(g.s.row0, b)};
            if (from == 0 && threadIdx.x == 0)
                *kv4_split(p, kRows, std::int64_t(head) * p.plan.tiles + tile0, s.seq) =
                    {slot, to < count ? shares.slot_of(start + count - 1) - slot + 1 : 0};
        } else {
            if (seq >= p.b.seqs) break;
            s = uniform_sequence(p.b, seq);
            at = tile;
            tile += p.plan.tiles;
            if (at * kRows >= s.n * R) {
                seq = next_sequence(seq, step, p.b.seqs);
                tile = shared ? std::int64_t(tile0) + p.plan.tiles : tile0;
                continue;
            }
        }
        piece(s, at, from, to, part);
    }
}

// Adds the sums that several work-groups left of one sequence's tile of rows, as
// the work-group that did the first part says: W waves for each row, which take the
// parts in turn. One does while sequences have few parts on average (1820 rows of
// 4 parts: with four waves a row 8.5 us instead of 4.8); with more of them four
// wait for a quarter each. Those 1820 rows now take 4.0, most of it the launch
// and two round trips.
template <int Rows, int W> __global__ __launch_bounds__(256) void kv4_join_kernel(Kv4AttendProblem p)
{
    constexpr int kAtOnce = 4, kRowsHere = kAttendWaves / W;
    __shared__ float sm_m[kAttendWaves], sm_top[kAttendWaves], sm_sum[kAttendWaves];
    __shared__ __align__(16) float sm_x[W > 1 ? kAttendWaves : 1][256];
    const int lane = threadIdx.x & 63, R = p.heads_q / p.c.heads, dim = p.c.dim, shift = 31 - __builtin_clz(unsigned(p.c.block));
    const int all_waves = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wave = all_waves % W;
    const int i = int(blockIdx.x % (Rows / kRowsHere)) * kRowsHere + all_waves / W;
    unsigned id = blockIdx.x / (Rows / kRowsHere);
    const int seq = int(id % unsigned(p.b.seqs));
    id /= unsigned(p.b.seqs);
    const int tile = int(id % unsigned(p.plan.tiles)), head = int(id / unsigned(p.plan.tiles));
    const int *const split = reinterpret_cast<const int *>(kv4_split(p, Rows, id, seq));
    const int slot = uniform_load(split, 0), parts = uniform_load(split, 1);  // not written where the sequence has no such rows
    const Kv8Sequence s = uniform_sequence(p.b, seq);
    const std::int64_t row = std::int64_t(tile) * Rows + i;
    if (row >= s.n * R || parts == 0) return;  // with W > 1 this is the same for all waves
    const std::int64_t pitch = std::int64_t(Rows) * (dim + 4);
    const float *const part = p.ws + (((std::int64_t(head) * p.plan.tiles + tile) * p.plan.parts + slot + seq) * Rows + i) * (dim + 4);
    float m = -__builtin_inff(), top = 0.0f, sum = 0.0f;
    f32x4 y = {0, 0, 0, 0};
    const float *const at = part + (4 * lane < dim ? 4 * lane : 0);
    for (int x0 = wave; x0 < parts; x0 += W * kAtOnce) {
        f32x4 v[kAtOnce];
        f32x4 stand[kAtOnce];  // m, sum and largest product
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int x = x0 + W * j < parts ? x0 + W * j : x0;
            v[j] = *reinterpret_cast<const f32x4 *>(at + x * pitch);
            stand[j] = *reinterpret_cast<const f32x4 *>(part + x * pitch + dim);
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            if (x0 + W * j >= parts) continue;
            // A part that saw nothing of its row weighs nothing: its sums are zeros.
            const float to = __builtin_fmaxf(m, stand[j][0]), a = rescale(m, to), b = rescale(stand[j][0], to);
            const float largest = __builtin_fmaxf(top * a, stand[j][2] * b);
            sum = sum * a + stand[j][1] * b;
            y = y * to_unit(a, top, largest) + v[j] * to_unit(b, stand[j][2], largest);
            m = to;
            top = largest;
        }
    }
    if constexpr (W > 1) {
        if (lane == 0) sm_m[wave] = m, sm_top[wave] = top, sm_sum[wave] = sum;
        if (4 * lane < dim) *reinterpret_cast<f32x4 *>(&sm_x[wave][4 * lane]) = y;
        __syncthreads();
        if (wave != 0) return;
        for (int w = 1; w < W; ++w) m = __builtin_fmaxf(m, sm_m[w]);
        top = 0.0f;
        for (int w = 0; w < W; ++w) top = __builtin_fmaxf(top, sm_top[w] * rescale(sm_m[w], m));
        sum = 0.0f;
        y = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float a = rescale(sm_m[w], m);
            sum += sm_sum[w] * a;
            if (4 * lane < dim) y += *reinterpret_cast<const f32x4 *>(&sm_x[w][4 * lane]) * to_unit(a, sm_top[w], top);
        }
    }
    if (4 * lane >= dim) return;
    y = in_values(y / sum, top);
    const std::int64_t fresh = divide(row, R);
    const KvSeen seen{s.len - s.n, s.len, std::int64_t(p.b.table_ld) << shift, 1, p.causal, p.window};
    if (seen.beyond_new(fresh)) y = y * __builtin_nanf("");
    __builtin_memcpy(p.O + (s.row0 + fresh) * p.ldo + (std::int64_t(head) * R + row - fresh * R) * p.hso + 4 * lane, &y, sizeof(y));
}

// Prompts: the waves of a work-group take row tiles of their own; the same keys
// and values pass through the compute unit's cache for all four. A wave keeps 32
// rows, so that a code is converted once for them.
//
// 2 prompts of 1024 rows behind 4096 tokens in f16: 206 us, 577 TFLOP/s. As it
// is, a SIMD is busy issuing: of its cycles vector instructions take 62% (the
// exponentials' longer turn not counted) and matrix instructions 40%, two of three
// of those for the second part of the weights and the first. Codes converted once
// for the four waves and laid in LDS need a quarter fewer vector instructions, but
// their barriers and reads cost more than that: 233 to 246 us when the rest took
// 216, with four waves or eight and two to four a SIMD. More than 32 rows a wave were
// not tried.
template <class T, int DC, bool Full, int MT>
__global__ __launch_bounds__(64 * kAttendWaves, 2) void kv4_rows_kernel(Kv4AttendProblem p)
{
    constexpr int PD = 32 * DC, kRows = 16 * MT, kDTiles = 2 * DC, kVWords = (DC + 3) / 4;
    typedef typename T::elem elem;
    const int lane = threadIdx.x & 63, c = lane & 15, kq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int dim = Full ? PD : p.c.dim, R = p.heads_q / p.c.heads;
    const int shift = 31 - __builtin_clz(unsigned(p.c.block)), block = 1 << shift;

    unsigned id = blockIdx.x;
    // Later tiles see more tokens. Where a sequence's and head's work-groups are
    // the second ones that come to the compute units, they go the other way, so
    // that each unit gets a long one and a short one (1 prompt of 2048
    // rows of 5120 tokens: 236 us against 264, 2 of 1024 behind 4096 207 against 214).
    const unsigned tiles = unsigned(p.plan.tiles), number = id % tiles;
    const bool back = (id - number) / unsigned(p.plan.cus) & 1;
    const int tile0 = int(back ? tiles - 1 - number : number);
    id /= tiles;
    const int head = int(id % unsigned(p.c.heads));
    const unsigned seqs_at_once = gridDim.x / (unsigned(p.plan.tiles) * unsigned(p.c.heads));
    const float factor = p.scale * kLog2e;
    const std::uint8_t *const codes_k = static_cast<const std::uint8_t *>(p.c.K), *const codes_v = static_cast<const std::uint8_t *>(p.c.V);
    const std::uint16_t *const scales_k = static_cast<const std::uint16_t *>(p.c.Ks), *const scales_v = static_cast<const std::uint16_t *>(p.c.Vs);
    // Lanes past the head's components read its first ones: their queries are
    // zero, their values give components that are not stored.
    const int k_at = c * (dim / 2), v_at = 4 * kq * (dim / 2) + (Full || c * 2 * DC < dim ? c * DC : 0);

    for (unsigned seq = id / unsigned(p.c.heads); seq < unsigned(p.b.seqs); seq += seqs_at_once) {
        const Kv8Sequence s = uniform_sequence(p.b, int(seq));
        const std::int64_t all_rows = s.n * R;
        const KvSeen seen{s.len - s.n, s.len, std::int64_t(p.b.table_ld) << shift, R, p.causal, p.window};
        const int *const table = p.b.table + std::int64_t(seq) * p.b.table_ld;
        for (std::int64_t tile = tile0;; tile += p.plan.tiles) {
            const std::int64_t row0 = (tile * kAttendWaves + wave) * kRows;
            if (tile * kAttendWaves * kRows >= all_rows) break;
            if (row0 >= all_rows) continue;

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
                QueryPieces<T, DC> raw;
                raw.load(src + kq * DC * 8, [&](int i) { return Full || (kq * DC + i) * 8 < dim; });
                row_factor[t] = query_operands<T, DC>(raw, q[t]);
            }
            int first_lo, first_n, last_lo, last_n;
            seen(row0, first_lo, first_n);
            seen(row0 + kRows < all_rows ? row0 + kRows - 1 : all_rows - 1, last_lo, last_n);
            // Turns of 32 tokens: begin .. end sees some row; inner .. outer every row in full.
            // (Positions reach 2^31 - 1, so that rounding up needs the sign bit.)
            const int limit = last_lo + last_n;
            const int begin = first_lo >> 5, end = int((unsigned(limit) + 31u) >> 5);
            const int inner = int((unsigned(last_lo) + 31u) >> 5), outer = (first_lo + first_n) >> 5;

            f32x4 o[MT][kDTiles] = {};
            float m[MT], l[MT];         // what scores are relative to; sum of the weights
            float top_w[MT], unit[MT];  // largest product when the unit was made; what products are multiplied by
#pragma unroll
            for (int t = 0; t < MT; ++t) m[t] = -__builtin_inff(), l[t] = top_w[t] = 0.0f, unit[t] = power(unit_of(0.0f));

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
                        }
                    }
                    ks[x] = *reinterpret_cast<const u32x2 *>(scales_k + h[x].token + 4 * kq);
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

            // Turns from .. to; Cut: some row does not see all of a turn.
            auto turns = [&](int from, int to, auto cut_) {
#pragma clang fp contract(off)  // as for few rows
                constexpr bool Cut = decltype(cut_)::value;
                int turn = from;
                if (turn >= to) return;
                bool good[2];  // of this turn's halves
                {
                    const Half first[2] = {half_at(32 * turn), half_at(32 * turn + 16)};
                    load_keys(first);
                    load_values(first);
                    good[0] = first[0].good, good[1] = first[1].good;
                }
                for (; turn < to; ++turn) {
                    const int t0 = 32 * turn, tn = turn + 1 < to ? t0 + 32 : t0;
                    const Half next[2] = {half_at(tn), half_at(tn + 16)};
                    f32x4 acc[2][MT];
                    float g[8];
                    __builtin_amdgcn_s_setprio(1);
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
                        if (!good[x]) {
#pragma unroll
                            for (int r = 0; r < 4; ++r) g[4 * x + r] = __builtin_nanf("");
                        }
                    }
                    __builtin_amdgcn_s_setprio(0);
                    load_keys(next);
                    good[0] = next[0].good, good[1] = next[1].good;
                    // Both groups of rows go side by side, with one look at all largest scores and
                    // one at all largest products (one after the other: 211 us instead of 206).
                    Frag ph[MT], pl[MT];
                    float z[MT][8], w[MT][8], a[MT];
                    unsigned sees[MT];  // bits of the tokens that the row sees
                    bool rises = false;
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        float top = -__builtin_inff();
                        sees[t] = 0;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            z[t][e] = acc[e / 4][t][e % 4] * g[e];
                            if (Cut) {
                                const bool yes = unsigned(t0 + 16 * (e / 4) + 4 * kq + e % 4 - lo_t[t]) < unsigned(n_t[t]);
                                z[t][e] = yes ? z[t][e] : -__builtin_inff();
                                sees[t] |= yes ? 1u << e : 0u;
                            }
                            top = __builtin_fmaxf(top, z[t][e]);
                        }
                        a[t] = top;
                        rises |= top > m[t];
                    }
                    const bool risen = __ballot(rises) != 0;
                    if (__builtin_expect(risen, 0)) {
#pragma unroll
                        for (int t = 0; t < MT; ++t) {
                            const float top = column_max(a[t]), to = top > m[t] ? top + kAbove : m[t];
                            a[t] = rescale(m[t], to);
                            m[t] = to;
                            l[t] *= a[t];
                        }
                    }
                    float largest[MT];
                    rises = risen;
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        const float base = __builtin_fmaxf(m[t], -3.402823466e38f);  // finite where a row has seen nothing
                        largest[t] = 0.0f;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            float pe = __builtin_amdgcn_exp2f(z[t][e] - base);
                            // A scale that is not finite makes the whole row NaN, by w or by its parts.
                            w[t][e] = pe * scale_of(vs[e / 4], e % 4);
                            if (Cut && !(sees[t] >> e & 1)) pe = w[t][e] = 0.0f;
                            l[t] += pe;
                            largest[t] = __builtin_fmaxf(largest[t], __builtin_fabsf(w[t][e]));
                        }
                        rises |= 0.5f * largest[t] > top_w[t];
                    }
                    if (__builtin_expect(__ballot(rises) != 0, 0)) {
#pragma unroll
                        for (int t = 0; t < MT; ++t) {
                            const float by = risen ? a[t] : 1.0f, to = __builtin_fmaxf(top_w[t] * by, column_max(largest[t])), b = to_unit(by, top_w[t], to);
#pragma unroll
                            for (int j = 0; j < kDTiles; ++j) o[t][j] *= b;
                            top_w[t] = to;
                            unit[t] = power(unit_of(to));
                        }
                    }
#pragma unroll
                    for (int t = 0; t < MT; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            std::uint32_t hi, lo;
                            split2(w[t][2 * e], w[t][2 * e + 1], unit[t], hi, lo);
                            ph[t].v[e] = hi;
                            pl[t].v[e] = lo;
                        }
                    __builtin_amdgcn_s_setprio(1);
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
                    __builtin_amdgcn_s_setprio(0);
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
                    y = in_values(y, top_w[t]);
                    __builtin_memcpy(dst + x, &y, sizeof(y));
                }
            }
        }
    }
}

template <class K> hipError_t launch_kv4_grid(K kernel, const Kv4AttendProblem &p, unsigned groups, unsigned threads, hipStream_t stream)
{
    Kv4AttendProblem q = p;
    void *args[] = {&q};
    return hipLaunchKernel(reinterpret_cast<const void *>(kernel), dim3(groups), dim3(threads), args, 0, stream);
}

template <class T, int DC, bool Full, int P> hipError_t launch_kv4_few(const Kv4AttendProblem &p, hipStream_t stream)
{
    constexpr int kRows = 16 / P;
    const std::int64_t per_seq = std::int64_t(p.plan.tiles) * p.c.heads;
    if (p.plan.slots == 0) {
        std::int64_t seqs = (std::int64_t(1) << 22) / per_seq;
        seqs = seqs < 1 ? 1 : seqs < p.b.seqs ? seqs : p.b.seqs;
        return launch_kv4_grid(&kv4_few_kernel<T, DC, Full, P>, p, unsigned(per_seq * seqs), 64 * kAttendWaves, stream);
    }
    const hipError_t e = launch_kv4_grid(&kv4_few_kernel<T, DC, Full, P>, p, unsigned(per_seq * p.plan.slots), 64 * kAttendWaves, stream);
    if (e != hipSuccess) return e;
    if (p.plan.slots > 8 * p.b.seqs) return launch_kv4_grid(&kv4_join_kernel<kRows, 4>, p, unsigned(per_seq * p.b.seqs * kRows), 256, stream);
    return launch_kv4_grid(&kv4_join_kernel<kRows, 1>, p, unsigned(per_seq * p.b.seqs * (kRows / 4)), 256, stream);
}

template <class T, int DC, bool Full> hipError_t launch_kv4_shape(const Kv4AttendProblem &p, hipStream_t stream)
{
    if (p.plan.rows) {
        const std::int64_t per_seq = std::int64_t(p.plan.tiles) * p.c.heads;
        std::int64_t seqs = (std::int64_t(1) << 22) / per_seq;
        seqs = seqs < 1 ? 1 : seqs < p.b.seqs ? seqs : p.b.seqs;
        constexpr int kGroups = DC > 4 ? 1 : 2;  // of 16 rows a wave, as plan_kv4_attend has it
        return launch_kv4_grid(&kv4_rows_kernel<T, DC, Full, kGroups>, p, unsigned(per_seq * seqs), 64 * kAttendWaves, stream);
    }
    return p.plan.copies == 4   ? launch_kv4_few<T, DC, Full, 4>(p, stream)
           : p.plan.copies == 2 ? launch_kv4_few<T, DC, Full, 2>(p, stream)
                                : launch_kv4_few<T, DC, Full, 1>(p, stream);
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
