/*
 * sgemm.h -- C ABI of the MI355X (gfx950) FP32 matrix multiply.
 *
 * Operation ("Shared Memory Tiling for Matrix Multiplication", opening
 * definition; "Matrix Multiplication -- Naive to Tiled", section 02):
 *
 *     C[i][j] = sum_{k=0}^{K-1} A[i][k] * B[k][j],   0 <= i < M, 0 <= j < N
 *
 * A is M x K, B is K x N, C is M x N, all float32 and row-major: element
 * (r, c) of a matrix with leading dimension ld lives at ptr[r * ld + c]
 * ("Matrix Multiplication -- Naive to Tiled", section 02 indexes A[row*K+i],
 * B[i*N+col], C[row*N+col]; leading dimensions generalise the row length as
 * the BLAS call of section 07 does). C is overwritten: its old contents are
 * never read (section 07's vendor call with alpha = 1, beta = 0; every kernel
 * on the pages stores with '='). Elements of C's rows beyond column N-1 (the
 * padding up to ldc) are never touched.
 *
 * Products are formed and summed in float32 (fused multiply-add, round to
 * nearest even). The summation order is the kernel's own; the result is within
 * 1e-5 * sum_k |A[i][k]| * |B[k][j]| + 1e-6 of the exact sum, and exact when
 * every partial sum is an integer below 2^24 (small-integer inputs).
 *
 * All matrix pointers are DEVICE pointers on the calling thread's current HIP
 * device. The caller owns every buffer; the library allocates nothing per
 * call (sgemm_ex_ws works in scratch memory the caller passes), keeps no
 * pointer after returning and has no mutable global state besides a
 * per-device cache of the device's architecture, so calls from several host
 * threads are safe. The one exception is sgemm_ex_noalloc, which works in a
 * static device buffer of the library's own (see there).
 */
#ifndef SGEMM_H
#define SGEMM_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes. Every entry point returns one; none ever exits the process
 * (unlike the pages' error macro, which prints and calls exit()). */
typedef enum sgemm_status {
    SGEMM_OK = 0,
    SGEMM_ERR_DIM = -1,      /* M, N or K negative                              */
    SGEMM_ERR_LD = -2,       /* lda < max(1,K), ldb < max(1,N) or ldc < max(1,N) */
    SGEMM_ERR_NULL = -3,     /* NULL matrix pointer with a non-empty extent      */
    SGEMM_ERR_VARIANT = -4,  /* unknown variant code                             */
    SGEMM_ERR_LAUNCH = -5,   /* the HIP launch itself failed (hipGetLastError)   */
    SGEMM_ERR_DEVICE = -6,   /* no usable HIP device, or it is not gfx950        */
    SGEMM_ERR_ALIAS = -7,    /* C's extent overlaps A's or B's                   */
    SGEMM_ERR_OP = -8,       /* transpose flag not SGEMM_OP_N or SGEMM_OP_T      */
    SGEMM_ERR_DTYPE = -9,    /* 16-bit type not SGEMM_LP_BF16 or SGEMM_LP_F16    */
    SGEMM_ERR_SCRATCH = -10, /* sgemm_ex_noalloc: the product needs more scratch
                                than the library's static buffer holds          */
    SGEMM_ERR_GROUP = -11,   /* sgemm_w4*: group not a positive multiple of 32   */
    SGEMM_ERR_CACHE = -12,   /* sgemm_kv8*: block, dim or alignment of the cache
                                not one the kernels take                        */
    SGEMM_ERR_HEADS = -13,   /* sgemm_kv8_attend: query heads not a positive
                                multiple of the cache's heads                   */
    SGEMM_ERR_MASK = -14     /* sgemm_kv8_attend: causal not 0 or 1, window
                                negative, or a window without causal            */
} sgemm_status;

/* 16-bit operand types of sgemm_lp. */
typedef enum sgemm_lp_type {
    SGEMM_LP_BF16 = 1,  /* bfloat16: the upper 16 bits of an IEEE binary32     */
    SGEMM_LP_F16 = 2    /* IEEE 754 binary16                                   */
} sgemm_lp_type;

/* Element types of the entry points that take float32 operands as well as
 * 16-bit ones (sgemm_w4*, sgemm_kv8*): SGEMM_F32 or an sgemm_lp_type. */
typedef enum sgemm_type {
    SGEMM_F32 = 0  /* IEEE binary32 */
} sgemm_type;

/* Transpose flags of sgemm_ex: how an operand is stored. */
typedef enum sgemm_op {
    SGEMM_OP_N = 0,  /* as is: op(X) = X                   */
    SGEMM_OP_T = 1   /* transposed: op(X) = X^T            */
} sgemm_op;

/* Kernel variants: the ladder from the pages' naive kernel to matrix cores.
 *  NAIVE    one work-item per element of C, operands straight from global
 *           memory ("Matrix Multiplication -- Naive to Tiled", section 02).
 *  TILED    T x T tiles of A and B staged in LDS, zero-filled at the edges,
 *           two barriers per K step (same page, sections 04-05), with the
 *           tile size T chosen per shape from 8, 16 and 32 (same page,
 *           exercise 2; "Naive GEMM vs Tiled GEMM", the kernel with 32 x 32
 *           tiles). TILED_T8, TILED_T16 and TILED_T32 fix T.
 *  REGBLOCK 128 x 128 LDS tiles, an 8 x 8 block of C per work-item in
 *           registers, 128-bit global loads, double-buffered LDS (same page,
 *           section 07; "From 306 ms to 86 ms", "Register blocking"); 64 x 64
 *           (4 x 4), 32 x 32 (2 x 2) or 16 x 16 (1 x 1) tiles for products
 *           with too few 128 x 128 tiles to occupy the device
 *           (sgemm_regblock_tile).
 *  MFMA     the same tiling fed to the CDNA matrix cores with
 *           v_mfma_f32_32x32x2_f32 (FP32 in, FP32 accumulate), with the tile
 *           shape chosen per product (sgemm_mfma_tile, sgemm_mfma_shape).
 *  BEST     whichever variant is fastest for the shape (currently MFMA). */
typedef enum sgemm_variant {
    SGEMM_BEST = -1,
    SGEMM_NAIVE = 0,
    SGEMM_TILED = 1,
    SGEMM_REGBLOCK = 2,
    SGEMM_MFMA = 3,
    SGEMM_TILED_T8 = 4,
    SGEMM_TILED_T16 = 5,
    SGEMM_TILED_T32 = 6
} sgemm_variant;

/*
 * C = A * B on `stream` (a hipStream_t of the current device; NULL means the
 * null stream).
 *
 * Arguments
 *   M, N, K        sizes; each >= 0.
 *   A, lda         M x K operand, lda >= max(1, K).
 *   B, ldb         K x N operand, ldb >= max(1, N).
 *   C, ldc         M x N result, ldc >= max(1, N); overwritten.
 *   stream         queue to launch on; the call returns without waiting.
 *   variant        an sgemm_variant code.
 *
 * Behaviour
 *   - Arguments are checked on the host, in this order, before any HIP call:
 *     sizes, leading dimensions, variant, then (only if M > 0 and N > 0)
 *     NULL pointers and overlap of C with A or B.
 *   - M == 0 or N == 0: nothing to do; returns SGEMM_OK without touching the
 *     GPU (pointers may then be NULL).
 *   - K == 0: the sum is empty, so the M x N window of C is set to 0
 *     (A and B are not read and may be NULL).
 *   - Otherwise one kernel is enqueued. Errors a kernel meets while running
 *     (a fault from a bad pointer, say) are not seen here; they surface at the
 *     caller's next synchronisation, as for any asynchronous HIP launch.
 *   - C must not overlap A or B (checked: SGEMM_ERR_ALIAS).
 *
 * Returns SGEMM_OK or a negative sgemm_status.
 */
int sgemm(int M, int N, int K,
          const float *A, int lda,
          const float *B, int ldb,
          float *C, int ldc,
          void *stream, int variant);

/*
 * The general form of the vendor call on "Matrix Multiplication -- Naive to
 * Tiled", section 07 (which uses alpha = 1, beta = 0 and no transposes):
 *
 *     C = alpha * op(A) * op(B) + beta * C
 *
 * with op(A) of M x K, op(B) of K x N and C of M x N, all row-major float32
 * on `stream` (as for sgemm).
 *
 * Arguments
 *   transA         SGEMM_OP_N: A is stored M x K, lda >= max(1, K);
 *                  SGEMM_OP_T: A is stored K x M (op(A) = A^T), lda >= max(1, M).
 *   transB         SGEMM_OP_N: B is stored K x N, ldb >= max(1, N);
 *                  SGEMM_OP_T: B is stored N x K (op(B) = B^T), ldb >= max(1, K).
 *   M, N, K        sizes of the product; each >= 0.
 *   alpha, beta    scalars.
 *   C, ldc         M x N, ldc >= max(1, N); read (when beta != 0) and written.
 *   stream, variant  as for sgemm; every variant takes every transpose pair.
 *
 * Behaviour (the BLAS conventions)
 *   - Checks, in this order, before any HIP call: transpose flags, sizes,
 *     leading dimensions, variant, then (only if M > 0 and N > 0) C == NULL,
 *     and, when A and B are read, NULL A or B and overlap of C with them.
 *   - M == 0 or N == 0: returns SGEMM_OK without touching the GPU.
 *   - beta == 0: C is not read (NaN or Inf in C does not propagate).
 *   - K == 0 or alpha == 0: A and B are not read (and may be NULL, or overlap
 *     C); C becomes beta * C, and with beta == 1 the call returns SGEMM_OK
 *     without touching the GPU.
 *   - Otherwise each element is alpha * s + beta * c (one fused multiply-add
 *     of alpha and s onto the rounded beta * c; alpha * s alone when beta ==
 *     0), s being the float32 sum of section 02 formed as for sgemm; the
 *     result is within 1e-5 * (|alpha| sum_k |op(A)[i][k]| |op(B)[k][j]| +
 *     |beta c|) + 1e-6 of the exact value.
 *   - sgemm(M, N, K, A, lda, B, ldb, C, ldc, stream, v) is exactly
 *     sgemm_ex(SGEMM_OP_N, SGEMM_OP_N, M, N, K, 1, A, lda, B, ldb, 0, C, ldc,
 *     stream, v).
 *
 * Returns SGEMM_OK or a negative sgemm_status.
 */
int sgemm_ex(int transA, int transB, int M, int N, int K,
             float alpha,
             const float *A, int lda,
             const float *B, int ldb,
             float beta,
             float *C, int ldc,
             void *stream, int variant);

/*
 * The host-side argument checks of sgemm() alone, with the same codes and in
 * the same order; makes no HIP call and touches no memory. Returns SGEMM_OK
 * when sgemm() would go on to launch (or return early for an empty C).
 */
int sgemm_check_args(int M, int N, int K,
                     const float *A, int lda,
                     const float *B, int ldb,
                     const float *C, int ldc,
                     int variant);

/* The host-side argument checks of sgemm_ex() alone (same codes, same
 * order); makes no HIP call and touches no memory. */
int sgemm_ex_check_args(int transA, int transB, int M, int N, int K,
                        float alpha,
                        const float *A, int lda,
                        const float *B, int ldb,
                        float beta,
                        const float *C, int ldc,
                        int variant);

/*
 * sgemm_ex with a device workspace, so that the matrix-core variant can run
 * products whose tiles would load the compute units unevenly on a split
 * schedule. Tiles are tuned per problem as section 07 and exercise 2 of
 * "Matrix Multiplication -- Naive to Tiled" describe; splitting a tile's K
 * range over several work-groups is this library's addition to that.
 *
 * Split schedule: the product's (tile, K slab) iterations, tile after tile,
 * are dealt out in equal runs to one work-group per compute unit (two with
 * 128 x 128 tiles). A tile whose slabs all fall to one work-group is
 * computed and stored as in sgemm_ex; a tile shared by several is computed
 * in pieces whose unscaled sums go to the workspace, and a second kernel adds
 * each shared tile's pieces in K order and applies alpha and beta. The result
 * is therefore the same on every run, and within the bound sgemm_ex states
 * (its last bits may differ from sgemm_ex's, whose sums are not split).
 *
 * Arguments: those of sgemm_ex, plus
 *   workspace        16-byte aligned device memory the call may use
 *                    (contents undefined afterwards; the caller owns it);
 *                    NULL, an address that is not 16-byte aligned, or
 *   workspace_bytes  smaller than sgemm_ex_workspace_size() for this product,
 *                    makes the call exactly sgemm_ex.
 * The library decides per product whether the split schedule is faster; only
 * the matrix-core variant (and SGEMM_BEST) uses it. Calls that share a
 * workspace must be ordered on one stream: concurrent calls race on it.
 *
 * Behaviour: as sgemm_ex, with one more check after sgemm_ex's: a non-empty
 * workspace that overlaps C, or A or B when they are read, is SGEMM_ERR_ALIAS.
 * Returns SGEMM_OK or a negative sgemm_status.
 */
int sgemm_ex_ws(int transA, int transB, int M, int N, int K,
                float alpha,
                const float *A, int lda,
                const float *B, int ldb,
                float beta,
                float *C, int ldc,
                void *workspace, size_t workspace_bytes,
                void *stream, int variant);

/* The host-side argument checks of sgemm_ex_ws() alone (same codes, same
 * order); makes no HIP call and touches no memory. */
int sgemm_ex_ws_check_args(int transA, int transB, int M, int N, int K,
                           float alpha,
                           const float *A, int lda,
                           const float *B, int ldb,
                           float beta,
                           const float *C, int ldc,
                           const void *workspace, size_t workspace_bytes,
                           int variant);

/*
 * Workspace bytes sgemm_ex_ws needs to run this product on the split
 * schedule on a device with `cus` compute units (cus <= 0: 256, an MI355X),
 * or 0 when it would not split it (the whole-tile schedule is estimated to
 * be as fast, or the arguments are invalid). Pure host logic: no HIP call.
 */
size_t sgemm_ex_workspace_size(int transA, int transB, int M, int N, int K, int cus);

/*
 * sgemm_ex_ws without a workspace argument, for callers that cannot allocate
 * device memory (code under stream capture, tight serving loops, harnesses
 * that forbid hipMalloc): the split schedule's partial tiles go to a static
 * device buffer the library holds, sgemm_ex_noalloc_scratch_bytes() bytes
 * (128 MiB: the largest workspace the split schedule asks for on a 256-CU
 * MI355X) on each GPU the library runs on, from when the library's code is
 * loaded on that GPU until the process ends. The call itself allocates
 * nothing and calls no allocating routine.
 *
 * Arguments and behaviour: those of sgemm_ex (same checks, same order), and
 * the same product as sgemm_ex_ws given a large enough workspace: the same
 * plan, kernels and bits. After the checks, a product that the matrix-core
 * variant (or SGEMM_BEST) would put on the split schedule with more scratch
 * than the buffer holds returns SGEMM_ERR_SCRATCH without launching anything
 * (not on a 256-CU MI355X, where every plan fits). The first call on a device
 * looks up that device's address of the buffer (SGEMM_ERR_DEVICE if that
 * fails).
 *
 * Every call on one GPU shares that GPU's buffer, and what a call leaves in
 * it is never read by the next (each partial tile is written before it is
 * read). Calls whose kernels may run at the same time on one GPU (different
 * streams with no ordering between them) race on the buffer: order them on
 * one stream, or use sgemm_ex_ws with a workspace per stream.
 */
int sgemm_ex_noalloc(int transA, int transB, int M, int N, int K,
                     float alpha,
                     const float *A, int lda,
                     const float *B, int ldb,
                     float beta,
                     float *C, int ldc,
                     void *stream, int variant);

/* The host-side checks of sgemm_ex_noalloc() alone, for a device with `cus`
 * compute units (cus <= 0: 256): sgemm_ex's checks, then SGEMM_ERR_SCRATCH
 * where the product would need more than the static buffer. Makes no HIP
 * call and touches no memory. */
int sgemm_ex_noalloc_check_args(int transA, int transB, int M, int N, int K,
                                float alpha,
                                const float *A, int lda,
                                const float *B, int ldb,
                                float beta,
                                const float *C, int ldc,
                                int variant, int cus);

/* Bytes of the static scratch buffer sgemm_ex_noalloc works in. */
size_t sgemm_ex_noalloc_scratch_bytes(void);

/*
 * The reduced-precision workload: the tensor-core variant "Matrix
 * Multiplication -- Naive to Tiled", section 07 names (16-bit inputs, FP32
 * accumulation), in the general form of sgemm_ex:
 *
 *     C = alpha * op(A) * op(B) + beta * C
 *
 * with A and B holding 16-bit encodings of type `dtype` (SGEMM_LP_BF16 or
 * SGEMM_LP_F16) and C float32. Every product of two 16-bit values is exact in
 * float32, and the products are summed in float32 on the matrix cores
 * (v_mfma_f32_32x32x16_bf16 / _f16), in an order of the kernel's own.
 *
 * Arguments are those of sgemm_ex with A and B typed `const void *` (16-bit
 * elements; leading dimensions in elements; any 2-byte alignment), and no
 * variant: the matrix-core kernel always runs (a one-work-item-per-element
 * kernel takes products whose row-contiguous operand is under 8 wide).
 *
 * Behaviour: as sgemm_ex (the same checks in the same order, with the type
 * first: SGEMM_ERR_DTYPE; the same BLAS read rules; C must not overlap A or B
 * when they are read). Returns SGEMM_OK or a negative sgemm_status.
 */
int sgemm_lp(int dtype, int transA, int transB, int M, int N, int K,
             float alpha,
             const void *A, int lda,
             const void *B, int ldb,
             float beta,
             float *C, int ldc,
             void *stream);

/* The host-side argument checks of sgemm_lp() alone (same codes, same
 * order); makes no HIP call and touches no memory. */
int sgemm_lp_check_args(int dtype, int transA, int transB, int M, int N, int K,
                        float alpha,
                        const void *A, int lda,
                        const void *B, int ldb,
                        float beta,
                        const float *C, int ldc);

/*
 * ---- Products whose stored operand is held in few bits ----
 *
 * sgemm_w4 multiplies by a matrix held in 4 bits, sgemm_kv8_attend attends
 * over keys and values held in 8; the other entry points make those operands
 * and read them back. As everywhere in this library products are summed in
 * float32 and results are float32; codes enter the matrix cores as the whole
 * numbers (W4) or floats (KV8) they stand for, which the 16-bit types hold
 * exactly, and scales multiply the float32 sums. float32 operands enter as
 * three bf16 parts that add up to them exactly (below 2^-110 their last bits
 * may be lost).
 *
 * The W4 form of an N x K matrix W, in groups of `group` k of a row (a
 * positive multiple of 32; the last group of a row may be shorter; K at most
 * 2^30):
 *
 *     W[n][k] = S[n][k / group] * (q[n][k] - z)
 *
 *   codes   q[n][k] in 0..15: byte W[n * ldw + k / 2], the low half for even
 *           k, the high half for odd k (unused at the end of an odd K);
 *   scales  S[n * lds + k / group], of type stype (SGEMM_F32, SGEMM_LP_BF16
 *           or SGEMM_LP_F16);
 *   zeros   z = Z[n * ldz + k / group], one byte of 0..15 (higher bits are
 *           ignored); with Z == NULL every z is 8.
 * Rows may start at any byte (codes, zeros) or element (scales).
 */

/*
 * C = alpha * A * W^T + beta * C with A of M x K (dtype SGEMM_F32,
 * SGEMM_LP_BF16 or SGEMM_LP_F16, row-major, lda >= max(1, K) elements), W of
 * N x K in the W4 form and C of M x N float32.
 *
 * Behaviour: as sgemm_lp. Checks, in this order, before any HIP call: types
 * (SGEMM_ERR_DTYPE), sizes, group, leading dimensions (ldw >= max(1,
 * ceil(K / 2)); lds and, with zeros, ldz >= max(1, ceil(K / group)); ldc >=
 * max(1, N)), then (only if M > 0 and N > 0) NULL C and, when A and W are
 * read (K > 0 and alpha != 0), NULL A, W or S and overlap of C with A, W, S
 * or Z. beta == 0 never reads C. One kernel is enqueued (several for more
 * columns or rows than one launch takes, from 131072 on, or K over 65536);
 * nothing is allocated. The result is the same on every run, and within
 *     (1e-5 + 2^-29 min(K, 65536) + 2^-40 K) *
 *         (|alpha| sum_k |A[m][k]| |W[n][k]| + |beta c|) + 1e-6
 * of the exact value: a float32 sum of up to min(K, 65536) / 32 groups, each
 * rounded by at most 2^-24, from 65536 k on several such sums added up in C,
 * and the sums inside a group, of the waves, and with beta c. A group's
 * products with the whole numbers q - z are summed before its scale
 * multiplies them, so that sum |A[m][k] (q - z)| over a group has to stay
 * within float32's range, and float32 elements of A below 2^-110 may lose
 * bits.
 */
int sgemm_w4(int dtype, int stype, int M, int N, int K, int group,
             float alpha,
             const void *A, int lda,
             const unsigned char *W, int ldw,
             const void *S, int lds,
             const unsigned char *Z, int ldz,
             float beta,
             float *C, int ldc,
             void *stream);

/* The host-side argument checks of sgemm_w4() alone. */
int sgemm_w4_check_args(int dtype, int stype, int M, int N, int K, int group,
                        float alpha,
                        const void *A, int lda,
                        const unsigned char *W, int ldw,
                        const void *S, int lds,
                        const unsigned char *Z, int ldz,
                        float beta,
                        const float *C, int ldc);

/*
 * How sgemm_w4 lays a product out over a device with `cus` compute units (cus
 * <= 0: 256), in shape[0..4]: the rows and columns of C that a work-group
 * takes (16 rows: the kernel for few rows), its waves along N and along K, and
 * for few rows the number of runs of K whose A it holds in LDS one after the
 * other (0: A goes straight to registers; 1 for the larger tiles). Pure host
 * logic. Returns SGEMM_OK, SGEMM_ERR_DTYPE, SGEMM_ERR_DIM or SGEMM_ERR_NULL
 * (shape NULL).
 */
int sgemm_w4_shape(int dtype, int M, int N, int K, int cus, int *shape);

/*
 * Quantises the N x K matrix B (dtype, row-major, ldb >= max(1, K)) to the W4
 * form. For each group of a row, with rounding to nearest, ties to even:
 *   without zeros (Z == NULL)  s = max |b| / 7, q = 8 + round(b / s) in 0..15;
 *   with zeros                 lo = min(0, b), hi = max(0, b), s = (hi - lo) /
 *                              15, z = round(-lo / s) in 0..15,
 *                              q = z + round(b / s) in 0..15.
 * hi - lo and the quotient that gives s are rounded to float32 and s then to
 * stype; the other quotients are by that stored s and rounded once. s == 0
 * gives codes (and z) of 8. An s that overflows is infinite: its quotients are
 * 0, and what is read back or multiplied is NaN. A group that holds a value that is not finite
 * gets the scale NaN and codes of 8, so that products with it show it.
 *
 * Checks: types, sizes, group, leading dimensions, then (N > 0 and K > 0)
 * NULL B, W or S and overlap of W, S or Z with B or one another.
 */
int sgemm_w4_quantize(int dtype, int stype, int N, int K, int group,
                      const void *B, int ldb,
                      unsigned char *W, int ldw,
                      void *S, int lds,
                      unsigned char *Z, int ldz,
                      void *stream);

/* Reads an N x K matrix in the W4 form back into B (dtype, row-major, ldb >=
 * max(1, K)): S * (q - z) in float32, rounded to dtype. The same checks. */
int sgemm_w4_dequantize(int dtype, int stype, int N, int K, int group,
                        const unsigned char *W, int ldw,
                        const void *S, int lds,
                        const unsigned char *Z, int ldz,
                        void *B, int ldb,
                        void *stream);

/* The host-side argument checks of sgemm_w4_quantize() and
 * sgemm_w4_dequantize() alone. */
int sgemm_w4_pack_check_args(int dtype, int stype, int N, int K, int group,
                             const void *B, int ldb,
                             const unsigned char *W, int ldw,
                             const void *S, int lds,
                             const unsigned char *Z, int ldz);

/*
 * A cache of keys and values in 8-bit floats (e4m3: 1 sign, 4 exponent and 3
 * fraction bits, bias 7, largest value 448, no infinities, NaN 0x7F / 0xFF),
 * in pages of `block` tokens, with one float32 scale for each page and head:
 * the value at token t, component d is code[page][head][t][d] *
 * scale[page][head].
 */
typedef struct sgemm_kv8_cache {
    void *K, *V;     /* pages x heads x block x dim codes, 16-byte aligned      */
    float *Ks, *Vs;  /* pages x heads scales                                    */
    int pages;       /* >= 1                                                    */
    int heads;       /* 1 to 65536                                              */
    int block;       /* tokens of a page: a power of two from 16 to 1024        */
    int dim;         /* components of a head: a multiple of 16 from 16 to 256   */
} sgemm_kv8_cache;

/*
 * The sequences of one call. Sequence b holds lens[b] tokens, of which this
 * call's operand (new keys and values, queries, or a copy) covers the last
 * starts[b + 1] - starts[b]: its rows starts[b] .. starts[b + 1] - 1, in
 * order. Token t of sequence b lives at place t % block of page
 * table[b * table_ld + t / block].
 *
 * table, lens and starts are DEVICE arrays, read by the kernels alone: what
 * they hold is not seen by the host's checks. The kernels treat it so:
 * lens[b] < 0 is 0; starts are cut to 0 .. rows and a falling pair covers no
 * rows; rows at positions before token 0 have no token; a page outside 0 ..
 * pages - 1, or a token behind the table's last column, is never read or
 * written. Rows of the operand before starts[0] or from starts[seqs] on are
 * left as they were. Where starts fall and rise again, a row that two
 * sequences cover takes part in both; as an output it holds either's result,
 * element by element.
 */
typedef struct sgemm_kv8_batch {
    const int *table;   /* seqs x table_ld page numbers                         */
    const int *lens;    /* seqs                                                 */
    const int *starts;  /* seqs + 1                                             */
    int seqs;
    int table_ld;       /* columns of table, >= 0                               */
    int rows;           /* rows of the operand                                  */
    int max_new;        /* how many rows of one sequence the launch is laid out
                           for; more than that is right as well, but slower     */
} sgemm_kv8_batch;

/*
 * Quantises the last rows of each sequence into its pages. K and V are rows x
 * heads x dim (dtype; component d of head h of row r at r * ld + h * hs + d,
 * in elements). For each page that receives rows, head, and K and V apart:
 *   need  = the smallest power of two s >= 2^-126 with max |x| / s <= 448
 *           over the finite new values (0 if they are all 0);
 *   scale = need if the page holds none of the sequence's earlier tokens,
 *           else the larger of need and the page's scale;
 *   code  = x / scale rounded to e4m3, ties to even (NaN for a value that is
 *           not finite); when the scale rises, the earlier tokens' codes are
 *           rounded to the new one.
 * With powers of two that last rounding changes only values that fall among
 * e4m3's subnormals. (A page's scale that the caller set to something else is
 * used as it is; x / scale, and old scale / new scale times an earlier code,
 * are then rounded to float32 before they are to e4m3.) A page that receives rows must belong to one sequence
 * and appear once in its row of the table: two writers leave codes and scale
 * of that page undefined (nothing else).
 *
 * Checks, in this order: dtype, sizes (pages, heads, seqs, table_ld, rows,
 * max_new), cache (block, dim, alignment), strides (elements must not share
 * places: heads inside a row, hs >= dim and ld >= (heads - 1) * hs + dim, or
 * rows inside a head, ld >= dim and hs >= (rows - 1) * ld + dim), then (seqs
 * > 0 and rows > 0) NULL pointers and overlap of the operand with the cache;
 * sgemm_kv8_write() alone also refuses a cache whose arrays overlap one another
 * or the batch's (keys that are the values as well may be read and attended
 * over, but would have two writers). One kernel is enqueued.
 */
int sgemm_kv8_write(const sgemm_kv8_cache *cache, const sgemm_kv8_batch *batch, int dtype,
                    const void *K, int ldk, int hsk,
                    const void *V, int ldv, int hsv,
                    void *stream);

/* The last rows of each sequence read back: code * scale in float32, rounded
 * to dtype, into K and V (rows x heads x dim, strides as above). A row whose
 * page is not one of the cache's reads NaN; a row before token 0 is left as
 * it was. The same checks; outputs that overlap each other or the batch's
 * arrays are refused as well. */
int sgemm_kv8_read(const sgemm_kv8_cache *cache, const sgemm_kv8_batch *batch, int dtype,
                   void *K, int ldk, int hsk,
                   void *V, int ldv, int hsv,
                   void *stream);

/* The host-side argument checks that sgemm_kv8_write() and sgemm_kv8_read()
 * share. */
int sgemm_kv8_check_args(const sgemm_kv8_cache *cache, const sgemm_kv8_batch *batch, int dtype,
                         const void *K, int ldk, int hsk,
                         const void *V, int ldv, int hsv);

/*
 * Softmax attention over the cache:
 *
 *     O[r][h] = sum_t p_t V_t,   p = softmax over t of scale * <Q[r][h], K_t>
 *
 * for query heads h = 0 .. heads_q - 1, a multiple of the cache's heads;
 * query head h reads the cache's head h / (heads_q / heads). Row r = starts[b]
 * + i of sequence b stands at position p = lens[b] - n + i, n being the
 * sequence's rows. It sees
 *   causal == 0              tokens 0 .. lens[b] - 1;
 *   causal == 1, window == 0 tokens 0 .. p;
 *   causal == 1, window > 0  tokens p - window + 1 .. p.
 * A row that sees no token gets zeros; one that sees a token on a page that
 * is not the cache's gets NaN, and so does one whose scores are all minus
 * infinity, or one of them plus infinity or NaN. Tokens a row does not see do
 * not reach it, not even as NaN.
 *
 * Scores are <Q, code> in float32 times scale * log2(e) * K's scale, and values
 * are multiplied by p * V's scale in three bf16 parts: <Q, code> and scale *
 * log2(e) * K's scale have to stay within float32's normal numbers, and weights
 * below 2^-110 may lose their last bits.
 *
 * Q is rows x heads_q x dim (dtype), O the same in float32 (strides as for
 * sgemm_kv8_write). Sequences too few to fill the device are split along
 * their tokens if `workspace` (device memory, 16-byte aligned) has at least
 * sgemm_kv8_attend_workspace_size() bytes; else they are not. Split or not,
 * the result is the same on every run; the two differ in their last bits.
 * Calls that share a workspace must be ordered on one stream.
 *
 * Checks, in this order: dtype, sizes, cache, heads (SGEMM_ERR_HEADS), mask
 * (SGEMM_ERR_MASK), strides, then (seqs > 0 and rows > 0) NULL pointers and
 * overlap of O with Q, the cache or the workspace. One or two kernels are
 * enqueued.
 */
int sgemm_kv8_attend(const sgemm_kv8_cache *cache, const sgemm_kv8_batch *batch, int dtype, int heads_q,
                     const void *Q, int ldq, int hsq,
                     float scale, int causal, int window,
                     float *O, int ldo, int hso,
                     void *workspace, size_t workspace_bytes,
                     void *stream);

/* The host-side argument checks of sgemm_kv8_attend() alone. */
int sgemm_kv8_attend_check_args(const sgemm_kv8_cache *cache, const sgemm_kv8_batch *batch, int dtype, int heads_q,
                                const void *Q, int ldq, int hsq,
                                float scale, int causal, int window,
                                const float *O, int ldo, int hso,
                                const void *workspace, size_t workspace_bytes);

/* Workspace bytes with which sgemm_kv8_attend splits this call's sequences on
 * a device with `cus` compute units (cus <= 0: 256), or 0 when it would not
 * split them (or the sizes are invalid). Pure host logic; reads no array. */
size_t sgemm_kv8_attend_workspace_size(const sgemm_kv8_cache *cache, const sgemm_kv8_batch *batch, int heads_q,
                                       int window, int cus);

/*
 * How sgemm_kv8_attend lays this call out on a device with `cus` compute units
 * (cus <= 0: 256), in shape[0..3]: the rows (new rows times query heads of a
 * cache head) of a wave's tile, the row tiles of a work-group (4: its waves
 * take tiles of their own; 1: they share one tile's tokens), the work-groups
 * along the rows of a sequence and head, and those that share one row tile's
 * tokens (given the workspace). Pure host logic; reads no array. Returns
 * SGEMM_OK, the cache's and batch's SGEMM_ERR_NULL, SGEMM_ERR_DIM or
 * SGEMM_ERR_CACHE, SGEMM_ERR_HEADS, SGEMM_ERR_MASK (window negative) or
 * SGEMM_ERR_NULL (shape NULL).
 */
int sgemm_kv8_attend_shape(const sgemm_kv8_cache *cache, const sgemm_kv8_batch *batch, int heads_q, int window, int cus,
                           int *shape);

/* Static English text for a status code ("unknown status" otherwise). */
const char *sgemm_status_string(int status);

/* Static name of a variant code ("naive", "tiled", "regblock", "mfma",
 * "best"), or NULL for an unknown code. */
const char *sgemm_variant_name(int variant);

/* The concrete variant SGEMM_BEST resolves to for an M x N x K product. */
int sgemm_best_variant(int M, int N, int K);

/*
 * Edge of the square tile (128, 64, 32 or 16) the REGBLOCK variant uses for an
 * M x N product on a device with `cus` compute units (cus <= 0: 256, an
 * MI355X): the pages' 128 x 128 tile ("From 306 ms to 86 ms", "Register
 * blocking") where C holds enough of them to occupy the compute units, else
 * a smaller one, tuned per problem as section 07 of "Matrix Multiplication --
 * Naive to Tiled" describes. Pure host logic: no HIP call. Returns the edge,
 * or SGEMM_ERR_DIM when M or N is negative.
 */
int sgemm_regblock_tile(int M, int N, int cus);

/*
 * The interior tile (BM x BN) the MFMA variant uses for an M x N x K product
 * on a device with `cus` compute units (cus <= 0: 256, an MI355X); tiles are
 * tuned per problem as section 07 and exercise 2 of "Matrix Multiplication --
 * Naive to Tiled" describe. The choice estimates each shape's launch time
 * from how its work-groups fall into rounds over the compute units and the
 * throughput measured for that shape, and takes the fastest; K counts only
 * for the 64 x 64 tile whose K range is split over its waves (taken for a K
 * that is not a multiple of 32 only with one tile per compute unit). Pure
 * host logic: no HIP call. Returns SGEMM_OK, SGEMM_ERR_DIM (M, N or K
 * negative) or SGEMM_ERR_NULL (BM or BN NULL).
 */
int sgemm_mfma_tile(int M, int N, int K, int cus, int *BM, int *BN);

/*
 * The whole kernel shape behind sgemm_mfma_tile's choice, in shape[0..5]:
 * BM, BN, BK (slab depth; for the split tile below, the k per chunk), the
 * waves per work-group along M and N, and the number of wave sets that
 * split the K range between them: 1; 2 for the 64 x 64 and 32 x 32 tiles
 * whose two sets share each slab, which put two waves on each SIMD where one
 * tile per compute unit would leave one; 4 for the 64 x 64 tile whose four
 * waves each hold the whole tile over a quarter of K's chunks (1 x 1 waves
 * per set). Pure host logic. Returns SGEMM_OK, SGEMM_ERR_DIM or
 * SGEMM_ERR_NULL (shape NULL).
 */
int sgemm_mfma_shape(int M, int N, int K, int cus, int *shape);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_H */
