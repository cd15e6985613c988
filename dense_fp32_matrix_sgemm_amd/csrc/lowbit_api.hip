// C ABI entry points of the products whose stored operand is held in few
// bits: host checks, device check, launch (as api.hip).
#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "gemm.hpp"
#include "lowbit.hpp"
#include "sgemm.h"

namespace {

int status_of(hipError_t e) { return e == hipSuccess ? SGEMM_OK : SGEMM_ERR_LAUNCH; }

}  // namespace

extern "C" int sgemm_w4(int dtype, int stype, int M, int N, int K, int group, float alpha, const void *A, int lda,
                        const unsigned char *W, int ldw, const void *S, int lds, const unsigned char *Z, int ldz,
                        float beta, float *C, int ldc, void *stream)
{
    const int rc = sgemm_w4_check_args(dtype, stype, M, N, K, group, alpha, A, lda, W, ldw, S, lds, Z, ldz, beta, C, ldc);
    if (rc != SGEMM_OK) return rc;
    if (M == 0 || N == 0) return SGEMM_OK;
    const bool product = K > 0 && alpha != 0.0f;
    if (!product && beta == 1.0f) return SGEMM_OK;
    const int cus = sgemm_impl::current_gfx950_cus();
    if (cus == 0) return SGEMM_ERR_DEVICE;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (!product) {
        const sgemm_impl::Problem p{nullptr, nullptr, C, 1, 1, ldc, M, N, K, cus, false, false, alpha, beta,
                                    sgemm_impl::MfmaTile::Big};
        return status_of(sgemm_impl::launch_scale(p, s));
    }
    const sgemm_impl::W4Problem p{A, W, S, Z, C, lda, ldw, lds, ldz, ldc, M, N, K, group, stype, cus, alpha, beta};
    return status_of(dtype == SGEMM_F32       ? sgemm_impl::launch_w4_f32(p, s)
                     : dtype == SGEMM_LP_BF16 ? sgemm_impl::launch_w4_bf16(p, s)
                                              : sgemm_impl::launch_w4_f16(p, s));
}

extern "C" int sgemm_w4_quantize(int dtype, int stype, int N, int K, int group, const void *B, int ldb,
                                 unsigned char *W, int ldw, void *S, int lds, unsigned char *Z, int ldz, void *stream)
{
    const int rc = sgemm_w4_pack_check_args(dtype, stype, N, K, group, B, ldb, W, ldw, S, lds, Z, ldz);
    if (rc != SGEMM_OK) return rc;
    if (N == 0 || K == 0) return SGEMM_OK;
    if (sgemm_impl::current_gfx950_cus() == 0) return SGEMM_ERR_DEVICE;
    const sgemm_impl::W4PackProblem p{const_cast<void *>(B), W, S, Z, ldb, ldw, lds, ldz, N, K, group, dtype, stype};
    return status_of(sgemm_impl::launch_w4_quantize(p, static_cast<hipStream_t>(stream)));
}

extern "C" int sgemm_w4_dequantize(int dtype, int stype, int N, int K, int group, const unsigned char *W, int ldw,
                                   const void *S, int lds, const unsigned char *Z, int ldz, void *B, int ldb,
                                   void *stream)
{
    const int rc = sgemm_w4_pack_check_args(dtype, stype, N, K, group, B, ldb, W, ldw, S, lds, Z, ldz);
    if (rc != SGEMM_OK) return rc;
    if (N == 0 || K == 0) return SGEMM_OK;
    if (sgemm_impl::current_gfx950_cus() == 0) return SGEMM_ERR_DEVICE;
    const sgemm_impl::W4PackProblem p{B, const_cast<unsigned char *>(W), const_cast<void *>(S), const_cast<unsigned char *>(Z),
                                      ldb, ldw, lds, ldz, N, K, group, dtype, stype};
    return status_of(sgemm_impl::launch_w4_dequantize(p, static_cast<hipStream_t>(stream)));
}

extern "C" int sgemm_kv8_write(const sgemm_kv8_cache *cache, const sgemm_kv8_batch *batch, int dtype, const void *K,
                               int ldk, int hsk, const void *V, int ldv, int hsv, void *stream)
{
    const int rc = sgemm_kv8_check_args(cache, batch, dtype, K, ldk, hsk, V, ldv, hsv);
    if (rc != SGEMM_OK) return rc;
    if (batch->seqs == 0 || batch->rows == 0) return SGEMM_OK;
    if (sgemm_impl::kv8_write_overlaps(*cache, *batch)) return SGEMM_ERR_ALIAS;
    if (sgemm_impl::current_gfx950_cus() == 0) return SGEMM_ERR_DEVICE;
    const sgemm_impl::Kv8Problem p{*cache, *batch, const_cast<void *>(K), const_cast<void *>(V), ldk, hsk, ldv, hsv, dtype};
    return status_of(sgemm_impl::launch_kv8_write(p, static_cast<hipStream_t>(stream)));
}

extern "C" int sgemm_kv8_read(const sgemm_kv8_cache *cache, const sgemm_kv8_batch *batch, int dtype, void *K, int ldk,
                              int hsk, void *V, int ldv, int hsv, void *stream)
{
    const int rc = sgemm_kv8_check_args(cache, batch, dtype, K, ldk, hsk, V, ldv, hsv);
    if (rc != SGEMM_OK) return rc;
    if (batch->seqs == 0 || batch->rows == 0) return SGEMM_OK;
    if (sgemm_impl::kv8_read_overlaps(*cache, *batch, dtype, K, ldk, hsk, V, ldv, hsv)) return SGEMM_ERR_ALIAS;
    if (sgemm_impl::current_gfx950_cus() == 0) return SGEMM_ERR_DEVICE;
    const sgemm_impl::Kv8Problem p{*cache, *batch, K, V, ldk, hsk, ldv, hsv, dtype};
    return status_of(sgemm_impl::launch_kv8_read(p, static_cast<hipStream_t>(stream)));
}

extern "C" int sgemm_kv8_attend(const sgemm_kv8_cache *cache, const sgemm_kv8_batch *batch, int dtype, int heads_q,
                                const void *Q, int ldq, int hsq, float scale, int causal, int window, float *O, int ldo,
                                int hso, void *workspace, std::size_t workspace_bytes, void *stream)
{
    const int rc = sgemm_kv8_attend_check_args(cache, batch, dtype, heads_q, Q, ldq, hsq, scale, causal, window, O, ldo, hso,
                                               workspace, workspace_bytes);
    if (rc != SGEMM_OK) return rc;
    if (batch->seqs == 0 || batch->rows == 0) return SGEMM_OK;
    const int cus = sgemm_impl::current_gfx950_cus();
    if (cus == 0) return SGEMM_ERR_DEVICE;
    sgemm_impl::Kv8Plan plan = sgemm_impl::plan_kv8_attend(*cache, *batch, heads_q, window, cus);
    const std::size_t need = sgemm_kv8_attend_workspace_size(cache, batch, heads_q, window, cus);
    const bool usable = workspace != nullptr && reinterpret_cast<std::uintptr_t>(workspace) % 16 == 0 && workspace_bytes >= need;
    if (!usable) plan.splits = 1;
    const sgemm_impl::Kv8AttendProblem p{*cache, *batch, Q, O, static_cast<float *>(workspace), ldq, hsq, ldo, hso, heads_q,
                                         scale, causal, window, plan};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return status_of(dtype == SGEMM_F32       ? sgemm_impl::launch_kv8_attend_f32(p, s)
                     : dtype == SGEMM_LP_BF16 ? sgemm_impl::launch_kv8_attend_bf16(p, s)
                                              : sgemm_impl::launch_kv8_attend_f16(p, s));
}
