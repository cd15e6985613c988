// C ABI entry points of a serving step (the 4-bit cache, rotary positions,
// page tables): host checks, device check, launch (as api.hip).
#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "gemm.hpp"
#include "sgemm.h"
#include "step.hpp"

namespace {

int status_of(hipError_t e) { return e == hipSuccess ? SGEMM_OK : SGEMM_ERR_LAUNCH; }

}  // namespace

extern "C" int sgemm_kv4_write(const sgemm_kv4_cache *cache, const sgemm_kv8_batch *batch, int dtype, const void *K,
                               int ldk, int hsk, const void *V, int ldv, int hsv, void *stream)
{
    const int rc = sgemm_kv4_check_args(cache, batch, dtype, K, ldk, hsk, V, ldv, hsv);
    if (rc != SGEMM_OK) return rc;
    if (batch->seqs == 0 || batch->rows == 0) return SGEMM_OK;
    if (sgemm_impl::kv4_write_overlaps(*cache, *batch)) return SGEMM_ERR_ALIAS;
    if (sgemm_impl::current_gfx950_cus() == 0) return SGEMM_ERR_DEVICE;
    const sgemm_impl::Kv4Problem p{*cache, *batch, const_cast<void *>(K), const_cast<void *>(V), ldk, hsk, ldv, hsv, dtype};
    return status_of(sgemm_impl::launch_kv4_write(p, static_cast<hipStream_t>(stream)));
}

extern "C" int sgemm_kv4_read(const sgemm_kv4_cache *cache, const sgemm_kv8_batch *batch, int dtype, void *K, int ldk,
                              int hsk, void *V, int ldv, int hsv, void *stream)
{
    const int rc = sgemm_kv4_check_args(cache, batch, dtype, K, ldk, hsk, V, ldv, hsv);
    if (rc != SGEMM_OK) return rc;
    if (batch->seqs == 0 || batch->rows == 0) return SGEMM_OK;
    if (sgemm_impl::kv4_read_overlaps(*cache, *batch, dtype, K, ldk, hsk, V, ldv, hsv)) return SGEMM_ERR_ALIAS;
    if (sgemm_impl::current_gfx950_cus() == 0) return SGEMM_ERR_DEVICE;
    const sgemm_impl::Kv4Problem p{*cache, *batch, K, V, ldk, hsk, ldv, hsv, dtype};
    return status_of(sgemm_impl::launch_kv4_read(p, static_cast<hipStream_t>(stream)));
}

extern "C" int sgemm_kv4_attend(const sgemm_kv4_cache *cache, const sgemm_kv8_batch *batch, int dtype, int heads_q,
                                const void *Q, int ldq, int hsq, float scale, int causal, int window, float *O, int ldo,
                                int hso, void *workspace, std::size_t workspace_bytes, void *stream)
{
    const int rc = sgemm_kv4_attend_check_args(cache, batch, dtype, heads_q, Q, ldq, hsq, scale, causal, window, O, ldo, hso,
                                               workspace, workspace_bytes);
    if (rc != SGEMM_OK) return rc;
    if (batch->seqs == 0 || batch->rows == 0) return SGEMM_OK;
    const int cus = sgemm_impl::current_gfx950_cus();
    if (cus == 0) return SGEMM_ERR_DEVICE;
    sgemm_impl::Kv4Plan plan = sgemm_impl::plan_kv4_attend(*cache, *batch, heads_q, window, cus);
    const std::size_t need = sgemm_kv4_attend_workspace_size(cache, batch, heads_q, window, cus);
    const bool usable = workspace != nullptr && reinterpret_cast<std::uintptr_t>(workspace) % 16 == 0 && workspace_bytes >= need;
    if (!usable) plan.slots = 0;
    const sgemm_impl::Kv4AttendProblem p{*cache, *batch, Q, O, static_cast<float *>(workspace), ldq, hsq, ldo, hso, heads_q,
                                         scale, causal, window, plan};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return status_of(dtype == SGEMM_F32       ? sgemm_impl::launch_kv4_attend_f32(p, s)
                     : dtype == SGEMM_LP_BF16 ? sgemm_impl::launch_kv4_attend_bf16(p, s)
                                              : sgemm_impl::launch_kv4_attend_f16(p, s));
}

extern "C" int sgemm_rope(int dtype, int otype, int rows, int dim, int rot, int interleaved, int inverse, float amplitude,
                          const int *positions, const double *freqs, const sgemm_rope_rows *first, const sgemm_rope_rows *second,
                          void *stream)
{
    const int rc = sgemm_rope_check_args(dtype, otype, rows, dim, rot, interleaved, inverse, amplitude, positions, freqs, first, second);
    if (rc != SGEMM_OK) return rc;
    if (rows == 0) return SGEMM_OK;
    const int cus = sgemm_impl::current_gfx950_cus();
    if (cus == 0) return SGEMM_ERR_DEVICE;
    const sgemm_impl::RopeProblem p{positions, freqs, {*first, second != nullptr ? *second : sgemm_rope_rows{}}, dtype, otype, rows, dim, rot,
                                    interleaved, inverse, amplitude};
    return status_of(sgemm_impl::launch_rope(p, cus, static_cast<hipStream_t>(stream)));
}

extern "C" int sgemm_kv_tables(const sgemm_kv_step *step, void *stream)
{
    const int rc = sgemm_kv_tables_check_args(step);
    if (rc != SGEMM_OK) return rc;
    if (sgemm_impl::current_gfx950_cus() == 0) return SGEMM_ERR_DEVICE;
    return status_of(sgemm_impl::launch_kv_tables(*step, static_cast<hipStream_t>(stream)));
}
