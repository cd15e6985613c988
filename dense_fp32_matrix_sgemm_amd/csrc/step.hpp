// A serving step's kernels (4-bit cache, rotary positions, page tables): their
// problems and launchers.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "lowbit.hpp"
#include "sgemm.h"
#include "step_plan.hpp"

namespace sgemm_impl {

// Writing and reading the 4-bit cache (seqs, rows > 0); strides in elements.
struct Kv4Problem {
    sgemm_kv4_cache c;
    sgemm_kv8_batch b;
    void *K, *V;
    std::int64_t ldk, hsk, ldv, hsv;
    int dtype;
    bool stream() const { return std::int64_t(b.rows) * c.heads * c.dim * 2 >= kStreamBytes; }  // 16-bit K, or V
};
hipError_t launch_kv4_write(const Kv4Problem &p, hipStream_t stream);
hipError_t launch_kv4_read(const Kv4Problem &p, hipStream_t stream);

struct Kv4AttendProblem {
    sgemm_kv4_cache c;
    sgemm_kv8_batch b;
    const void *Q;
    float *O;
    float *ws;  // plan.slots > 0
    std::int64_t ldq, hsq, ldo, hso;
    int heads_q;
    float scale;
    int causal, window;
    Kv4Plan plan;
};
hipError_t launch_kv4_attend_f32(const Kv4AttendProblem &p, hipStream_t stream);
hipError_t launch_kv4_attend_bf16(const Kv4AttendProblem &p, hipStream_t stream);
hipError_t launch_kv4_attend_f16(const Kv4AttendProblem &p, hipStream_t stream);

// Turning rows by their positions (rows > 0).
struct RopeProblem {
    const int *positions;
    const double *freqs;
    sgemm_rope_rows x[2];  // x[1].heads == 0: one operand
    int dtype, otype, rows, dim, rot, interleaved, inverse;
    float amplitude;
    bool stream() const { return std::int64_t(rows) * (x[0].heads + x[1].heads) * dim * 2 >= kStreamBytes; }  // 16-bit outputs
};
hipError_t launch_rope(const RopeProblem &p, int cus, hipStream_t stream);

hipError_t launch_kv_tables(const sgemm_kv_step &t, hipStream_t stream);

}  // namespace sgemm_impl
