// sgemm_kv8_attend with f32 queries.
#include "kv8_attend.hpp"

namespace sgemm_impl {
hipError_t launch_kv8_attend_f32(const Kv8AttendProblem &p, hipStream_t stream) { return launch_attend<F32>(p, stream); }
}  // namespace sgemm_impl
