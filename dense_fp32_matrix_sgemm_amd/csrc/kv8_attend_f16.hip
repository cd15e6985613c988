// sgemm_kv8_attend with f16 queries.
#include "kv8_attend.hpp"

namespace sgemm_impl {
hipError_t launch_kv8_attend_f16(const Kv8AttendProblem &p, hipStream_t stream) { return launch_attend<F16>(p, stream); }
}  // namespace sgemm_impl
