// sgemm_kv4_attend with f16 queries.
#include "kv4_attend.hpp"

namespace sgemm_impl {
hipError_t launch_kv4_attend_f16(const Kv4AttendProblem &p, hipStream_t stream) { return launch_kv4<F16>(p, stream); }
}  // namespace sgemm_impl
