// sgemm_kv4_attend with float32 queries.
#include "kv4_attend.hpp"

namespace sgemm_impl {
hipError_t launch_kv4_attend_f32(const Kv4AttendProblem &p, hipStream_t stream) { return launch_kv4<F32>(p, stream); }
}  // namespace sgemm_impl
