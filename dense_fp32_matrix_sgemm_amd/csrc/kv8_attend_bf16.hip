// sgemm_kv8_attend with bf16 queries.
#include "kv8_attend.hpp"

namespace sgemm_impl {
hipError_t launch_kv8_attend_bf16(const Kv8AttendProblem &p, hipStream_t stream) { return launch_attend<BF16>(p, stream); }
}  // namespace sgemm_impl
