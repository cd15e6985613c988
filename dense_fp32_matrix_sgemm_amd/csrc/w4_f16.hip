// sgemm_w4 with f16 rows.
#include "w4.hpp"

namespace sgemm_impl {
hipError_t launch_w4_f16(const W4Problem &p, hipStream_t stream) { return launch_w4<F16>(p, stream); }
}  // namespace sgemm_impl
