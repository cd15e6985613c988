// sgemm_w4 with f32 rows.
#include "w4.hpp"

namespace sgemm_impl {
hipError_t launch_w4_f32(const W4Problem &p, hipStream_t stream) { return launch_w4<F32>(p, stream); }
}  // namespace sgemm_impl
