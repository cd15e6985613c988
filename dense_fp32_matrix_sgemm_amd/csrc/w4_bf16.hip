// sgemm_w4 with bf16 rows.
#include "w4.hpp"

namespace sgemm_impl {
hipError_t launch_w4_bf16(const W4Problem &p, hipStream_t stream) { return launch_w4<BF16>(p, stream); }
}  // namespace sgemm_impl
