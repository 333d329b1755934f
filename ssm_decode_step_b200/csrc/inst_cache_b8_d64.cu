// Cache-step kernel instances for 8-bit codes and Dk = 64.
#include "qstate_launch_impl.cuh"

namespace qs {
QS_INSTANTIATE_CACHE(8, 64)
}  // namespace qs
