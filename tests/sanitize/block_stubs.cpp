// Host-only stand-ins for the launchers of the gated block, the weight-only
// products and the optimizer, next to launch_stubs.cpp: they fail as on a
// machine without a GPU.
#include "adamw/adamw.h"
#include "gated/gated.h"
#include "gemv/gemv.h"

namespace fp8q {
namespace gated {
hipError_t launch_gated(const GatedArgs&, float*, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_grouped_gated(const GatedArgs&, float*, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_backward(const BackwardArgs&, hipStream_t) { return hipErrorNoDevice; }
}  // namespace gated
namespace gemv {
hipError_t launch(const Args&, hipStream_t) { return hipErrorNoDevice; }
}  // namespace gemv
namespace adamw {
hipError_t launch_step(int32_t, const fp8q_adamw_tensor*, const void* const*, const Options&, hipStream_t) {
    return hipErrorNoDevice;
}
}  // namespace adamw
}  // namespace fp8q
