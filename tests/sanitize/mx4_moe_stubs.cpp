// Host-only stand-ins for the FP4 and MoE kernel launchers, next to
// launch_stubs.cpp: they fail as on a machine without a GPU.
#include "moe/moe.h"
#include "mx4/mx4.h"

namespace fp8q {
namespace mx4 {
hipError_t launch_quant_rows(const QuantArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_quant_cols(const QuantArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_quant_scatter(const ScatterArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_dequant(const DequantArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_gemm(const GemmArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_grouped_gemm(const GemmArgs&, hipStream_t) { return hipErrorNoDevice; }
}  // namespace mx4
namespace moe {
hipError_t launch_dispatch(const DispatchArgs&, hipStream_t) { return hipErrorNoDevice; }
// (the plan of the parts lives with the kernels; any size that grows with the
// arguments serves the checks)
int64_t balance_workspace_bytes(int64_t tokens, int64_t experts, int64_t seqs) {
    return 16 * (tokens / 64 + seqs + 1) * (experts + 1);
}
hipError_t launch_balance(const BalanceArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_balance_backward(const BalanceArgs&, hipStream_t) { return hipErrorNoDevice; }
}  // namespace moe
}  // namespace fp8q
