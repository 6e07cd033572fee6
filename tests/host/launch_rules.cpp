// The kernels' launch sizes, as C functions for the CPU tests: the headers
// that the launchers themselves use.
#include "moe/moe_launch.hpp"

using namespace fp8q;

extern "C" {

int launch_fits(int64_t blocks, int threads) { return launchable({blocks, threads}); }

int64_t moe_backward_tokens() { return moe::kBackwardTokens; }
void moe_backward_shape(int64_t tokens, int64_t* blocks, int* threads) {
    const LaunchShape s = moe::backward_shape(tokens);
    *blocks = s.blocks;
    *threads = s.threads;
}

}  // extern "C"
