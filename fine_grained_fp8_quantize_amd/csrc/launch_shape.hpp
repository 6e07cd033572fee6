// launch_shape.hpp -- how large a kernel launch may be (internal, host code
// only; it needs no HIP header, so that the shapes can be tested alone).
#pragma once

#include <stdint.h>

namespace fp8q {

// A one-dimensional launch.
struct LaunchShape {
    int64_t blocks;
    int threads;  // per block
};

// A dispatch packet holds the grid's size in work-items in 32 bits.
inline bool launchable(LaunchShape s) {
    return s.blocks >= 0 && s.blocks <= 0x7FFFFFFFLL && s.blocks * s.threads <= 0xFFFFFFFFLL;
}

}  // namespace fp8q
