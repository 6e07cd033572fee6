// host_checks.hpp -- argument checks shared by the C ABI sources (internal,
// host code only).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace fp8q {

// FP8Q_OK, or FP8Q_ERR_HIP with the error kept for fp8q_last_hip_error()
// (defined in api.cpp, which owns the thread's last error).
int hip_status(hipError_t e);

// With FP8Q_DEBUG=1: checks the segment arrays of a grouped call on the host (a
// synchronizing copy); otherwise FP8Q_OK (defined in api.cpp).
int debug_segments(int32_t groups, const int32_t* group_offsets, const int32_t* group_rows, int64_t total,
                   hipStream_t stream);

inline bool is_aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// A grid of more than 2^31 - 1 blocks is not launchable.
inline bool blocks_ok(int64_t blocks) { return blocks >= 0 && blocks <= 0x7FFFFFFFLL; }

// a * b with both >= 0, or -1 past `limit`.
inline int64_t mul_limit(int64_t a, int64_t b, int64_t limit) {
    return a == 0 || b <= limit / a ? a * b : -1;
}

}  // namespace fp8q
