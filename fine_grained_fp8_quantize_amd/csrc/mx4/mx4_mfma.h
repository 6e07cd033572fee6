// mx4_mfma.h -- the scaled FP4 matrix instruction with its accumulator held in
// place (internal, device code).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8q {
namespace mx4 {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));

// acc += (B tile) * (A tile)^T with the accumulator in place in AGPRs. The
// 256 accumulator registers of a 128 x 128 wave tile are all the AGPRs there
// are: left to itself, the register allocator gives results other registers
// than their inputs and copies them back and forth inside the K loop (752
// copies per 512 MFMAs). The tied operand rules that out. The compiler does
// not see a matrix instruction here, so it is up to the code that reads
// accumulators to wait first (mfma_settle).
template <int T>
__device__ __forceinline__ void mfma_in_place(v4f& acc, v4i b, v4i a, uint32_t sb, uint32_t sa) {
#define FP8Q_MFMA(lo, hi)                                                                                         \
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[" lo "," lo ",0] op_sel_hi:[" hi "," hi \
                 ",0] cbsz:4 blgp:4"                                                                              \
                 : "+a"(acc)                                                                                      \
                 : "v"(b), "v"(a), "v"(sb), "v"(sa))
    if constexpr (T == 0) FP8Q_MFMA("0", "0");
    else if constexpr (T == 1) FP8Q_MFMA("1", "0");
    else if constexpr (T == 2) FP8Q_MFMA("0", "1");
    else FP8Q_MFMA("1", "1");
#undef FP8Q_MFMA
}
// More wait states than the last MFMA's results take, before the code that
// follows. Every accumulator passes through an (empty) instruction behind the
// wait, so that nothing that reads one can be moved ahead of it.
template <int N, int M>
__device__ __forceinline__ void mfma_settle(v4f (&acc)[N][M]) {
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
        for (int i = 0; i < M; ++i) asm volatile("" : "+a"(acc[j][i]));
}

}  // namespace mx4
}  // namespace fp8q
