// The kernels' launch sizes, as C functions for the CPU tests: the headers
// that the launchers themselves use.
#include "moe/moe_launch.hpp"
#include "mx4/mx4_launch.hpp"

using namespace fp8q;

static void put(LaunchShape s, int64_t* blocks, int* threads) {
    *blocks = s.blocks;
    *threads = s.threads;
}

extern "C" {

int launch_fits(int64_t blocks, int threads) { return launchable({blocks, threads}); }

int64_t moe_backward_tokens() { return moe::kBackwardTokens; }
void moe_backward_shape(int64_t tokens, int64_t* blocks, int* threads) {
    put(moe::backward_shape(tokens), blocks, threads);
}

void fp4_quant_rows_shape(int64_t groups, int64_t rows, int64_t cols, int64_t* blocks, int* threads) {
    put(mx4::quant_rows_shape(groups, rows, cols), blocks, threads);
}
void fp4_quant_cols_shape(int64_t groups, int64_t rows, int64_t cols, int64_t* blocks, int* threads) {
    put(mx4::quant_cols_shape(groups, rows, cols), blocks, threads);
}
void fp4_gemm_shape(int64_t m, int64_t n, int64_t kt, int64_t* blocks, int* threads) {
    put(mx4::gemm_shape(mx4::gemm_form(m, n, true), m, n, kt), blocks, threads);
}
void fp4_grouped_shape(int64_t m_total, int64_t n, int64_t kt, int64_t groups, int64_t* blocks, int* threads) {
    put(mx4::grouped_shape(mx4::grouped_form(m_total, n, groups, true), m_total, n, kt, groups), blocks, threads);
}

// kernel (0 rows, 1 tiles, 2 grouped tiles), ms and nt
static void put_form(mx4::GemmForm f, int* out) {
    out[0] = (int)f.kernel;
    out[1] = f.ms;
    out[2] = f.nt;
}
void fp4_gemm_form(int64_t m, int64_t n, int scales16, int* out) { put_form(mx4::gemm_form(m, n, scales16), out); }
void fp4_grouped_form(int64_t m_total, int64_t n, int64_t groups, int scales16, int* out) {
    put_form(mx4::grouped_form(m_total, n, groups, scales16), out);
}

}  // extern "C"
