// adamw.hip -- AdamW over many tensors for gfx950.
//
// The step is a stream: with FP32 parameters, bf16 gradients and a bf16 copy
// it reads and writes 28 bytes an element with 32-bit states, 16.1 with 8-bit
// ones, and HBM bounds it: 64M elements 305 us, 5.9 TB/s, and 128M in 8 bits 373
// us, 5.5 TB/s (a copy of 1 GiB: 5.1). A launch takes up to 64 tensors (56 with
// 8-bit states), whose table is a kernel argument: it is captured with the
// launch, and nothing has to be copied to the device first. A workgroup takes
// 1024 elements of one of them, a thread four consecutive ones, so that every
// load and store of a wave is contiguous. (Four times the elements per thread
// were no faster where there are many, 64M: 311 and 306 us, and their code takes
// longer to fetch and run where there are few, 56 tensors of 20011: 10.7 and 7.9
// us, with 8-bit states 13.7 and 7.5.)
#include "adamw/adamw.h"

#include <hip/hip_runtime.h>

#include <algorithm>

#include "fp8q_device.h"
#include "launch_shape.hpp"

// The arithmetic is that of the formula, one rounding per operation: results
// do not depend on which multiplications the compiler could join with which
// additions.
#pragma clang fp contract(off)

namespace fp8q {
namespace adamw {
namespace {

// beta^t by squaring, the same on host and device.
__host__ __device__ inline double int_pow(double x, int64_t t) {
    double y = 1.0;
    for (; t > 0; t >>= 1) {
        if (t & 1) y *= x;
        x *= x;
    }
    return y;
}

// What the step's options come to, rounded once.
struct Factors {
    float decay;      // 1 - lr * weight_decay
    float step_size;  // lr / (1 - beta1^t)
    float root;       // 1 / sqrt(1 - beta2^t)
};
__host__ __device__ inline Factors factors(double lr, double weight_decay, double beta1, double beta2, int64_t t) {
    Factors f;
    f.decay = (float)(1.0 - lr * weight_decay);
    f.step_size = (float)(lr / (1.0 - int_pow(beta1, t)));
    f.root = (float)(1.0 / sqrt(1.0 - int_pow(beta2, t)));
    return f;
}

constexpr int kVec = 4;                                // consecutive elements of a thread
constexpr int kChunk = kThreads * kVec;                // elements of a workgroup
constexpr int kBlock = 128;                            // elements that share a scale
static_assert(kBlock == 32 * kVec, "a block is half a wave");
constexpr int64_t kMostBlocks = FP8Q_ADAMW_MAX_NUMEL / kChunk;  // of one tensor
static_assert(FP8Q_ADAMW_MAX_NUMEL % kChunk == 0 && kMostBlocks * kThreads <= 0xFFFFFFFFLL &&
                  (kMostBlocks + 1) * kThreads > 0xFFFFFFFFLL,
              "the largest tensor is the largest launch");

struct Entry {
    void* param;
    const void* grad;
    void* exp_avg;
    void* exp_avg_sq;
    uint16_t* copy;
    int64_t numel;
};
struct Scales {
    float* exp_avg;
    float* exp_avg_sq;
};

// Tensors of a launch: as many as fit 4 KB of kernel arguments, and one lane
// each for the search of a workgroup's.
template <bool BITS8>
struct Table {
    static constexpr int kMost = BITS8 ? 56 : 64;
    Entry t[kMost];
    Scales s[BITS8 ? kMost : 1];
    int32_t first[kMost];  // first workgroup of each tensor
    uint64_t vec;          // bit i: the arrays of tensor i can be accessed four elements at a time
    int32_t place;         // place of t[0] in the call
    int32_t count;
};

struct Step {
    double lr, beta1, beta2, weight_decay;
    const float* lr_dev;
    const int64_t* step_dev;
    const float* grad_scale;
    int64_t step;
    Factors f;                    // where neither lr_dev nor step_dev is given
    float b1, c1, b2, c2, eps;    // beta1, 1 - beta1, beta2, 1 - beta2
    uint32_t seed_lo, seed_hi;
};
static_assert(sizeof(Table<true>) + sizeof(Step) <= 4096 && sizeof(Table<false>) + sizeof(Step) <= 4096,
              "kernel arguments");

// A 32-bit mixing step (odd multipliers: the golden ratio and the root of two).
__device__ __forceinline__ uint32_t mix(uint32_t x) {
    x = (x ^ (x >> 16)) * 0x9E3779B9u;
    x = (x ^ (x >> 15)) * 0x6A09E667u;
    return x ^ (x >> 16);
}

// The magnitude code of y in [0, 448] (a NaN counts as 448), rounded up where
// the 16 random bits pass what is cut off. Normal codes: the bits of y, of which
// the last 20 are cut; below 2^-6: multiples of 2^-9, cut off in units of 2^-29.
__device__ __forceinline__ uint32_t stochastic_e4m3(float y, uint32_t bits16) {
    y = __builtin_fminf(y, kE4M3Max);
    const bool normal = y >= 0x1p-6f;
    const uint32_t fixed = normal ? __float_as_uint(y) : (uint32_t)(y * 0x1p29f);
    const uint32_t code = ((fixed + (bits16 << 4)) >> 20) - (normal ? 120u << 3 : 0u);
    return code < 126u ? code : 126u;  // (448 itself has no code above)
}

__device__ __forceinline__ float4 decode4(uint32_t codes) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, true);
    return make_float4(lo[0], lo[1], hi[0], hi[1]);
}

// How a chunk is accessed: four elements at a time where all four exist, with
// no look at the end in chunks that lie before it; or one at a time, at any
// address.
enum class Access { kWhole, kTail, kSingle };

// Four elements of a tensor, from `at` on, of which `left` exist.
template <class T>
struct Four {
    T x[4];
};
template <class T, Access A>
__device__ __forceinline__ Four<T> load4(const T* p, int64_t at, int left) {
    Four<T> v = {};
    if (A == Access::kWhole || (A == Access::kTail && left == 4)) {
        typedef T vec_t __attribute__((ext_vector_type(4)));
        const vec_t w = __builtin_nontemporal_load(reinterpret_cast<const vec_t*>(p + at));
#pragma unroll
        for (int i = 0; i < 4; ++i) v.x[i] = w[i];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < left) v.x[i] = p[at + i];
    }
    return v;
}
template <class T, Access A>
__device__ __forceinline__ void store4(T* p, int64_t at, int left, const Four<T>& v) {
    if (A == Access::kWhole || (A == Access::kTail && left == 4)) {
        typedef T vec_t __attribute__((ext_vector_type(4)));
        vec_t w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = v.x[i];
        __builtin_nontemporal_store(w, reinterpret_cast<vec_t*>(p + at));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < left) p[at + i] = v.x[i];
    }
}

__device__ __forceinline__ uint32_t word_of(const Four<uint8_t>& c) {
    return c.x[0] | c.x[1] << 8 | c.x[2] << 16 | (uint32_t)c.x[3] << 24;
}
__device__ __forceinline__ Four<uint8_t> bytes_of(uint32_t w) {
    return {{(uint8_t)w, (uint8_t)(w >> 8), (uint8_t)(w >> 16), (uint8_t)(w >> 24)}};
}

template <bool F32>
using Elem = typename std::conditional<F32, float, uint16_t>::type;
__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }

__device__ __forceinline__ Four<uint16_t> to_bf16(const float (&x)[4]) {
    const uint32_t lo = pack_bf16x2(x[0], x[1]), hi = pack_bf16x2(x[2], x[3]);
    return {{(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, (uint16_t)(hi >> 16)}};
}

// Codes of a thread's four elements of a block (half a wave), and its scale.
template <bool ROOT>
__device__ __forceinline__ uint32_t encode4(const float (&x)[4], const uint32_t (&bits16)[4], float& scale) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = umax32(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    top = row16_max(top);
    top = umax32(top, (uint32_t)__shfl_xor((int)top, 16));
    // The scale is a product by its definition; the quotient would differ in the last place of about half of the scales
    // (64M elements: 198.7 us, with a division 203.2).
    // A block that FP32 does not hold reads back as NaN: with an infinite scale the codes of 1 that roots above zero get
    // at least would be infinities, beside which their elements would never move again.
    scale = top < 0x7F800000u ? __uint_as_float(top) * (1.0f / kE4M3Max) : __builtin_nanf("");
    // the quotient of IEEE division, by the reciprocal and one correction (see fp8q_device.h) but for tiny scales; a
    // scale of zero, or a NaN, divides nothing
    GroupScale gs;
    gs.s = scale > 0.0f ? scale : 1.0f;
    gs.slow = !(gs.s >= kSmallScale);
    gs.y = 1.0f / gs.s;
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = quot_fast(__builtin_fabsf(x[i]), gs);
    if (gs.slow) {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = __builtin_fabsf(x[i]) / gs.s;
    }
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t code = stochastic_e4m3(y[i], bits16[i]);
        if (ROOT && code == 0 && x[i] > 0.0f) code = 1;
        code |= (__float_as_uint(x[i]) >> 24) & 0x80u;
        word |= code << (8 * i);
    }
    return word;
}

template <bool P32, bool G32, bool BITS8, Access A>
__device__ __forceinline__ void chunk(const Entry& t, const Scales& scales, int64_t base, const Step& s,
                                      const Factors& f, float grad_scale, uint32_t key) {
    using P = Elem<P32>;
    using G = Elem<G32>;
    P* const param = static_cast<P*>(t.param);
    const G* const grad = static_cast<const G*>(t.grad);
    const int64_t at = base + threadIdx.x * kVec, rest = t.numel - at;
    const int left = rest < 0 ? 0 : (rest < kVec ? (int)rest : kVec);
    const Four<P> p = load4<P, A>(param, at, left);
    const Four<G> g = load4<G, A>(grad, at, left);
    Four<float> m, v;
    Four<uint8_t> mc, vc;
    float ms = 0.0f, vs = 0.0f;
    if constexpr (BITS8) {
        mc = load4<uint8_t, A>(static_cast<const uint8_t*>(t.exp_avg), at, left);
        vc = load4<uint8_t, A>(static_cast<const uint8_t*>(t.exp_avg_sq), at, left);
        if (left > 0) {
            ms = scales.exp_avg[at / kBlock];
            vs = scales.exp_avg_sq[at / kBlock];
        }
    } else {
        m = load4<float, A>(static_cast<const float*>(t.exp_avg), at, left);
        v = load4<float, A>(static_cast<const float*>(t.exp_avg_sq), at, left);
    }
    if constexpr (BITS8) {
        const float4 a = decode4(word_of(mc)), b = decode4(word_of(vc));
        const float am[4] = {a.x, a.y, a.z, a.w}, bm[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m.x[i] = am[i] * ms;
            const float r = bm[i] * vs;
            v.x[i] = r * r;
        }
    }
    float np[4], root[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float gi = as_float(g.x[i]) * grad_scale;
        m.x[i] = m.x[i] * s.b1 + gi * s.c1;
        v.x[i] = v.x[i] * s.b2 + (gi * gi) * s.c2;
        root[i] = sqrtf(v.x[i]);
        np[i] = as_float(p.x[i]) * f.decay - (m.x[i] / (root[i] * f.root + s.eps)) * f.step_size;
    }
    if constexpr (P32) {
        Four<float> w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w.x[i] = np[i];
        store4<float, A>(param, at, left, w);
        if (t.copy) store4<uint16_t, A>(t.copy, at, left, to_bf16(np));
    } else {
        store4<uint16_t, A>(param, at, left, to_bf16(np));
    }
    if constexpr (BITS8) {
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t bits = mix((uint32_t)(at + i) ^ key);
            lo[i] = bits & 0xFFFFu;
            hi[i] = bits >> 16;
            // elements past the tensor must not count in its last block
            if (A != Access::kWhole && i >= left) m.x[i] = root[i] = 0.0f;
        }
        float sm, sv;
        const uint32_t cm = encode4<false>(m.x, lo, sm), cv = encode4<true>(root, hi, sv);
        store4<uint8_t, A>(static_cast<uint8_t*>(t.exp_avg), at, left, bytes_of(cm));
        store4<uint8_t, A>(static_cast<uint8_t*>(t.exp_avg_sq), at, left, bytes_of(cv));
        if (left > 0 && at % kBlock == 0) {
            scales.exp_avg[at / kBlock] = sm;
            scales.exp_avg_sq[at / kBlock] = sv;
        }
    } else {
        store4<float, A>(static_cast<float*>(t.exp_avg), at, left, m);
        store4<float, A>(static_cast<float*>(t.exp_avg_sq), at, left, v);
    }
}

template <bool P32, bool G32, bool BITS8>
__global__ __launch_bounds__(kThreads) void step_kernel(Table<BITS8> table, Step s) {
    const float grad_scale = s.grad_scale ? *s.grad_scale : 1.0f;
    if (!(__builtin_fabsf(grad_scale) < __builtin_inff())) return;
    const int lane = threadIdx.x & 63;
    const int mine = lane < table.count ? table.first[lane] : 0x7FFFFFFF;
    const int i = __builtin_amdgcn_readfirstlane(__popcll(__ballot(mine <= (int)blockIdx.x)) - 1);
    const Entry t = table.t[i];
    const Scales scales = table.s[BITS8 ? i : 0];
    const int64_t base = (int64_t)((int)blockIdx.x - table.first[i]) * kChunk;
    Factors f = s.f;
    uint32_t step32 = (uint32_t)s.step;
    if (s.lr_dev || s.step_dev) {
        int64_t step = s.step_dev ? *s.step_dev : s.step;
        step = step < 1 ? 1 : step;
        step32 = (uint32_t)step;
        f = factors(s.lr_dev ? (double)*s.lr_dev : s.lr, s.weight_decay, s.beta1, s.beta2, step);
    }
    uint32_t key = 0;
    if constexpr (BITS8) {
        key = mix(mix(mix(s.seed_lo) + s.seed_hi) + step32);
        key = mix(mix(key + (uint32_t)(table.place + i)) + (uint32_t)(base >> 32));
    }
    if (((table.vec >> i) & 1) && base + kChunk <= t.numel)
        chunk<P32, G32, BITS8, Access::kWhole>(t, scales, base, s, f, grad_scale, key);
    else if ((table.vec >> i) & 1)
        chunk<P32, G32, BITS8, Access::kTail>(t, scales, base, s, f, grad_scale, key);
    else
        chunk<P32, G32, BITS8, Access::kSingle>(t, scales, base, s, f, grad_scale, key);
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

template <bool BITS8>
void launch(const Table<BITS8>& table, const Step& s, const Options& o, int64_t blocks, hipStream_t stream) {
    const dim3 grid((unsigned)blocks), block(kThreads);
    if (o.param_f32) {
        if (o.grad_f32)
            hipLaunchKernelGGL((step_kernel<true, true, BITS8>), grid, block, 0, stream, table, s);
        else
            hipLaunchKernelGGL((step_kernel<true, false, BITS8>), grid, block, 0, stream, table, s);
    } else {
        if (o.grad_f32)
            hipLaunchKernelGGL((step_kernel<false, true, BITS8>), grid, block, 0, stream, table, s);
        else
            hipLaunchKernelGGL((step_kernel<false, false, BITS8>), grid, block, 0, stream, table, s);
    }
}

template <bool BITS8>
hipError_t launch_tables(int32_t count, const fp8q_adamw_tensor* tensors, const void* const* grads, const Step& s,
                         const Options& o, hipStream_t stream) {
    Table<BITS8> table;
    for (int32_t at = 0; at < count;) {
        // consecutive tensors, so that a place is known from the first one's
        table.place = at;
        table.count = 0;
        table.vec = 0;
        int64_t blocks = 0;
        while (table.count < Table<BITS8>::kMost && at < count) {
            const fp8q_adamw_tensor& t = tensors[at];
            const void* const grad = grads[at];
            const int64_t need = grad ? (t.numel + kChunk - 1) / kChunk : 0;
            if (!launchable({blocks + need, kThreads})) break;  // (no tensor alone: kMostBlocks)
            const int j = table.count++;
            ++at;
            table.t[j] = Entry{t.param, grad, t.exp_avg, t.exp_avg_sq, t.copy, t.numel};
            if (BITS8) table.s[j] = Scales{t.exp_avg_scale, t.exp_avg_sq_scale};
            table.first[j] = (int32_t)blocks;
            const int states = BITS8 ? 4 : 16;
            const bool vec = aligned(t.param, o.param_f32 ? 16 : 8) && aligned(grad, o.grad_f32 ? 16 : 8) &&
                             aligned(t.exp_avg, states) && aligned(t.exp_avg_sq, states) && aligned(t.copy, 8);
            if (vec) table.vec |= 1ULL << j;
            blocks += need;
        }
        if (blocks == 0) continue;
        launch<BITS8>(table, s, o, blocks, stream);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_step(int32_t count, const fp8q_adamw_tensor* tensors, const void* const* grads, const Options& o,
                       hipStream_t stream) {
    Step s = {};
    s.lr = o.lr; s.beta1 = o.beta1; s.beta2 = o.beta2; s.weight_decay = o.weight_decay;
    s.lr_dev = o.lr_dev; s.step_dev = o.step_dev; s.grad_scale = o.grad_scale; s.step = o.step;
    if (!o.lr_dev && !o.step_dev) s.f = factors(o.lr, o.weight_decay, o.beta1, o.beta2, o.step);
    s.b1 = (float)o.beta1; s.c1 = (float)(1.0 - o.beta1);
    s.b2 = (float)o.beta2; s.c2 = (float)(1.0 - o.beta2);
    s.eps = o.eps;
    s.seed_lo = (uint32_t)o.seed; s.seed_hi = (uint32_t)(o.seed >> 32);
    return o.bits8 ? launch_tables<true>(count, tensors, grads, s, o, stream)
                   : launch_tables<false>(count, tensors, grads, s, o, stream);
}

}  // namespace adamw
}  // namespace fp8q
