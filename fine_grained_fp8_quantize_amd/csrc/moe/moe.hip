// moe.hip -- MoE routing kernels for gfx950: the expert-sorted row layout of
// a batch's routes, and the balance loss with its gradient (formulas in
// include/fp8q_moe.h).
//
// The data are small (16384 tokens of 256 fp32 logits: 17 MB, 3 us of HBM each
// way), so what these kernels cost is latency: a launch (2 to 3 us each in a
// stream of them), the loads that follow one another, and the exponentials and
// wave reductions of the scores.
#include "moe/moe.h"

#include "fp8q_device.h"
#include "moe/moe_launch.hpp"

#include <math.h>

#include <type_traits>

namespace fp8q {
namespace moe {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;

__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ int wave_inclusive_sum(int v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int u = __shfl_up(v, d);
        if (lane >= d) v += u;
    }
    return v;
}

// Lane exchange inside the vector unit (DPP); lanes that receive nothing get
// `none`.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ float dpp(float v, float none) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp((int)__float_as_uint(none), (int)__float_as_uint(v),
                                                                 CTRL, ROWS, 0xF, false));
}

// Reductions over the wave, the result in every lane: four steps inside the
// rows of 16 lanes, then row 15's value to the next row and row 31's to the
// upper half, which leaves the whole in lane 63. No LDS permutes: their
// latency, six in a row per reduction, is what a row's scores would wait for.
__device__ __forceinline__ float lane63(float v) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp<0xB1>(v, 0.f);
    v += dpp<0x4E>(v, 0.f);
    v += dpp<0x141>(v, 0.f);
    v += dpp<0x140>(v, 0.f);
    v += dpp<0x142, 0xA>(v, 0.f);
    v += dpp<0x143, 0xC>(v, 0.f);
    return lane63(v);
}
__device__ __forceinline__ float wave_fmax(float v) {
    v = fmaxf(v, dpp<0xB1>(v, -INFINITY));
    v = fmaxf(v, dpp<0x4E>(v, -INFINITY));
    v = fmaxf(v, dpp<0x141>(v, -INFINITY));
    v = fmaxf(v, dpp<0x140>(v, -INFINITY));
    v = fmaxf(v, dpp<0x142, 0xA>(v, -INFINITY));
    v = fmaxf(v, dpp<0x143, 0xC>(v, -INFINITY));
    return lane63(v);
}

// ---------------------------------------------------------------- dispatch

// Routes of one part, counted per expert in LDS (integer sums: any order
// gives the same). 131072 routes, 256 experts: 3.0 us.
__global__ __launch_bounds__(kThreads) void dispatch_count_kernel(DispatchArgs p, int64_t per_part) {
    __shared__ int hist[kMaxExperts];
    const int tid = threadIdx.x;
    if (tid < p.experts) hist[tid] = 0;
    __syncthreads();
    const int64_t beg = (int64_t)blockIdx.x * per_part, end = min(beg + per_part, p.routes);
    for (int64_t i = beg + tid; i < end; i += kThreads) {
        const int64_t e = (int64_t)p.ids[i] - p.first;
        if (e >= 0 && e < p.experts) atomicAdd(&hist[e], 1);
    }
    __syncthreads();
    if (tid < p.experts) p.counts[(int64_t)blockIdx.x * p.experts + tid] = hist[tid];
}

// Destinations of one part's routes. A wave owns a contiguous run of the
// part; its routes' places are: start of the expert's segment + routes of
// earlier parts + of earlier waves + of earlier lanes and rounds of its own.
// Lanes with the same expert find each other with one ballot per bit of the
// expert's number. SINGLE: the part is the whole batch, and the counts are
// its own. 256 experts, 64 parts, a wave's rounds of 64 routes depending on one
// another through `next`: 65536 routes (one round) 6.1 us, 131072 (two) 6.8,
// 262144 8.4, 524288 12.3, 1048576 (16) 20.6. So a round is 0.7 to 1 us, and
// what comes before, the reads of all parts' counts and the sums between five
// barriers, 5 us with the launch. 256 routes, SINGLE: 3.0 us.
template <bool SINGLE>
__global__ __launch_bounds__(kThreads) void dispatch_place_kernel(DispatchArgs p, int64_t per_part, int parts) {
    __shared__ int next[kWaves][kMaxExperts];
    __shared__ int wave_total[kWaves];
    __shared__ int part_sums[2][kThreads];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int experts = p.experts;
    for (int i = lane; i < experts; i += 64) next[wave][i] = 0;
    wave_lds_fence();
    const int64_t per_wave = per_part / kWaves;  // a multiple of 64
    const int64_t beg = (int64_t)blockIdx.x * per_part + wave * per_wave;
    const int64_t end = min(beg + per_wave, p.routes);
    for (int64_t i = beg + lane; i < end; i += 64) {
        const int64_t e = (int64_t)p.ids[i] - p.first;
        if (e >= 0 && e < experts) atomicAdd(&next[wave][e], 1);
    }
    int total = 0, before = 0;
    if constexpr (!SINGLE) {
        // all parts' counts: `shares` threads per expert take every shares-th
        // part each, so that few loads follow each other
        const int width = 64 << (32 - __clz((experts - 1) >> 6)), shares = kThreads / width;
        const int e = tid & (width - 1);
        if (e < experts) {
#pragma unroll 8
            for (int c = tid / width; c < parts; c += shares) {
                const int v = p.counts[(int64_t)c * experts + e];
                total += v;
                before += c < (int)blockIdx.x ? v : 0;
            }
        }
        part_sums[0][tid] = total;
        part_sums[1][tid] = before;
        __syncthreads();
        total = before = 0;
        if (tid < experts) {
            for (int i = tid; i < kThreads; i += width) {
                total += part_sums[0][i];
                before += part_sums[1][i];
            }
        }
    }
    __syncthreads();
    if (SINGLE && tid < experts) {
#pragma unroll
        for (int w = 0; w < kWaves; ++w) total += next[w][tid];
    }
    // start of every expert's segment: running sum of the padded counts
    const int padded = (int)(((int64_t)total + p.align - 1) / p.align * p.align);
    const int incl = wave_inclusive_sum(padded);
    if (lane == 63) wave_total[wave] = incl;
    __syncthreads();
    int start = incl - padded;
    for (int w = 0; w < wave; ++w) start += wave_total[w];
    if (tid < experts) {
        if (blockIdx.x == 0) {
            p.offsets[tid] = start;
            p.rows[tid] = total;
            if (tid == experts - 1) p.offsets[experts] = start + padded;
        }
        int at = start + before;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const int v = next[w][tid];
            next[w][tid] = at;
            at += v;
        }
    }
    __syncthreads();
    const int bits = 32 - __clz(experts - 1);  // (__clz(0) = 32: one expert, no bits)
    for (int64_t i0 = beg; i0 < end; i0 += 64) {
        const int64_t i = i0 + lane;
        const int64_t id = i < end ? (int64_t)p.ids[i] - p.first : -1;
        const bool valid = id >= 0 && id < experts;
        const int e = valid ? (int)id : 0;
        unsigned long long peers = __ballot(valid);
        for (int b = 0; b < bits; ++b) {
            const bool set = (e >> b) & 1;
            const unsigned long long m = __ballot(set);
            peers &= set ? m : ~m;
        }
        const int rank = __popcll(peers & ((1ull << lane) - 1));
        int dst = -1;
        if (valid) dst = next[wave][e] + rank;
        wave_lds_fence();
        if (valid && rank == 0) next[wave][e] += __popcll(peers);
        wave_lds_fence();
        if (i < end) p.dst[i] = dst;
    }
}

// ----------------------------------------------------------------- balance

// The tokens are cut into parts of `chunk` tokens, sequence by sequence. A
// part's workgroup leaves its score sums and route counts per expert and one
// record; the finish kernel adds a sequence's parts in order.
struct Part {
    int seq, first;  // its sequence (-1: unused) and that sequence's first part
    int tokens, routes;
};

constexpr int kChunk = 64;
constexpr int64_t kMaxParts = 1024;  // beyond the sequences' ragged ends

struct BalancePlan {
    int64_t chunk, parts;
    Part* info;
    float* sums;    // [parts][experts]
    int* counts;    // [parts][experts]
    float* losses;  // one per workgroup of the finish kernel
    unsigned* done;
    int64_t bytes;
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

BalancePlan plan_of(int64_t tokens, int64_t experts, int64_t seqs, void* workspace) {
    BalancePlan b;
    b.chunk = kChunk * (tokens > kChunk * kMaxParts ? ceil_div(tokens, kChunk * kMaxParts) : 1);
    b.parts = ceil_div(tokens, b.chunk) + seqs;
    char* at = static_cast<char*>(workspace);
    b.info = reinterpret_cast<Part*>(at);
    at += b.parts * sizeof(Part);
    b.sums = reinterpret_cast<float*>(at);
    at += b.parts * experts * sizeof(float);
    b.counts = reinterpret_cast<int*>(at);
    at += b.parts * experts * sizeof(int);
    b.losses = reinterpret_cast<float*>(at);
    at += seqs * ceil_div(experts, 64) * sizeof(float);
    b.done = reinterpret_cast<unsigned*>(at);
    at += sizeof(unsigned);
    b.bytes = at - static_cast<char*>(workspace);
    return b;
}

// Tokens [beg, end) of sequence s, kept inside the batch.
__device__ __forceinline__ void sequence_span(const BalanceArgs& p, int s, int64_t& beg, int64_t& end) {
    beg = 0;
    end = p.tokens;
    if (p.seq_offsets) {
        beg = p.seq_offsets[s];
        end = p.seq_offsets[s + 1];
    }
    beg = beg < 0 ? 0 : (beg > p.tokens ? p.tokens : beg);
    end = end < beg ? beg : (end > p.tokens ? p.tokens : end);
}

// The sequence of part `slot`, its first part and the part's first token;
// false past the last. Every lane of the wave must take part.
__device__ __forceinline__ bool find_part(const BalanceArgs& p, int64_t chunk, int64_t slot, int& seq, int64_t& first,
                                          int64_t& beg, int64_t& end) {
    const int lane = threadIdx.x & 63;
    int64_t before = 0;
    for (int base = 0; base < p.seqs; base += 64) {
        int64_t b = 0, e = 0;
        if (base + lane < p.seqs) sequence_span(p, base + lane, b, e);
        const int parts = (int)((uint32_t)(e - b + chunk - 1) / (uint32_t)chunk);  // (32-bit: tokens < 2^31)
        const int incl = wave_inclusive_sum(parts);
        const int all = __builtin_amdgcn_readfirstlane(__shfl(incl, 63));
        if (slot < before + all) {
            const int l = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)__ballot(before + incl > slot)) - 1);
            seq = base + l;
            first = before + __builtin_amdgcn_readlane(incl - parts, l);
            beg = __builtin_amdgcn_readlane((int)b, l) + (slot - first) * chunk;
            end = min((int64_t)__builtin_amdgcn_readlane((int)e, l), beg + chunk);
            return true;
        }
        before += all;
    }
    return false;
}

constexpr int kTokensAtOnce = 4;  // rows a wave has in flight

// A lane's share of rows t0, t0 + 1, ... (the last one again past it): experts
// [V lane, V lane + V), -inf past the last. VEC (shares of four and more): rows
// start on boundaries of four logits, 16 or 8 bytes, which are one load.
// Whether a lane reads whole shares is decided once, so that no row's load waits
// for another's.
template <int V, bool F32, bool VEC>
__device__ __forceinline__ void load_rows(const BalanceArgs& p, int64_t t0, int64_t last, float (&x)[kTokensAtOnce][V]) {
    const int e0 = V * (threadIdx.x & 63);
    if (VEC && e0 + V <= p.experts) {
#pragma unroll
        for (int u = 0; u < kTokensAtOnce; ++u) {
            const int64_t at = min(t0 + u, last) * p.ld + e0;
#pragma unroll
            for (int i = 0; i + 3 < V; i += 4) {
                if constexpr (F32) {
                    const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(p.logits) + at + i);
                    x[u][i] = v.x, x[u][i + 1] = v.y, x[u][i + 2] = v.z, x[u][i + 3] = v.w;
                } else {
                    const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.logits) + at + i);
                    x[u][i] = bf16_lo(v.x), x[u][i + 1] = bf16_hi(v.x);
                    x[u][i + 2] = bf16_lo(v.y), x[u][i + 3] = bf16_hi(v.y);
                }
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int u = 0; u < kTokensAtOnce; ++u) x[u][i] = -INFINITY;
        if (e0 + i >= p.experts) continue;
#pragma unroll
        for (int u = 0; u < kTokensAtOnce; ++u) {
            const int64_t at = min(t0 + u, last) * p.ld + e0 + i;
            if constexpr (F32) x[u][i] = static_cast<const float*>(p.logits)[at];
            else x[u][i] = __uint_as_float((uint32_t)static_cast<const uint16_t*>(p.logits)[at] << 16);
        }
    }
}

template <int V, bool F32, bool VEC>
__device__ __forceinline__ void store_row(void* base, int64_t row, int experts, const float (&x)[V]) {
    const int e0 = V * (threadIdx.x & 63);
    if (VEC && e0 + V <= experts) {
#pragma unroll
        for (int i = 0; i + 3 < V; i += 4) {
            if constexpr (F32)
                *reinterpret_cast<float4*>(static_cast<float*>(base) + row + e0 + i) =
                    make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
            else
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + row + e0 + i) =
                    make_uint2(pack_bf16x2(x[i], x[i + 1]), pack_bf16x2(x[i + 2], x[i + 3]));
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (e0 + i >= experts) continue;
        if constexpr (F32) static_cast<float*>(base)[row + e0 + i] = x[i];
        else static_cast<uint16_t*>(base)[row + e0 + i] = (uint16_t)pack_bf16x2(x[i], 0.0f);
    }
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// log sigmoid(x) = min(x, 0) - log(1 + exp(-|x|)): the scores of a row are a
// softmax of these, which holds where the sigmoids themselves underflow.
__device__ __forceinline__ float log_sigmoid(float x) {
    return fminf(x, 0.0f) - kLn2 * __builtin_amdgcn_logf(1.0f + fast_exp(-fabsf(x)));
}

// Scores of one row, lane l holding experts [V l, V l + V); x past the last
// expert must be -inf. A row without a finite score gets zeros, a NaN reaches every
// score of its row.
template <int V, bool SIGMOID>
__device__ __forceinline__ void row_scores(const float (&x)[V], float (&s)[V]) {
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        s[i] = SIGMOID ? log_sigmoid(x[i]) : x[i];
        top = fmaxf(top, s[i]);
    }
    top = wave_fmax(top);
    top = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        s[i] = fast_exp(s[i] - top);
        sum += s[i];
    }
    sum = wave_sum(sum);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] *= inv;
}

// Whether a token has a valid route, for the wave (every lane gets it).
__device__ __forceinline__ int valid_route(const BalanceArgs& p, int64_t token) {
    const int lane = threadIdx.x & 63;
    int id = -1;
    if (lane < p.topk) id = p.ids[token * p.topk + lane];
    return id >= 0 && id < p.experts ? id : -1;
}

// One part: every wave takes four rows at a time, loads them together and adds
// their scores in registers; the waves' sums meet in LDS in wave order. 16384
// x 256 fp32: 10.4 us, 1.6 TB/s: a round trip for the part's place, one for its
// rows, then about 500 vector instructions for each four rows of a wave.
template <int V, bool F32, bool SIGMOID, bool VEC>
__global__ __launch_bounds__(kThreads) void balance_part_kernel(BalanceArgs p, BalancePlan b) {
    __shared__ float sums[kWaves][64 * V];
    __shared__ int hist[64 * V];
    __shared__ int seen[2];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if (blockIdx.x == 0 && tid == 0) *b.done = 0;  // for the finish kernel
    int seq;
    int64_t first, beg, end;
    if (!find_part(p, b.chunk, blockIdx.x, seq, first, beg, end)) {
        if (tid == 0) b.info[blockIdx.x] = Part{-1, 0, 0, 0};
        return;
    }
    if (tid < 64 * V) hist[tid] = 0;
    if (tid < 2) seen[tid] = 0;
    __syncthreads();
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    int tokens = 0, routes = 0;
    // wave w takes the w-th run of the part's tokens
    const int64_t run = b.chunk / kWaves;
    const int64_t stop = min(end, beg + (wave + 1) * run);
    for (int64_t t0 = beg + wave * run; t0 < stop; t0 += kTokensAtOnce) {
        float x[kTokensAtOnce][V];
        int id[kTokensAtOnce];
#pragma unroll
        for (int u = 0; u < kTokensAtOnce; ++u) {
            const int64_t t = t0 + u;
            id[u] = t < stop ? valid_route(p, t) : -1;
        }
        load_rows<V, F32, VEC>(p, t0, stop - 1, x);
#pragma unroll
        for (int u = 0; u < kTokensAtOnce; ++u) {
            // (rows that are not counted go through the same steps, so that the
            // four rows' reductions overlap)
            const unsigned long long valid = __ballot(id[u] >= 0);
            if (id[u] >= 0) atomicAdd(&hist[id[u]], 1);
            tokens += valid != 0;
            routes += __popcll(valid);
            float s[V];
            row_scores<V, SIGMOID>(x[u], s);
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] += valid != 0 ? s[i] : 0.0f;
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) sums[wave][V * lane + i] = acc[i];
    if (lane == 0) {
        atomicAdd(&seen[0], tokens);
        atomicAdd(&seen[1], routes);
    }
    __syncthreads();
    if (tid < p.experts) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) v += sums[w][tid];
        b.sums[(int64_t)blockIdx.x * p.experts + tid] = v;
        b.counts[(int64_t)blockIdx.x * p.experts + tid] = hist[tid];
    }
    if (tid == 0) b.info[blockIdx.x] = Part{seq, (int)first, seen[0], seen[1]};
}

// Adds up one sequence's parts for 64 experts per workgroup (16 waves share
// the parts), then writes its counts and coefficients; the last workgroup to
// finish adds the losses, in their order. 260 parts of 256 experts in 4
// sequences: 8.8 us, five dependent trips to memory (records, sums, the loss's
// hand-over in two, the losses). Every workgroup reads every part's record, so
// the cost grows with sequences times parts (256 experts, both kernels through
// the binding: 16384 tokens in 4, 100, 1000 sequences 18, 25, 142 us; 4096
// sequences of 64 tokens 886 us; 32768 of one token 26.6 ms).
__global__ __launch_bounds__(kThreads) void balance_finish_kernel(BalanceArgs p, BalancePlan b, int slices) {
    __shared__ float sums[kWaves][64];
    __shared__ int counts[kWaves][64];
    __shared__ unsigned bits[kThreads];
    static_assert(kMaxSeqs <= 32 * kThreads, "a bit for every sequence");
    __shared__ int live, seq_first, seq_parts, seq_tokens, seq_routes;
    __shared__ int last;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int s = (int)(blockIdx.x / slices), e = (int)(blockIdx.x % slices) * 64 + lane;
    if (tid == 0) live = seq_first = seq_parts = seq_tokens = seq_routes = 0;
    bits[tid] = 0;
    __syncthreads();
    // this sequence's totals, and how many sequences have a counted token: one
    // bit each, so that no load waits for another
    for (int64_t i = tid; i < b.parts; i += kThreads) {
        const Part a = b.info[i];
        if (a.seq == s) {
            if (a.first == i) seq_first = (int)i;
            atomicAdd(&seq_parts, 1);
            atomicAdd(&seq_tokens, a.tokens);
            atomicAdd(&seq_routes, a.routes);
        }
        if (a.tokens > 0) atomicOr(&bits[a.seq >> 5], 1u << (a.seq & 31));
    }
    __syncthreads();
    if (bits[tid]) atomicAdd(&live, __popc(bits[tid]));
    __syncthreads();
    float sum = 0.0f;
    int count = 0;
    if (e < p.experts) {
#pragma unroll 4
        for (int i = wave; i < seq_parts; i += kWaves) {
            const int64_t at = (int64_t)(seq_first + i) * p.experts + e;
            sum += b.sums[at];
            count += b.counts[at];
        }
    }
    sums[wave][lane] = sum;
    counts[wave][lane] = count;
    __syncthreads();
    if (wave == 0) {
        for (int w = 1; w < kWaves; ++w) {
            sum += sums[w][lane];
            count += counts[w][lane];
        }
        float part = 0.0f;
        if (e < p.experts) {
            const float f = seq_tokens > 0 ? p.alpha * (float)p.experts * (float)count / (float)seq_routes : 0.0f;
            const float w = seq_tokens > 0 ? f / ((float)seq_tokens * (float)live) : 0.0f;
            p.counts[(int64_t)s * p.experts + e] = count;
            p.coef[(int64_t)s * p.experts + e] = w;
            part = w * sum;
        }
        part = wave_sum(part);
        if (lane == 0) {
            b.losses[blockIdx.x] = part;
            last = __hip_atomic_fetch_add(b.done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
        }
    }
    __syncthreads();
    if (!last || wave != 0) return;
    // a lane adds up to 8192 terms (32768 sequences, 1024 experts) one after the
    // other, of any sizes: in FP32 small ones behind a large one would be lost
    double v = 0.0;
    for (unsigned i = lane; i < gridDim.x; i += 64)
        v += (double)__hip_atomic_load(&b.losses[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const float loss = wave_sum((float)v);
    if (lane == 0) *p.loss = loss;
}

// Four rows per wave, scores computed again rather than read (they would be as
// many bytes as the logits): 16384 x 256 fp32: 11.7 us, 2.9 TB/s read and written.
template <int V, bool F32, bool SIGMOID, bool VEC>
__global__ __launch_bounds__(kBackwardThreads) void balance_backward_kernel(BalanceArgs p) {
    static_assert(kBackwardRows == kBackwardThreads / 64 * kTokensAtOnce, "every wave takes its rows once");
    const int lane = threadIdx.x & 63;
    const int64_t t0 = p.token0 + ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * kTokensAtOnce;
    if (t0 >= p.tokens) return;
    float x[kTokensAtOnce][V];
    int id[kTokensAtOnce];
#pragma unroll
    for (int u = 0; u < kTokensAtOnce; ++u) {
        const int64_t t = t0 + u;
        id[u] = t < p.tokens ? valid_route(p, t) : -1;
    }
    load_rows<V, F32, VEC>(p, t0, p.tokens - 1, x);
    const float g = p.grad ? *p.grad : 1.0f;
    // the sequence of the first row: the last one that starts at or before it
    int seq = 0;
    if (p.seq_offsets) {
        int hi = p.seqs;  // seq_offsets[seq] <= t0 < seq_offsets[hi]
        while (hi - seq > 1) {
            const int mid = (seq + hi) / 2;
            if (p.seq_offsets[mid] <= t0) seq = mid; else hi = mid;
        }
    }
    float w[V];
    int have = -1;
#pragma unroll
    for (int u = 0; u < kTokensAtOnce; ++u) {
        const int64_t t = t0 + u;
        if (t >= p.tokens) break;
        if (p.seq_offsets)
            while (seq + 1 < p.seqs && p.seq_offsets[seq + 1] <= t) ++seq;
        if (have != seq) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = V * lane + i;
                w[i] = e < p.experts ? p.coef[(int64_t)seq * p.experts + e] : 0.0f;
            }
            have = seq;
        }
        const bool counted = __ballot(id[u] >= 0) != 0;
        float s[V], d[V];
        row_scores<V, SIGMOID>(x[u], s);
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) dot += s[i] * w[i];
        dot = wave_sum(dot);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            d[i] = g * s[i] * (w[i] - dot);
            if (SIGMOID) d[i] *= 1.0f / (1.0f + fast_exp(x[u][i]));
            d[i] = counted ? d[i] : 0.0f;
        }
        store_row<V, F32, VEC>(p.dlogits, t * p.ld_d, p.experts, d);
    }
}

// One launch for the values-per-lane, type, score and alignment of the
// arguments.
template <int V, class F>
hipError_t with_types(const BalanceArgs& p, bool vec, F&& launch) {
    using N = std::integral_constant<int, V>;
    const auto aligned = [&](auto f32, auto sigmoid) {
        if constexpr (V >= 4) {
            if (vec) return launch(N{}, f32, sigmoid, std::true_type{});
        }
        launch(N{}, f32, sigmoid, std::false_type{});
    };
    if (p.f32) {
        if (p.sigmoid) aligned(std::true_type{}, std::true_type{});
        else aligned(std::true_type{}, std::false_type{});
    } else {
        if (p.sigmoid) aligned(std::false_type{}, std::true_type{});
        else aligned(std::false_type{}, std::false_type{});
    }
    return hipGetLastError();
}

// Four logits (16 or 8 bytes) at a time stay aligned in every row.
bool rows_aligned(const void* p, int64_t ld, bool f32) {
    return reinterpret_cast<uintptr_t>(p) % (f32 ? 16 : 8) == 0 && ld % 4 == 0;
}

template <class F>
hipError_t with_width(const BalanceArgs& p, bool vec, F&& launch) {
    if (p.experts <= 64) return with_types<1>(p, vec, launch);
    if (p.experts <= 128) return with_types<2>(p, vec, launch);
    if (p.experts <= 256) return with_types<4>(p, vec, launch);
    if (p.experts <= 512) return with_types<8>(p, vec, launch);
    return with_types<16>(p, vec, launch);
}

}  // namespace

hipError_t launch_dispatch(const DispatchArgs& p, hipStream_t stream) {
    const dim3 block(kThreads);
    int64_t parts = ceil_div(p.routes, kThreads);
    if (parts > kDispatchParts) parts = kDispatchParts;
    // One workgroup does it all while its waves stay within 4 rounds of 64
    // routes: a second launch costs more (2048 routes to 256 experts: 4.9 against
    // 6.5 us; 4096: 6.8 either way; 8192: 10.8 against 7.2).
    if (p.routes <= 4 * kThreads) {
        const int64_t per_part = ceil_div(p.routes > 0 ? p.routes : 1, kThreads) * kThreads;
        hipLaunchKernelGGL((dispatch_place_kernel<true>), dim3(1), block, 0, stream, p, per_part, 1);
        return hipGetLastError();
    }
    const int64_t per_part = ceil_div(ceil_div(p.routes, parts), kThreads) * kThreads;
    parts = ceil_div(p.routes, per_part);
    hipLaunchKernelGGL(dispatch_count_kernel, dim3((unsigned)parts), block, 0, stream, p, per_part);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((dispatch_place_kernel<false>), dim3((unsigned)parts), block, 0, stream, p, per_part, (int)parts);
    return hipGetLastError();
}

int64_t balance_workspace_bytes(int64_t tokens, int64_t experts, int64_t seqs) {
    return plan_of(tokens, experts, seqs, nullptr).bytes;
}

hipError_t launch_balance(const BalanceArgs& p, hipStream_t stream) {
    const BalancePlan b = plan_of(p.tokens, p.experts, p.seqs, p.workspace);
    const bool vec = rows_aligned(p.logits, p.ld, p.f32);
    const hipError_t e = with_width(p, vec, [&](auto v, auto f32, auto sigmoid, auto aligned) {
        hipLaunchKernelGGL((balance_part_kernel<decltype(v)::value, decltype(f32)::value, decltype(sigmoid)::value,
                                                decltype(aligned)::value>),
                           dim3((unsigned)b.parts), dim3(kThreads), 0, stream, p, b);
    });
    if (e != hipSuccess) return e;
    const int slices = (int)ceil_div(p.experts, 64);
    hipLaunchKernelGGL(balance_finish_kernel, dim3((unsigned)(p.seqs * slices)), dim3(kThreads), 0, stream, p, b, slices);
    return hipGetLastError();
}

hipError_t launch_balance_backward(const BalanceArgs& p, hipStream_t stream) {
    const bool vec = rows_aligned(p.logits, p.ld, p.f32) && rows_aligned(p.dlogits, p.ld_d, p.f32);
    for (int64_t t0 = 0; t0 < p.tokens; t0 += kBackwardTokens) {
        BalanceArgs a = p;
        a.token0 = t0;
        const LaunchShape shape = backward_shape(p.tokens - t0 < kBackwardTokens ? p.tokens - t0 : kBackwardTokens);
        const hipError_t e = with_width(a, vec, [&](auto v, auto f32, auto sigmoid, auto aligned) {
            hipLaunchKernelGGL((balance_backward_kernel<decltype(v)::value, decltype(f32)::value,
                                                        decltype(sigmoid)::value, decltype(aligned)::value>),
                               dim3((unsigned)shape.blocks), dim3(shape.threads), 0, stream, a);
        });
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace moe
}  // namespace fp8q
