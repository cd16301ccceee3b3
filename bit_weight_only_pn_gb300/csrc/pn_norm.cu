// pn_norm.cu -- a block's output into the residual stream, with the norms
// before and after it, its gate and its scale, and the next GEMV's input.
//
//   z = post(y)    r' = r + scale * gate * z    x = fp16(pre(r'))
//   rms:   v / sqrt(mean(v^2) + eps) * w + b
//   layer: (v - mean) / sqrt(mean((v - mean)^2) + eps) * w + b
//
// One pass over memory: a row's values stay in registers from its loads to its
// stores, so y, r and a gate of every token are read once and r' and x written
// once.  The variance is that of the differences from the mean (a second walk over
// the registers), so a large mean costs no bits.  Everything is fp32 and rounded
// where it is stored: x is made of r' before that is rounded.
//
// Bound by memory: 8192 rows of 5120 fp32 values (y, r in, r', x out) take 90 us, 6.5
// TB/s; with a gate for each token, mean and variance norms and their vectors, 4096 rows
// of 6144, 76 us, 5.3 TB/s (two barriers a row, between which a block's loads wait).
// One row of 5120: 2.7 us, launch and latency; rows that do not lie for vectors of
// four, 5003 values each: 114 us for 8192, 4.9 TB/s.
#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "pn_device.cuh"
#include "pn_internal.h"

namespace pn {
namespace {

constexpr int kWarpRowHidden = 1024;           // rows up to this size are a warp's
constexpr int kWarpRowThreads = 128;
constexpr unsigned kFewBlocks = 256;

// A thread has N groups of V values of a row: those of group k begin at place +
// k * step, and lie wholly inside the row or outside, where they count as 0.  Loads of
// a thread's groups stand together, without a branch between them (groups outside
// the row read its last one): loaded and used one group after the other, each waited
// for the one before, and 13 rows of 5003 took 12 us.
template <int V, int N>
struct Groups {
    int place, step, hidden;
    __device__ __forceinline__ int at(int k) const { return place + k * step; }
    __device__ __forceinline__ bool inside(int k) const { return at(k) < hidden; }
    // from row element 0 at p; every element is its thread's alone, which reads it before it
    // writes it (r' may take the place of r)
    template <bool kF16>
    __device__ __forceinline__ void load(const void* p, float (&v)[N][V]) const {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int from = min(at(k), hidden - V);
            if constexpr (kF16) {
                const __half* h = static_cast<const __half*>(p) + from;
                if constexpr (V == 4) {
                    const uint2 w = __ldcs(reinterpret_cast<const uint2*>(h));
                    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w.x)), b = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
                    v[k][0] = a.x; v[k][1] = a.y; v[k][2] = b.x; v[k][3] = b.y;
                } else {
                    v[k][0] = __half2float(*h);
                }
            } else {
                const float* f = static_cast<const float*>(p) + from;
                if constexpr (V == 4) {
                    const float4 w = __ldcs(reinterpret_cast<const float4*>(f));
                    v[k][0] = w.x; v[k][1] = w.y; v[k][2] = w.z; v[k][3] = w.w;
                } else {
                    v[k][0] = *f;
                }
            }
        }
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) v[k][i] = inside(k) ? v[k][i] : 0.0f;
    }
    // v = f(v, a vector's values)
    template <typename F>
    __device__ __forceinline__ void with(const float* p, float (&v)[N][V], F f) const {
        float w[N][V];
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const float* from = p + min(at(k), hidden - V);
            if constexpr (V == 4) {
                const float4 u = *reinterpret_cast<const float4*>(from);
                w[k][0] = u.x; w[k][1] = u.y; w[k][2] = u.z; w[k][3] = u.w;
            } else {
                w[k][0] = *from;
            }
        }
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) v[k][i] = f(v[k][i], w[k][i]);
    }
    // what is read later comes nearer
    __device__ __forceinline__ void prefetch(const void* p, int size) const {
#pragma unroll
        for (int k = 0; k < N; ++k) prefetch_l1(static_cast<const uint8_t*>(p) + static_cast<int64_t>(min(at(k), hidden - V)) * size);
    }
};

template <int V>
__device__ __forceinline__ void store_half(__half* p, int64_t at, const float* v) {
    if constexpr (V == 4) {
        const __half2 a = __floats2half2_rn(v[0], v[1]), b = __floats2half2_rn(v[2], v[3]);
        __stcs(reinterpret_cast<uint2*>(p + at), make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b)));
    } else {
        p[at] = __float2half_rn(v[0]);
    }
}

template <int V>
__device__ __forceinline__ void store(void* p, int64_t at, bool f16, const float* v) {
    if (f16) return store_half<V>(static_cast<__half*>(p), at, v);
    float* f = static_cast<float*>(p) + at;
    if constexpr (V == 4) __stcs(reinterpret_cast<float4*>(f), make_float4(v[0], v[1], v[2], v[3]));
    else __stcs(f, v[0]);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    return v;
}

// Number, mean and sum of squared differences from it, of values.
struct Moments {
    float n, mean, m2;
};
// The same over the lanes, in all of them: sums of n and of n mean give the common
// mean, and what a lane's mean is off it adds n times its square.
__device__ __forceinline__ Moments over_lanes(const Moments& m) {
    const float n = warp_sum(m.n), mean = warp_sum(m.n * m.mean) / fmaxf(n, 1.0f), off = m.mean - mean;
    return {n, mean, warp_sum(fmaf(m.n * off, off, m.m2))};
}

// A row's norm, with one barrier (none where the row is a warp's); `part` is its own
// place in shared memory.
template <int V, int N, bool kWarpRow>
__device__ __forceinline__ void norm_row(float (&v)[N][V], const Groups<V, N>& g, int kind, const float* weight, const float* bias, float eps, float* part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    float mean = 0.0f, squares;
    if (kind == PN_NORM_LAYER) {
        // about the thread's own mean first: a large mean costs no bits
        float n = 0.0f, sum = 0.0f;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            n += g.inside(k) ? static_cast<float>(V) : 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) sum += v[k][i];
        }
        Moments m{n, sum / fmaxf(n, 1.0f), 0.0f};
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (g.inside(k))
#pragma unroll
                for (int i = 0; i < V; ++i) m.m2 = fmaf(v[k][i] - m.mean, v[k][i] - m.mean, m.m2);
        m = over_lanes(m);
        if constexpr (!kWarpRow) {
            if (lane == 0) {
                part[warp] = m.n;
                part[32 + warp] = m.mean;
                part[64 + warp] = m.m2;
            }
            __syncthreads();
            m = over_lanes(lane < warps ? Moments{part[lane], part[32 + lane], part[64 + lane]} : Moments{0.0f, 0.0f, 0.0f});
        }
        mean = m.mean;
        squares = m.m2;
    } else {
        squares = 0.0f;
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) squares = fmaf(v[k][i], v[k][i], squares);
        squares = warp_sum(squares);
        if constexpr (!kWarpRow) {
            if (lane == 0) part[warp] = squares;
            __syncthreads();
            squares = warp_sum(lane < warps ? part[lane] : 0.0f);
        }
    }
    const float inv = 1.0f / sqrtf(squares * (1.0f / static_cast<float>(g.hidden)) + eps);
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) v[k][i] = (v[k][i] - mean) * inv;
    if (weight) g.with(weight, v, [](float x, float w) { return x * w; });
    if (bias) g.with(bias, v, [](float x, float w) { return x + w; });
}

// Groups of a thread, a block's threads at most, and blocks to an SM at least: what the registers allow.
template <int kN, int kThreads, int kBlocks>
struct Split {
    static constexpr int N = kN, threads = kThreads, blocks = kBlocks;
};

template <int V, typename S, bool kWarpRow, bool kYF16, bool kRF16>
__global__ void __launch_bounds__(S::threads, S::blocks) norm_kernel(const NormArgs a) {
    constexpr int N = S::N;
    __shared__ float parts[kWarpRow ? 1 : 2 * 96];     // a place to each of a row's norms
    const int64_t t = kWarpRow ? static_cast<int64_t>(blockIdx.x) * (kWarpRowThreads / 32) + (threadIdx.x >> 5) : blockIdx.x;
    if (t >= a.tokens) return;                         // (a whole warp, of rows that are warps')
    const int threads = kWarpRow ? 32 : blockDim.x;
    const Groups<V, N> g{static_cast<int>(kWarpRow ? threadIdx.x & 31 : threadIdx.x) * V, threads * V, a.hidden};
    const uint8_t* y = static_cast<const uint8_t*>(a.y) + t * a.y_stride * (kYF16 ? 2 : 4);
    const uint8_t* residual = static_cast<const uint8_t*>(a.residual) + t * a.residual_stride * (kRF16 ? 2 : 4);
    const float* gate = a.gate + t * a.gate_stride;
    // r is on its way beside y, but where two rows do not fit a thread's registers
    constexpr bool kLate = N * V > 16;
    float v[N][V] = {}, r[N][V] = {};
    if (a.y) g.template load<kYF16>(y, v);
    if (a.residual) {
        if (kLate) g.prefetch(residual, kRF16 ? 2 : 4);
        else g.template load<kRF16>(residual, r);
    }
    if (a.gate && (a.gate_stride != 0 || gridDim.x <= kFewBlocks)) g.prefetch(gate, 4);
    if (gridDim.x <= kFewBlocks) {             // (later rows find the vectors in L1)
        if (a.post_weight) g.prefetch(a.post_weight, 4);
        if (a.pre_weight) g.prefetch(a.pre_weight, 4);
    }
    if (a.post != PN_NORM_NONE) norm_row<V, N, kWarpRow>(v, g, a.post, a.post_weight, a.post_bias, a.eps, parts);
    if (kLate && a.residual) g.template load<kRF16>(residual, r);
    if (a.gate) g.with(gate, v, [](float x, float w) { return x * w; });
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) r[k][i] = g.inside(k) && a.y ? fmaf(a.scale, v[k][i], r[k][i]) : r[k][i];
    if (a.residual_out)
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (g.inside(k)) store<V>(a.residual_out, t * a.out_stride + g.at(k), kRF16, r[k]);
    if (!a.x) return;
    if (a.pre != PN_NORM_NONE) norm_row<V, N, kWarpRow>(r, g, a.pre, a.pre_weight, a.pre_bias, a.eps, kWarpRow ? parts : parts + 96);
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (g.inside(k)) store_half<V>(a.x, t * a.hidden + g.at(k), r[k]);
}

template <int V, typename S, bool kWarpRow, bool kYF16, bool kRF16>
cudaError_t launch(const NormArgs& a, cudaStream_t s) {
    const int groups = (a.hidden + V - 1) / V, threads = kWarpRow ? kWarpRowThreads : ((groups + S::N - 1) / S::N + 31) / 32 * 32;
    const int64_t blocks = kWarpRow ? (a.tokens + kWarpRowThreads / 32 - 1) / (kWarpRowThreads / 32) : a.tokens;
    norm_kernel<V, S, kWarpRow, kYF16, kRF16><<<static_cast<unsigned>(blocks), threads, 0, s>>>(a);
    return cudaGetLastError();
}
template <int V, typename S, bool kWarpRow>
cudaError_t launch(const NormArgs& a, cudaStream_t s) {
    if (a.y_f16) return a.residual_f16 ? launch<V, S, kWarpRow, true, true>(a, s) : launch<V, S, kWarpRow, true, false>(a, s);
    return a.residual_f16 ? launch<V, S, kWarpRow, false, true>(a, s) : launch<V, S, kWarpRow, false, false>(a, s);
}

// The first of its list with no fewer groups to a thread than `least` with which the block
// (of rows that are warps': a warp) has threads enough.
template <int V, bool kWarpRow, typename S, typename... More>
cudaError_t choose(const NormArgs& a, int least, cudaStream_t s) {
    if constexpr (sizeof...(More) > 0) {
        if (S::N < least || (a.hidden + V - 1) / V > S::N * (kWarpRow ? 32 : S::threads)) return choose<V, kWarpRow, More...>(a, least, s);
    }
    return launch<V, S, kWarpRow>(a, s);
}
template <int N>
using OfWarp = Split<N, kWarpRowThreads, 1>;

}  // namespace

static_assert(kWarpRowHidden <= 4 * 8 * 32 && kWarpRowHidden <= 32 * 32 && PN_MAX_HIDDEN <= 4 * 16 * 512 && PN_MAX_HIDDEN <= 64 * 512, "the longest rows fit");

cudaError_t launch_norm(const NormArgs& a, int num_sms, cudaStream_t s) {
    // fours where every row lies for them
    auto fits = [](const void* p, uintptr_t bytes, int64_t stride) { return !p || (reinterpret_cast<uintptr_t>(p) % bytes == 0 && stride % 4 == 0); };
    const bool fours = a.hidden % 4 == 0 && fits(a.y, a.y_f16 ? 8 : 16, a.y_stride) && fits(a.residual, a.residual_f16 ? 8 : 16, a.residual_stride) &&
                       fits(a.residual_out, a.residual_f16 ? 8 : 16, a.out_stride) && fits(a.gate, 16, a.gate_stride) && fits(a.post_weight, 16, 0) &&
                       fits(a.post_bias, 16, 0) && fits(a.pre_weight, 16, 0) && fits(a.pre_bias, 16, 0) && fits(a.x, 8, 0);
    // (rows of 128 with four groups to a lane, three of them outside: 200000 of them 100 us instead of 47; rows of 1280
    // and 2048 as a warp's: 57 and 60 us for 16384, as a block's 45 and 54)
    if (a.hidden <= kWarpRowHidden) return fours ? choose<4, true, OfWarp<1>, OfWarp<2>, OfWarp<4>, OfWarp<8>>(a, 0, s) : choose<1, true, OfWarp<8>, OfWarp<32>>(a, 0, s);
    const bool many = a.tokens > num_sms;
    // Few rows: as many threads to each as there are.  Many: four groups to a thread keep most bytes on their way; above
    // 6144 values eight, of fp32 without spilling (102 registers, in microseconds: 4096 rows of 8192 73 against 82 with
    // 64, of 10240 90 and 104), of fp16 with two blocks to an SM (fewer bytes to a group: 55 against 61).
    if (!fours)
        return choose<1, false, Split<8, 1024, 1>, Split<16, 512, 2>, Split<32, 512, 1>, Split<32, 640, 1>, Split<64, 512, 1>>(a, many ? 16 : 0, s);
    if (!many) return choose<4, false, Split<1, 1024, 1>, Split<2, 1024, 1>, Split<4, 1024, 1>, Split<8, 640, 1>, Split<16, 512, 1>>(a, 0, s);
    const bool halves = (!a.y || a.y_f16) && (!a.residual || a.residual_f16);
    if (halves && a.hidden <= 4 * 8 * 512) return choose<4, false, Split<4, 384, 3>, Split<8, 512, 2>>(a, 0, s);
    return choose<4, false, Split<4, 384, 3>, Split<8, 640, 1>, Split<16, 512, 1>>(a, 0, s);
}

}  // namespace pn
