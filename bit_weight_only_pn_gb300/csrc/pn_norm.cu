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
#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "pn_device.cuh"
#include "pn_internal.h"

namespace pn {
namespace {

constexpr int kWarpRowHidden = 1024;           // rows up to this size are a warp's
constexpr int kWarpRowThreads = 128;

// V values of a row from element `at` on.  Every element belongs to one thread of
// one block, which reads it before it writes it: r' may take the place of r.
template <int V>
__device__ __forceinline__ void load(const void* p, int64_t at, bool f16, float* v) {
    if (f16) {
        const __half* h = static_cast<const __half*>(p) + at;
        if constexpr (V == 4) {
            const uint2 w = __ldcs(reinterpret_cast<const uint2*>(h));
            v[0] = half_bits_to_float(w.x & 0xFFFFu);
            v[1] = half_bits_to_float(w.x >> 16);
            v[2] = half_bits_to_float(w.y & 0xFFFFu);
            v[3] = half_bits_to_float(w.y >> 16);
        } else {
            v[0] = __half2float(*h);
        }
    } else {
        const float* f = static_cast<const float*>(p) + at;
        if constexpr (V == 4) {
            const float4 w = __ldcs(reinterpret_cast<const float4*>(f));
            v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
        } else {
            v[0] = *f;
        }
    }
}

template <int V>
__device__ __forceinline__ void load_vector(const float* p, int at, float* v) {
    if constexpr (V == 4) {
        const float4 w = *reinterpret_cast<const float4*>(p + at);
        v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
    } else {
        v[0] = p[at];
    }
}

template <int V>
__device__ __forceinline__ void store_half(__half* p, int64_t at, const float* v) {
    if constexpr (V == 4) {
        const __half2 a = __floats2half2_rn(v[0], v[1]), b = __floats2half2_rn(v[2], v[3]);
        *reinterpret_cast<uint2*>(p + at) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    } else {
        p[at] = __float2half_rn(v[0]);
    }
}

template <int V>
__device__ __forceinline__ void store(void* p, int64_t at, bool f16, const float* v) {
    if (f16) return store_half<V>(static_cast<__half*>(p), at, v);
    float* f = static_cast<float*>(p) + at;
    if constexpr (V == 4) *reinterpret_cast<float4*>(f) = make_float4(v[0], v[1], v[2], v[3]);
    else *f = v[0];
}

// Sum over the threads of a row (a warp or the block), the same bits in all of
// them.  Every call of a row takes a place of its own in `part`.
template <bool kWarpRow>
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    if constexpr (!kWarpRow) {
        const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        if (lane == 0) part[threadIdx.x >> 5] = v;
        __syncthreads();
        v = lane < warps ? part[lane] : 0.0f;
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    }
    return v;
}

// A thread has N groups of V values: those of group k begin at (k * threads +
// its place in the row) * V, and lie wholly inside the row or outside.
template <int V, int N, bool kWarpRow>
__device__ __forceinline__ void norm_row(float (&v)[N][V], int kind, const float* weight, const float* bias, float eps, int hidden,
                                         int place, int step, float* part) {
    const float each = 1.0f / static_cast<float>(hidden);
    if (kind == PN_NORM_LAYER) {
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) sum += v[k][i];            // (values behind the row's end are 0)
        const float mean = row_sum<kWarpRow>(sum, part) * each;
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (place + k * step < hidden)
#pragma unroll
                for (int i = 0; i < V; ++i) v[k][i] -= mean;
    }
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) sum = fmaf(v[k][i], v[k][i], sum);
    const float inv = 1.0f / sqrtf(row_sum<kWarpRow>(sum, part + 32) * each + eps);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int at = place + k * step;
        if (at >= hidden) continue;
        float w[V], b[V];
        if (weight) load_vector<V>(weight, at, w);
        if (bias) load_vector<V>(bias, at, b);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            v[k][i] *= inv;
            if (weight) v[k][i] *= w[i];
            if (bias) v[k][i] += b[i];
        }
    }
}

template <int V, int N, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? kWarpRowThreads : 1024) norm_kernel(const NormArgs a) {
    __shared__ float parts[kWarpRow ? 1 : 4 * 32];     // a place to each of a row's sums
    const int threads = kWarpRow ? 32 : blockDim.x, place = (kWarpRow ? threadIdx.x & 31 : threadIdx.x) * V, step = threads * V;
    const int64_t t = kWarpRow ? static_cast<int64_t>(blockIdx.x) * (kWarpRowThreads / 32) + (threadIdx.x >> 5) : blockIdx.x;
    if (t >= a.tokens) return;                         // (a whole warp, of rows that are warps')
    // r is on its way beside y, but where two rows do not fit a thread's registers
    constexpr bool kLate = N * V > 16;
    float v[N][V], r[N][V];
    auto load_residual = [&](int k) {
        const int at = place + k * step;
#pragma unroll
        for (int i = 0; i < V; ++i) r[k][i] = 0.0f;
        if (a.residual && at < a.hidden) load<V>(a.residual, t * a.residual_stride + at, a.residual_f16, r[k]);
    };
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int at = place + k * step;
#pragma unroll
        for (int i = 0; i < V; ++i) v[k][i] = 0.0f;
        if (a.y && at < a.hidden) load<V>(a.y, t * a.y_stride + at, a.y_f16, v[k]);
        if (!kLate) load_residual(k);
    }
    if (a.post != PN_NORM_NONE) norm_row<V, N, kWarpRow>(v, a.post, a.post_weight, a.post_bias, a.eps, a.hidden, place, step, parts);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int at = place + k * step;
        if (kLate) load_residual(k);
        if (!a.y || at >= a.hidden) continue;
        float g[V];
        if (a.gate) load_vector<V>(a.gate + t * a.gate_stride, at, g);
#pragma unroll
        for (int i = 0; i < V; ++i) r[k][i] = fmaf(a.scale, a.gate ? v[k][i] * g[i] : v[k][i], r[k][i]);
    }
    if (a.residual_out)
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int at = place + k * step;
            if (at < a.hidden) store<V>(a.residual_out, t * a.out_stride + at, a.out_f16, r[k]);
        }
    if (!a.x) return;
    if (a.pre != PN_NORM_NONE) norm_row<V, N, kWarpRow>(r, a.pre, a.pre_weight, a.pre_bias, a.eps, a.hidden, place, step, kWarpRow ? parts : parts + 64);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int at = place + k * step;
        if (at < a.hidden) store_half<V>(a.x, t * a.hidden + at, r[k]);
    }
}

template <int V, int N, bool kWarpRow>
cudaError_t launch(const NormArgs& a, cudaStream_t s) {
    const int groups = (a.hidden + V - 1) / V, threads = kWarpRow ? kWarpRowThreads : ((groups + N - 1) / N + 31) / 32 * 32;
    const int64_t blocks = kWarpRow ? (a.tokens + kWarpRowThreads / 32 - 1) / (kWarpRowThreads / 32) : a.tokens;
    norm_kernel<V, N, kWarpRow><<<static_cast<unsigned>(blocks), threads, 0, s>>>(a);
    return cudaGetLastError();
}

// The least N of its list with which the block has at most 1024 threads (of rows that
// are warps': a warp), but no less than `least`.
template <int V, bool kWarpRow, int N, int... More>
cudaError_t choose(const NormArgs& a, int least, cudaStream_t s) {
    if constexpr (sizeof...(More) > 0) {
        if (N < least || (a.hidden + V - 1) / V > N * (kWarpRow ? 32 : 1024)) return choose<V, kWarpRow, More...>(a, least, s);
    }
    return launch<V, N, kWarpRow>(a, s);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, int num_sms, cudaStream_t s) {
    // fours where every row lies for them
    auto fits = [](const void* p, uintptr_t bytes, int64_t stride) { return !p || (reinterpret_cast<uintptr_t>(p) % bytes == 0 && stride % 4 == 0); };
    const bool fours = a.hidden % 4 == 0 && fits(a.y, a.y_f16 ? 8 : 16, a.y_stride) && fits(a.residual, a.residual_f16 ? 8 : 16, a.residual_stride) &&
                       fits(a.residual_out, a.out_f16 ? 8 : 16, a.out_stride) && fits(a.gate, 16, a.gate_stride) && fits(a.post_weight, 16, 0) &&
                       fits(a.post_bias, 16, 0) && fits(a.pre_weight, 16, 0) && fits(a.pre_bias, 16, 0) && fits(a.x, 8, 0);
    if (a.hidden <= kWarpRowHidden) return fours ? choose<4, true, 2, 4, 8>(a, 0, s) : choose<1, true, 8, 16, 32>(a, 0, s);
    const bool many = a.tokens > num_sms;
    return fours ? choose<4, false, 1, 2, 4, 8>(a, many ? 4 : 0, s) : choose<1, false, 4, 8, 16, 32>(a, many ? 16 : 0, s);
}

}  // namespace pn
