// pn_norm.cu -- a block's output into the residual stream, with the norms
// before and after it, its gate and its scale, and the next GEMV's input.
//
//   z = post(y)    r' = r + scale * gate * z    x = fp16(pre(r'))
//   rms:   v / sqrt(mean(v^2) + eps) * w + b
//   layer: (v - mean) / sqrt(mean((v - mean)^2) + eps) * w + b
//
// One pass over memory: a row's values stay with their threads from its loads to its
// stores, in registers but for some that the longer splits spill (at the rule), so y, r
// and a gate of every token are read once and r' and x written once.  The variance is
// that of the differences from the mean (a second walk over the registers), so a large
// mean costs no bits.  Everything is fp32 and rounded where it is stored: x is made of r'
// before that is rounded.  A row's sums do not depend on how many threads have it.
//
// Bound by memory: 8192 rows of 5120 fp32 values (y, r in, r', x out) take 85 us, 6.9
// TB/s; with a gate for each token, mean and variance norms and their vectors, 4096 rows
// of 6144, 76 us, 5.3 TB/s (two barriers a row, between which a block's loads wait).
// One row of 5120: 3.3 us, launch and latency; rows that do not lie for vectors of
// four, 5003 values each: 93 us for 8192, 6.2 TB/s.
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

// A segment of a row: 256 values, of which a lane has 8, in groups of V = 4 or 1 that lie
// a warp's width apart.  (Rows that are a warp's: a warp's width.)
template <int V, bool kWarpRow>
constexpr int kOfSegment = kWarpRow ? 1 : 8 / V;       // groups of a lane

// A thread has N groups of V values of a row, J of each of its segments, which are `step`
// values apart.  A group lies wholly inside the row or outside, where it counts as 0.  Loads of
// a thread's groups stand together, without a branch between them (groups outside
// the row read its last one): loaded and used one group after the other, each waited
// for the one before, and 13 rows of 5003 took 12 us.
template <int V, int N, int J>
struct Groups {
    int place, step, hidden;
    __device__ __forceinline__ int at(int k) const { return place + k / J * step + k % J * (32 * V); }
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

// Sums over the lanes of N values (1, 2, 4 or 8) of each, that of value k in s[0] of lanes
// k * 32 / N on.  The lanes exchange halves of what they have, so 2 values take 5 shuffles as
// one does, and 8 take 9; the order, lanes 16, 8, 4, 2 and 1 apart, is the same for any N.
template <int N>
__device__ __forceinline__ void sum_each(float (&s)[N]) {
    const int lane = threadIdx.x & 31;
    int d = 16;
#pragma unroll
    for (int n = N; n > 1; n /= 2, d /= 2)
#pragma unroll
        for (int j = 0; j < n / 2; ++j) {
            const bool upper = lane & d;
            const float send = upper ? s[j] : s[j + n / 2];
            s[j] = (upper ? s[j + n / 2] : s[j]) + __shfl_xor_sync(0xFFFFFFFFu, send, d);
        }
#pragma unroll
    for (; d >= 1; d /= 2) s[0] += __shfl_xor_sync(0xFFFFFFFFu, s[0], d);
}

// The sum of x(0) .. x(n - 1), n up to 128.
template <typename F>
__device__ __forceinline__ float sum_of(int n, F x) {
    const int lane = threadIdx.x & 31;
    float s = lane < n ? x(lane) : 0.0f;
    if (n > 32) {
        const float a = lane + 32 < n ? x(lane + 32) : 0.0f, b = lane + 64 < n ? x(lane + 64) : 0.0f, c = lane + 96 < n ? x(lane + 96) : 0.0f;
        s = (s + a) + (b + c);
    }
    return warp_sum(s);
}

// A row's mean (of layer norms; else 0) and the sum of squares about it, in one order
// however many threads have the row: its segments are summed apart, and their sums
// together, which every warp does for itself behind the one barrier.  `part`: the row's
// own place in shared memory, [2][segments of the block].
template <int V, int N, int J>
__device__ __forceinline__ void block_moments(const float (&v)[N][V], const Groups<V, N, J>& g, bool layer, float* part, float& mean, float& squares) {
    constexpr int S = N / J;                   // segments of a warp
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int segments = (g.hidden + 255) / 256, segment = lane * S / 32 * warps + warp;       // whose sums the lane will have
    const bool mine = lane % (32 / S) == 0;
    auto count = [&](int i) { return static_cast<float>(max(min(g.hidden - 256 * i, 256), 0)); };
    float s[S];
    mean = 0.0f;
    if (!layer) {
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) s[k / J] = k % J || i ? fmaf(v[k][i], v[k][i], s[k / J]) : __fmul_rn(v[k][i], v[k][i]);
        sum_each(s);
        if (mine) part[segment] = s[0];
        __syncthreads();
        squares = sum_of(segments, [&](int i) { return part[i]; });
        return;
    }
    // about the segment's own mean: a large mean costs no bits
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) s[k / J] = k % J || i ? s[k / J] + v[k][i] : v[k][i];
    sum_each(s);
    const float of_segment = s[0] / fmaxf(count(segment), 1.0f);
#pragma unroll
    for (int j = 0; j < S; ++j) {
        const float m = __shfl_sync(0xFFFFFFFFu, of_segment, j * (32 / S));
        s[j] = 0.0f;
#pragma unroll
        for (int k = j * J; k < j * J + J; ++k)
            if (g.inside(k))
#pragma unroll
                for (int i = 0; i < V; ++i) s[j] = fmaf(v[k][i] - m, v[k][i] - m, s[j]);
    }
    sum_each(s);
    float* part2 = part + S * warps;
    if (mine) {
        part[segment] = of_segment;
        part2[segment] = s[0];
    }
    __syncthreads();
    mean = sum_of(segments, [&](int i) { return __fmul_rn(count(i), part[i]); }) / static_cast<float>(g.hidden);
    // what a segment's mean is off the row's adds its count times the square
    squares = sum_of(segments, [&](int i) {
        const float off = part[i] - mean;
        return fmaf(__fmul_rn(count(i), off), off, part2[i]);
    });
}

// The same of a row that is a warp's, whose split goes by the row's length alone.
template <int V, int N, int J>
__device__ __forceinline__ void warp_moments(const float (&v)[N][V], const Groups<V, N, J>& g, bool layer, float& mean, float& squares) {
    mean = 0.0f;
    if (!layer) {
        squares = 0.0f;
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) squares = fmaf(v[k][i], v[k][i], squares);
        squares = warp_sum(squares);
        return;
    }
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
    mean = m.mean;
    squares = m.m2;
}

// A row's norm, with one barrier (none where the row is a warp's).  (Each rounding is
// written out: no form of the kernel may join two of them that another one does not.)
template <int V, int N, int J, bool kWarpRow>
__device__ __forceinline__ void norm_row(float (&v)[N][V], const Groups<V, N, J>& g, int kind, const float* weight, const float* bias, float eps, float* part) {
    float mean, squares;
    if constexpr (kWarpRow) warp_moments(v, g, kind == PN_NORM_LAYER, mean, squares);
    else block_moments(v, g, kind == PN_NORM_LAYER, part, mean, squares);
    const float inv = 1.0f / sqrtf(fmaf(squares, 1.0f / static_cast<float>(g.hidden), eps));
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) v[k][i] = __fmul_rn(__fsub_rn(v[k][i], mean), inv);
    if (weight) g.with(weight, v, [](float x, float w) { return __fmul_rn(x, w); });
    if (bias) g.with(bias, v, [](float x, float w) { return __fadd_rn(x, w); });
}

// Groups of a thread, a block's threads at most, and blocks to an SM at least: what the registers allow.
template <int kN, int kThreads, int kBlocks>
struct Split {
    static constexpr int N = kN, threads = kThreads, blocks = kBlocks;
};

template <int V, typename S, bool kWarpRow, bool kYF16, bool kRF16>
__global__ void __launch_bounds__(S::threads, S::blocks) norm_kernel(const NormArgs a) {
    constexpr int N = S::N;
    constexpr int J = kOfSegment<V, kWarpRow>, kPart = kWarpRow ? 1 : 2 * (N / J) * (S::threads / 32);
    __shared__ float parts[2 * kPart];                 // a place to each of a row's norms
    const int64_t t = kWarpRow ? static_cast<int64_t>(blockIdx.x) * (kWarpRowThreads / 32) + (threadIdx.x >> 5) : blockIdx.x;
    if (t >= a.tokens) return;                         // (a whole warp, of rows that are warps')
    const int warp = kWarpRow ? 0 : threadIdx.x >> 5, warps = kWarpRow ? 1 : blockDim.x >> 5;
    const Groups<V, N, J> g{(warp * (J * 32) + static_cast<int>(threadIdx.x & 31)) * V, warps * (J * 32) * V, a.hidden};
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
    if (a.post != PN_NORM_NONE) norm_row<V, N, J, kWarpRow>(v, g, a.post, a.post_weight, a.post_bias, a.eps, parts);
    if (kLate && a.residual) g.template load<kRF16>(residual, r);
    if (a.gate) g.with(gate, v, [](float x, float w) { return __fmul_rn(x, w); });
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) r[k][i] = g.inside(k) && a.y ? fmaf(a.scale, v[k][i], r[k][i]) : r[k][i];
    if (a.residual_out)
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (g.inside(k)) store<V>(a.residual_out, t * a.out_stride + g.at(k), kRF16, r[k]);
    if (!a.x) return;
    if (a.pre != PN_NORM_NONE) norm_row<V, N, J, kWarpRow>(r, g, a.pre, a.pre_weight, a.pre_bias, a.eps, parts + kPart);
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
    // Few rows: as many threads to each as there are.  Many: four groups to a thread keep most bytes on their way (up to 5120
    // values without spilling: 8192 rows 85 us, 93 with the registers of 384 threads); above 6144 values eight, of fp32
    // without spilling (96 registers, in microseconds: 4096 rows of 8192 73 against 82 with 64, of 10240 90 and 104), of fp16
    // with two blocks to an SM (fewer bytes to a group: 55 against 61).  Spilled are 56 bytes of a thread's at 5124 to 6144
    // fp32 values, 236 to 280 of fp16 rows above, 260 to 380 of fp32 rows above 20480, as many of odd rows.
    if (!fours)
        return choose<1, false, Split<8, 1024, 1>, Split<16, 512, 2>, Split<32, 512, 1>, Split<32, 640, 1>, Split<64, 512, 1>>(a, many ? 16 : 0, s);
    if (!many) return choose<4, false, Split<2, 1024, 1>, Split<4, 1024, 1>, Split<8, 640, 1>, Split<16, 512, 1>>(a, 0, s);
    const bool halves = (!a.y || a.y_f16) && (!a.residual || a.residual_f16);
    if (halves && a.hidden <= 4 * 8 * 512) return choose<4, false, Split<4, 320, 3>, Split<4, 384, 3>, Split<8, 512, 2>>(a, 0, s);
    return choose<4, false, Split<4, 320, 3>, Split<4, 384, 3>, Split<8, 640, 1>, Split<16, 512, 1>>(a, 0, s);
}

}  // namespace pn
