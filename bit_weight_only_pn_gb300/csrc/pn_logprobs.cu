// pn_logprobs.cu -- log probabilities of given tokens, entropy and the top
// alternatives of rows of logits.
//
// With x = scale * logit, m the row's largest logit, d = logit - m and e =
// exp(scale d):  S = sum e,  T = sum e d,
//   ln p(token) = scale d - ln S,   entropy = ln S - scale T / S
// (both terms of the entropy are positive or zero, so nothing cancels).
//
// One pass over memory.  A cluster of 1 to 8 thread blocks has a row, each block a
// contiguous part of it; a thread keeps a running m, S and T for 32 values at a
// time, and the place of its largest.
//
// Top k (at most 32): by the 64-bit number (order of the logit, ~index), so there
// are no ties and the lowest index wins.  The k largest of a block's 256 thread
// maxima bound the k-th largest of its part from below, the largest of the
// cluster's bounds that of the row.  A value of the top k is at or above the bound,
// and so is its thread's maximum: only the (at most k) threads of a block whose
// maximum passes it have their values looked at again, from L2, by a warp each,
// which collects in a sorted list, a lane to an entry, what passes; that is little
// more than k values in all, and never more than 32 to a warp.  The first block
// ranks them.
#include <cooperative_groups.h>
#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "pn_device.cuh"
#include "pn_internal.h"

namespace cg = cooperative_groups;

namespace pn {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMostCluster = 8;
constexpr int kMostEntries = kMostCluster * kWarps * 32;
constexpr float kHuge = 1.7e38f;               // differences of numbers up to it are finite

using Key = unsigned long long;

// The order of logits as that of whole numbers, the lower index first where they
// are equal; 0 for NaN and what is not above -kHuge, which have no probability.
__device__ __forceinline__ Key key_of(float x, uint32_t index) {
    if (!(x > -kHuge)) return 0;
    const uint32_t u = __float_as_uint(x + 0.0f);      // -0 is 0
    return (static_cast<Key>(u & 0x80000000u ? ~u : u | 0x80000000u) << 32) | (0xFFFFFFFFu - index);
}
__device__ __forceinline__ uint32_t index_of(Key k) { return 0xFFFFFFFFu - static_cast<uint32_t>(k); }
__device__ __forceinline__ float logit_of(Key k) {
    const uint32_t u = static_cast<uint32_t>(k >> 32);
    return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}

// NaN and -inf as -kHuge (they count where nothing else is there, and what they
// gave is dropped when something is), +inf as kHuge.
__device__ __forceinline__ float bounded(float x) { return fminf(fmaxf(x, -kHuge), kHuge); }

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Sums relative to a largest value.
struct Sums {
    float m, s, t;
    // to the larger reference `to`
    __device__ __forceinline__ void move(float to, float scale_log2) {
        const float by = m - to, f = exp2_fast(by * scale_log2);
        t = f == 0.0f ? 0.0f : f * fmaf(s, by, t);
        s *= f;
        m = to;
    }
    __device__ __forceinline__ void join(Sums o, float scale_log2) {
        const float to = fmaxf(m, o.m);
        move(to, scale_log2);
        o.move(to, scale_log2);
        s += o.s;
        t += o.t;
    }
};

// 16 bytes of a row: value i of vector v is the row's element v * kVec - skew + i.
template <typename T>
struct RowOf {
    static constexpr int kVec = 16 / sizeof(T);
    const T* p;                // aligned to 16 bytes, `skew` elements before the row
    int skew, vocab;
    __device__ __forceinline__ void load(int v, float (&x)[kVec]) const {
        const int at = v * kVec - skew;
        if (at >= 0 && at + kVec <= vocab) {
            if constexpr (kVec == 4) {
                const float4 w = __ldcg(reinterpret_cast<const float4*>(p) + v);
                x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w;
            } else {
                const uint4 w = __ldcg(reinterpret_cast<const uint4*>(p) + v);
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[2 * i] = half_bits_to_float(u[i] & 0xFFFFu);
                    x[2 * i + 1] = half_bits_to_float(u[i] >> 16);
                }
            }
        } else {                               // the row's ends: nothing outside it is read
#pragma unroll
            for (int i = 0; i < kVec; ++i) x[i] = at + i >= 0 && at + i < vocab ? static_cast<float>(p[v * kVec + i]) : -INFINITY;
        }
    }
};

// Lane i holds the i-th largest of a list; `add` joins it (all lanes the same).
__device__ __forceinline__ Key insert(Key mine, Key add) {
    const int lane = threadIdx.x & 31;
    const Key above = __shfl_up_sync(0xFFFFFFFFu, mine, 1);
    const int at = __popc(__ballot_sync(0xFFFFFFFFu, mine > add));
    return lane < at ? mine : lane == at ? add : above;
}

template <typename T, bool kTop>
__global__ void __launch_bounds__(kThreads, 4) logprobs_kernel(const LogprobsArgs a) {
    using Row = RowOf<T>;
    constexpr int kVec = Row::kVec, kUnroll = 32 / kVec;
    cg::cluster_group cluster = cg::this_cluster();
    __shared__ Sums warp_sums[kWarps], block_sums;
    __shared__ Key lists[kTop ? kWarps * 32 : 1];      // the warps' thread maxima in order
    __shared__ Key winners[32];                        // the largest thread maxima
    __shared__ Key bound;                              // the k-th of them
    __shared__ uint32_t entries;                       // (first block of a cluster)
    __shared__ Key entry[kTop ? kMostEntries : 1];
    const int parts = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t r = blockIdx.x / parts;
    const T* begin = static_cast<const T*>(a.logits) + r * a.stride;
    Row row;
    row.skew = static_cast<int>((reinterpret_cast<uintptr_t>(begin) & 15) / sizeof(T));
    row.p = begin - row.skew;
    row.vocab = a.vocab;
    const int vectors = (row.skew + a.vocab + kVec - 1) / kVec;
    const int v0 = static_cast<int>(static_cast<int64_t>(vectors) * rank / parts), v1 = static_cast<int>(static_cast<int64_t>(vectors) * (rank + 1) / parts);
    const float c = a.scale * 1.4426950408889634f;

    if (kTop && threadIdx.x < 32) {
        winners[threadIdx.x] = 0;
        if (threadIdx.x == 0) {
            bound = 0;
            entries = 0;
        }
    }
    Sums mine{-kHuge, 0.0f, 0.0f};
    float best = -INFINITY;
    uint32_t best_at = 0;
    for (int v = v0 + static_cast<int>(threadIdx.x); v < v1; v += kThreads * kUnroll) {
        float x[kUnroll][kVec];
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
            if (v + j * kThreads < v1) row.load(v + j * kThreads, x[j]);
            else
#pragma unroll
                for (int i = 0; i < kVec; ++i) x[j][i] = -INFINITY;
        }
        float most = x[0][0];
#pragma unroll
        for (int j = 0; j < kUnroll; ++j)
#pragma unroll
            for (int i = 0; i < kVec; ++i) most = fmaxf(most, x[j][i]);
        if (kTop && most > best) {             // (NaN: fmaxf passes over it)
            best = most;
#pragma unroll
            for (int j = kUnroll - 1; j >= 0; --j)
#pragma unroll
                for (int i = kVec - 1; i >= 0; --i)
                    if (x[j][i] == most) best_at = static_cast<uint32_t>((v + j * kThreads) * kVec - row.skew + i);
        }
        most = bounded(most);
        if (most > mine.m) mine.move(most, c);
        const float less = -mine.m;
        float s[2] = {0.0f, 0.0f}, t[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < kUnroll; ++j)
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const float d = bounded(x[j][i]) + less, e = exp2_fast(d * c);
                s[i & 1] += e;
                t[i & 1] = fmaf(e, d, t[i & 1]);
            }
        mine.s += s[0] + s[1];
        mine.t += t[0] + t[1];
    }
    Sums all = mine;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1)
        all.join(Sums{__shfl_xor_sync(0xFFFFFFFFu, all.m, d), __shfl_xor_sync(0xFFFFFFFFu, all.s, d), __shfl_xor_sync(0xFFFFFFFFu, all.t, d)}, c);
    if (lane == 0) warp_sums[warp] = all;
    Key key = 0;
    if constexpr (kTop) {
        // the warp's thread maxima in order, the largest in lane 0
        key = key_of(best, best_at);
#pragma unroll
        for (int size = 2; size <= 32; size *= 2)
#pragma unroll
            for (int d = size / 2; d >= 1; d /= 2) {
                const Key o = __shfl_xor_sync(0xFFFFFFFFu, key, d);
                const bool larger = ((lane & size) == 0 || size == 32) == ((lane & d) == 0);
                key = larger == (key > o) ? key : o;
            }
        lists[warp * 32 + lane] = key;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        all = warp_sums[0];
        for (int w = 1; w < kWarps; ++w) all.join(warp_sums[w], c);
        block_sums = all;
    }
    if constexpr (kTop) {
        // its place among the block's: how many of each other warp's list are larger
        if (key != 0) {
            int place = lane;
#pragma unroll
            for (int o = 1; o < kWarps; ++o) {
                const Key* list = lists + (warp + o) % kWarps * 32;
                int n = 0;
#pragma unroll
                for (int step = 16; step >= 1; step /= 2) n += list[n + step - 1] > key ? step : 0;
                place += n + (n == 31 && list[31] > key);
            }
            if (place < a.top) winners[place] = key;
            if (place == a.top - 1) bound = key;
        }
    }
    cluster.sync();
    // the row's sums, in the blocks' order, and its bound
    Key least = 1;
    all = *cluster.map_shared_rank(&block_sums, 0);
    for (int o = 1; o < parts; ++o) all.join(*cluster.map_shared_rank(&block_sums, o), c);
    const bool none = all.m == -kHuge;         // no token at all
    const float log_sum = logf(all.s);
    if constexpr (kTop) {
        for (int o = 0; o < parts; ++o) {
            const Key b = *cluster.map_shared_rank(&bound, o);
            least = b > least ? b : least;
        }
    }
    auto log_p = [&](float logit) {
        return none || !(logit > -kHuge) ? -INFINITY : fmaf(fminf(logit, kHuge) - all.m, a.scale, -log_sum);
    };
    if (rank == 0) {
        for (int i = threadIdx.x; i < a.count; i += kThreads) {
            const int token = a.tokens[r * a.count + i];
            a.logprobs[r * a.count + i] = token >= 0 && token < a.vocab ? log_p(static_cast<float>(begin[token])) : -INFINITY;
        }
        if (threadIdx.x == 0 && a.entropy) a.entropy[r] = none ? 0.0f : fmaxf(fmaf(-a.scale, all.t / all.s, log_sum), 0.0f);
    }
    if constexpr (kTop) {
        // a winner to a warp: its thread's values that reach the bound
        Key list = 0;
        for (int w = warp; w < a.top; w += kWarps) {
            const Key winner = winners[w];
            if (winner < least) break;                 // so are those behind it
            const int thread = ((static_cast<int>(index_of(winner)) + row.skew) / kVec - v0) % kThreads;
            for (int first = v0 + thread; first < v1; first += 32 * kThreads) {
                const int v = first + lane * kThreads;
                float x[kVec];
                if (v < v1) row.load(v, x);
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    const Key k = v < v1 ? key_of(x[i], static_cast<uint32_t>(v * kVec - row.skew + i)) : 0;
                    for (uint32_t in = __ballot_sync(0xFFFFFFFFu, k >= least); in; in &= in - 1)
                        list = insert(list, __shfl_sync(0xFFFFFFFFu, k, __ffs(in) - 1));
                }
            }
        }
        uint32_t* counter = cluster.map_shared_rank(&entries, 0);
        Key* to = cluster.map_shared_rank(entry, 0);
        const int have = __popc(__ballot_sync(0xFFFFFFFFu, list != 0));
        uint32_t at = 0;
        if (lane == 0 && have) at = atomicAdd(counter, static_cast<uint32_t>(have));
        at = __shfl_sync(0xFFFFFFFFu, at, 0);
        if (lane < have) to[at + lane] = list;
        cluster.sync();
        if (rank != 0) return;
        const int n = static_cast<int>(entries);
        int32_t* tokens = a.top_tokens + r * a.top;
        float* values = a.top_logprobs + r * a.top;
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const Key k = entry[i];
            int place = 0;
            for (int o = 0; o < n; ++o) place += entry[o] > k;
            if (place < a.top) {
                tokens[place] = static_cast<int32_t>(index_of(k));
                values[place] = log_p(logit_of(k));
            }
        }
        for (int i = n + threadIdx.x; i < a.top; i += kThreads) {      // fewer tokens than that
            tokens[i] = -1;
            values[i] = -INFINITY;
        }
    } else {
        cluster.sync();                        // no block leaves while its sums may still be read
    }
}

template <typename T, bool kTop>
cudaError_t launch(const LogprobsArgs& a, int parts, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.rows * parts));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = parts;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<T, kTop>, a);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobsArgs& a, int num_sms, cudaStream_t s) {
    // blocks to a row: until the GPU is full, none with less than 2048 values
    int parts = 1;
    while (parts < kMostCluster && a.rows * parts * 2 <= static_cast<int64_t>(num_sms) * 4 && a.vocab / (parts * 2) >= 2048) parts *= 2;
    if (a.f16) return a.top ? launch<__half, true>(a, parts, s) : launch<__half, false>(a, parts, s);
    return a.top ? launch<float, true>(a, parts, s) : launch<float, false>(a, parts, s);
}

}  // namespace pn
