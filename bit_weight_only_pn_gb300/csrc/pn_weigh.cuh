// pn_weigh.cuh -- what the kernels of the weight that cached tokens gather share.
#pragma once

#include <cstdint>

#include "pn_attn.cuh"

namespace pn {

struct WeighParams {
    WeighArgs a;
    KvCache cache;
    int group;                 // query heads per key/value head
    float scale_log2;          // scale * log2 e
    float scale_rest;          // what that left of it, relative to it
    uint64_t timeout_ns;
    int stall;                 // testing aid: see pn_set_test_stall
    uint32_t* status;          // may be null
};

// A row's lse as the exponent's argument takes it.  exp2(x f - lse log2 e), with x f
// and lse log2 e some tens, would carry the roundings of f and of lse log2 e in all
// of the row's probabilities (2^-20 each).  So the argument gets a multiple of 2^-6,
// which a sum with x f takes up without a rounding before its own, and what is left,
// with f's rounding where x = lse, becomes a factor near 1 of the row's probabilities.
struct LogSum {
    float less, factor;
};
__device__ __forceinline__ LogSum log_sum_of(float lse, float scale_rest) {
    if (fabsf(lse) == INFINITY) return {-INFINITY, 0.0f};              // a row that gives nothing
    constexpr float kLog2e = 1.44269502f, kLog2eRest = 1.92596299e-8f;       // log2 e in two parts
    const float hi = lse * kLog2e, lo = fmaf(lse, kLog2e, -hi) + lse * kLog2eRest;
    const float near = rintf(hi * 64.0f) * 0.015625f;
    // 2^u for |u| a little above 2^-7, by its series
    const float u = ((near - hi) - lo + hi * scale_rest) * 0.693147181f;
    return {-near, fabsf(u) < 1.0f ? fmaf(u, fmaf(u, fmaf(u, fmaf(u, 0.0416666667f, 0.166666667f), 0.5f), 1.0f), 1.0f) : 1.0f};
}

// The same rounded to one number (2^-24 of it off), for sums of many rows, where these
// roundings meet: a second number for each would cost more than it gives.
__device__ __forceinline__ float less_of(float lse, float scale_rest) {
    if (fabsf(lse) == INFINITY) return -INFINITY;
    constexpr float kLog2e = 1.44269502f, kLog2eRest = 1.92596299e-8f;
    const float hi = lse * kLog2e, lo = fmaf(lse, kLog2e, -hi) + lse * kLog2eRest;
    return fmaf(hi, scale_rest, -lo) - hi;
}

struct WeighRequest {
    int n, q0, pos0, len, rows;
    __device__ __forceinline__ void read(const WeighParams& P, int b) {
        const WeighArgs& a = P.a;
        const int T = static_cast<int>(a.tokens);
        q0 = min(max(a.starts[b], 0), T);
        n = min(min(max(a.starts[b + 1], q0), T) - q0, a.max_queries);
        const int64_t room = static_cast<int64_t>(a.max_pages) << P.cache.page_shift;
        len = static_cast<int>(min(static_cast<int64_t>(max(a.lens[b], 0)), room));
        pos0 = len - n;
        rows = n * P.group;
    }
};

// Units of a head's kTokens tokens that a request has: none without queries.
template <int kTokens>
__device__ __forceinline__ int units_of(const WeighRequest& r) { return r.n > 0 ? (r.len + kTokens - 1) / kTokens : 0; }

// scan[i]: units of all heads before thread i's requests, of which it has as many as
// is returned; scan[kThreads] all of them.
template <int kTokens, int kThreads>
__device__ __forceinline__ int scan_units(const WeighParams& P, uint64_t* scan, uint64_t* warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, each = (P.a.batch + kThreads - 1) / kThreads;
    const int b0 = min(static_cast<int>(threadIdx.x) * each, P.a.batch), b1 = min(b0 + each, P.a.batch);
    uint64_t mine = 0;
    for (int b = b0; b < b1; ++b) {
        WeighRequest r;
        r.read(P, b);
        mine += static_cast<uint64_t>(units_of<kTokens>(r)) * P.cache.heads;
    }
    uint64_t in = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint64_t o = __shfl_up_sync(0xFFFFFFFFu, in, d);
        if (lane >= d) in += o;
    }
    if (lane == 31) warp_sums[warp] = in;
    __syncthreads();
    uint64_t at = in - mine;
    for (int w = 0; w < warp; ++w) at += warp_sums[w];
    scan[threadIdx.x] = at;
    if (threadIdx.x == kThreads - 1) scan[kThreads] = at + mine;
    __syncthreads();
    return each;
}

// Unit u (there is one): its request, head and place among the head's units.
template <int kTokens, int kThreads>
__device__ __forceinline__ void locate(const WeighParams& P, const uint64_t* scan, int each, uint64_t u, WeighRequest& r, int& b, int& h, int& unit) {
    int lo = 0, hi = kThreads - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (scan[mid] <= u) lo = mid;
        else hi = mid - 1;
    }
    b = lo * each;
    u -= scan[lo];
    for (;; ++b) {
        r.read(P, b);
        const uint64_t units = static_cast<uint64_t>(units_of<kTokens>(r)) * P.cache.heads;
        if (u < units) break;
        u -= units;
    }
    const uint64_t of_head = static_cast<uint64_t>(units_of<kTokens>(r));
    h = static_cast<int>(u / of_head);
    unit = static_cast<int>(u - h * of_head);
}

// Query rows to a key/value head up to which a warp takes its tokens through all of
// them (weigh_few_kernel); a warp's share of shared memory holds no more.  Above, where
// heads allow it, the kernel for many rows (pn_weigh_tc.cu).  Microseconds here, there; 64
// ragged requests to 16384 tokens, 4 key/value heads:
//   of 64:  64 rows 89, 153; 96 rows 125, 171
//   of 128: 48 rows 104, 172; 64 rows 144, 176
//   of 256: 12 rows 90, 204; 32 rows 175, 196
// One request of 8192 and 96, 64, 32 rows of 64, 128, 256: 13.7, 12.0; 13.1, 12.2; 12.7, 12.9.
constexpr int weigh_few_rows(int head_dim) { return head_dim == 64 ? 96 : head_dim == 128 ? 64 : 32; }
bool weigh_tc_takes(const WeighArgs& a, const KvGeometry& g);
cudaError_t launch_weigh_tc(const WeighParams& P, int num_sms, cudaStream_t s);

}  // namespace pn
