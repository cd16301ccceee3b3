// pn_verify.cu -- drafted tokens against the target's probabilities, with given
// random numbers, and the token that follows the accepted ones.
//
// Draft i with token x is accepted while u_i q_i(x) < p_i(x).  The next token
// is drawn by inverting the cumulated weights of one row: max(p - q, 0) of the
// row of the first draft turned down, or p of the row behind the last draft.
// Weights are held as whole multiples of 2^-42 in 64 bits, so their sums do
// not depend on the order in which they are added and the drawn token is the
// same however the row is split.
//
// Bound by the read of that one row (two with q): a cluster of thread blocks
// shares it.  Each warp sums a contiguous part; block sums meet through
// distributed shared memory; the block that holds the threshold splits the
// warp's part that holds it over all its threads (a second read, from L2), and
// the one thread whose few weights hold it walks them.  (With the part left to
// its own warp that second read was a third of the time.)
#include <cooperative_groups.h>
#include <cstdint>

#include <cuda_runtime.h>

#include "pn_internal.h"

namespace cg = cooperative_groups;

namespace pn {
namespace {

constexpr int kVerifyThreads = 256;             // four blocks to an SM: 64 requests of 8 blocks run at once
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyCluster = 8;

// A weight in multiples of 2^-42: nothing for NaN and below zero, at most 1.
__device__ __forceinline__ int64_t whole(float w) {
    return w > 0.0f ? __float2ll_rn(__fmul_rn(fminf(w, 1.0f), 4398046511104.0f)) : 0;
}

struct Row {
    const float* p;
    const float* q;            // null: no draft row
    int skip;                  // token whose weight is nothing (a certain draft turned down), -1 none
};

__device__ __forceinline__ int64_t weight(const Row& r, int j) {
    const float p = r.p[j];
    if (r.q) return whole(__fsub_rn(p, r.q[j]));
    return j == r.skip ? 0 : whole(p);
}

// Weights are summed without 64-bit conversions (a third of the time: 64 requests of
// 151936 tokens 20 us, with them 30): with t =
// 2^21 w, a = rint(t) by adding 1.5 2^23 and the rest t - a, which is exact, times
// 2^21 rounded the same way, whole(w) = 2^21 a + rint(2^21 (t - a)) -- the first
// part is even, so ties go as in one rounding -- and both parts of up to 512
// weights add up in 32 bits.
struct Sum {
    uint32_t high = 0, low = 0;
    __device__ __forceinline__ void add(float w) {
        constexpr float kMagic = 12582912.0f;      // 1.5 2^23
        const float t = __fmul_rn(fminf(fmaxf(w, 0.0f), 1.0f), 2097152.0f);   // (NaN: 0)
        const float a = __fadd_rn(t, kMagic);
        const float b = __fmaf_rn(__fsub_rn(t, __fsub_rn(a, kMagic)), 2097152.0f, kMagic);
        high += __float_as_uint(a) - 0x4B400000u;
        low += __float_as_uint(b) - 0x4B400000u;
    }
    __device__ __forceinline__ int64_t value() const {
        return (static_cast<int64_t>(static_cast<int32_t>(high)) << 21) + static_cast<int32_t>(low);
    }
};

// The sum of the weights j .. j + 3 for j = j0, j0 + step, ... below j1; rows 16-byte aligned, all multiples of 4.
__device__ __forceinline__ int64_t sum_fours(const Row& r, int j0, int j1, int step) {
    Sum s;
    if (r.q) {
#pragma unroll 4
        for (int j = j0; j < j1; j += step) {
            const float4 p = __ldcg(reinterpret_cast<const float4*>(r.p + j)), q = __ldcg(reinterpret_cast<const float4*>(r.q + j));
            s.add(__fsub_rn(p.x, q.x));
            s.add(__fsub_rn(p.y, q.y));
            s.add(__fsub_rn(p.z, q.z));
            s.add(__fsub_rn(p.w, q.w));
        }
    } else {
#pragma unroll 8
        for (int j = j0; j < j1; j += step) {
            const float4 p = __ldcg(reinterpret_cast<const float4*>(r.p + j));
            s.add(j == r.skip ? 0.0f : p.x);
            s.add(j + 1 == r.skip ? 0.0f : p.y);
            s.add(j + 2 == r.skip ? 0.0f : p.z);
            s.add(j + 3 == r.skip ? 0.0f : p.w);
        }
    }
    return s.value();
}

__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    return v;
}

__global__ void __launch_bounds__(kVerifyThreads, 4) verify_kernel(const VerifyArgs a) {
    cg::cluster_group cluster = cg::this_cluster();
    __shared__ int64_t sums[kVerifyWarps];
    __shared__ int64_t block_total[2];
    const int b = blockIdx.x / kVerifyCluster, rank = blockIdx.x % kVerifyCluster;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int K = a.drafts, V = a.vocab;
    const int count = a.counts ? min(max(a.counts[b], 0), K) : K;
    const float* target = a.target + static_cast<int64_t>(b) * (K + 1) * a.target_stride;
    const float* draft = a.draft ? a.draft + static_cast<int64_t>(b) * K * a.draft_stride : nullptr;

    // every warp finds the number of accepted drafts (lane i tests draft i)
    int token = -1;
    bool ok = false;
    if (lane < count) {
        token = a.tokens[static_cast<int64_t>(b) * K + lane];
        if (token >= 0 && token < V) {
            const float p = target[lane * a.target_stride + token];
            const float q = draft ? draft[lane * a.draft_stride + token] : 1.0f;
            ok = __fmul_rn(a.uniforms[static_cast<int64_t>(b) * (K + 1) + lane], q) < p;
        }
    }
    const int accepted = min(__ffs(~__ballot_sync(0xFFFFFFFFu, ok)) - 1, count);
    const bool turned = accepted < count;
    Row row{target + static_cast<int64_t>(accepted) * a.target_stride, nullptr, -1};
    if (turned) {
        if (draft) row.q = draft + static_cast<int64_t>(accepted) * a.draft_stride;
        else row.skip = __shfl_sync(0xFFFFFFFFu, token, accepted & 31);
    }
    // contiguous parts: V over the cluster's warps, in multiples of 32
    constexpr int kParts = kVerifyCluster * kVerifyWarps;
    const int each = (V + kParts * 32 - 1) / (kParts * 32) * 32;
    const int j0 = min((rank * kVerifyWarps + warp) * each, V), j1 = min(j0 + each, V);

    int32_t* out = a.out + static_cast<int64_t>(b) * (K + 1);
    if (rank == 0 && warp == 0) {
        if (lane == 0) a.accepted[b] = accepted;
        for (int i = lane; i <= K; i += 32)
            if (i != accepted) out[i] = i < accepted ? a.tokens[static_cast<int64_t>(b) * K + i] : -1;
    }
    const float u = a.uniforms[static_cast<int64_t>(b) * (K + 1) + K];
    for (int pass = 0; pass < 2; ++pass) {
        int64_t s = 0;
        // fours where both rows lie for it (vocab a multiple of 4, so the parts are too)
        const bool fours = V % 4 == 0 && ((reinterpret_cast<uintptr_t>(row.p) | reinterpret_cast<uintptr_t>(row.q)) & 15) == 0;
        if (fours) {
            s = sum_fours(row, j0 + 4 * lane, j1, 128);
        } else {
#pragma unroll 8
            for (int j = j0 + lane; j < j1; j += 32) s += weight(row, j);
        }
        s = warp_sum(s);
        if (lane == 0) sums[warp] = s;
        __syncthreads();
        if (threadIdx.x == 0) {
            int64_t t = 0;
            for (int w = 0; w < kVerifyWarps; ++w) t += sums[w];
            block_total[pass] = t;
        }
        cluster.sync();
        int64_t before = 0, total = 0;
#pragma unroll
        for (int r = 0; r < kVerifyCluster; ++r) {
            const int64_t t = *cluster.map_shared_rank(&block_total[pass], r);
            before += r < rank ? t : 0;
            total += t;
        }
        if (total == 0 && pass == 0 && turned) {   // nothing left of the row: draw from the target itself
            row.q = nullptr;
            row.skip = -1;
            __syncthreads();                       // sums are written again
            continue;
        }
        if (total == 0) {
            if (rank == 0 && threadIdx.x == 0) out[accepted] = -1;
            break;
        }
        int64_t at = __double2ll_rd(static_cast<double>(u) * static_cast<double>(total));
        at = min(max(at, static_cast<int64_t>(0)), total - 1);
        if (at < before || at >= before + block_total[pass]) break;      // another block's
        int owner = 0;
        while (at >= before + sums[owner]) before += sums[owner++];
        const int o0 = min((rank * kVerifyWarps + owner) * each, V), o1 = min(o0 + each, V);
        const int piece = (o1 - o0 + 4 * kVerifyThreads - 1) / (4 * kVerifyThreads) * 4;
        const int k0 = min(o0 + static_cast<int>(threadIdx.x) * piece, o1), k1 = min(k0 + piece, o1);
        int64_t mine = 0;
        if (fours) {
            mine = sum_fours(row, k0, k1, 4);
        } else {
            for (int j = k0; j < k1; ++j) mine += weight(row, j);
        }
        int64_t upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t o = __shfl_up_sync(0xFFFFFFFFu, upto, d);
            if (lane >= d) upto += o;
        }
        __syncthreads();                           // everyone has read sums
        if (lane == 31) sums[warp] = upto;
        __syncthreads();
        before += upto - mine;
        for (int w = 0; w < warp; ++w) before += sums[w];
        if (at >= before && at < before + mine) {
            int j = k0;
            for (; j < k1 - 1; ++j) {
                before += weight(row, j);
                if (before > at) break;
            }
            out[accepted] = j;
        }
        break;
    }
    cluster.sync();                                // no block leaves while its sums may still be read
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.batch) * kVerifyCluster);
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kVerifyCluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, verify_kernel, a);
}

}  // namespace pn
