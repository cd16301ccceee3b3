// pn_kv.cu -- what stands around the cache: pages and slots for a step's
// tokens, the query/key norms and rotation with the write into the 4-bit
// cache, and the cache read back.
#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "pn_device.cuh"
#include "pn_internal.h"
#include "pn_kv.cuh"

namespace pn {
namespace {

// ------------------------------------------------------------------- plan --
//
// Three prefix sums over the requests decide everything: tokens (starts),
// pages taken (a request that would pass the free pages takes none) and pages
// given back.  Every block scans all requests by itself (a few KB from L2)
// instead of waiting for another block, keeps the result in shared memory and
// then fills its share of the maps and of the table; block 0 writes the
// per-request outputs.  Nothing is read that any block writes: taken pages
// come from the ring's [head, tail), given ones go behind its tail, table
// entries are read below `held` and written from it on.

constexpr int kPlanThreads = 1024;

struct Scan3 {
    int64_t tok, need, back;
};
__device__ __forceinline__ Scan3 add3(const Scan3& a, const Scan3& b) {
    return {a.tok + b.tok, a.need + b.need, a.back + b.back};
}
__device__ __forceinline__ Scan3 shfl_up3(const Scan3& v, int d) {
    return {__shfl_up_sync(0xFFFFFFFFu, v.tok, d), __shfl_up_sync(0xFFFFFFFFu, v.need, d),
            __shfl_up_sync(0xFFFFFFFFu, v.back, d)};
}

// Exclusive prefix over the block's threads; *total gets the sum.  `part`
// holds one entry per warp; the caller synchronises before part is reused.
__device__ Scan3 block_scan(Scan3 v, Scan3* part, Scan3* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Scan3 in = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const Scan3 o = shfl_up3(in, d);
        if (lane >= d) in = add3(in, o);
    }
    if (lane == 31) part[warp] = in;
    __syncthreads();
    if (warp == 0) {
        Scan3 w = lane < static_cast<int>(blockDim.x >> 5) ? part[lane] : Scan3{0, 0, 0};
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const Scan3 o = shfl_up3(w, d);
            if (lane >= d) w = add3(w, o);
        }
        part[lane] = w;
    }
    __syncthreads();
    *total = part[(blockDim.x >> 5) - 1];
    const Scan3 ex = {in.tok - v.tok, in.need - v.need, in.back - v.back};
    return warp ? add3(part[warp - 1], ex) : ex;
}

__device__ __forceinline__ int64_t wrap(int64_t i, int64_t n) {
    const int64_t r = i % n;
    return r < 0 ? r + n : r;
}

struct PlanParams {
    KvPlanArgs a;
    int shift;                 // log2(page_size)
    int each;                  // requests per thread of the scan
};

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanParams P) {
    extern __shared__ int plan_smem[];
    __shared__ Scan3 part[32];
    const KvPlanArgs& a = P.a;
    int* starts = plan_smem;                   // [batch + 1]
    int* first = plan_smem + a.batch + 1;      // [batch]: >= 0 the request's first page of the ring, -1 refused, <= -2 given back
    const int tid = threadIdx.x;
    const int b0 = min(tid * P.each, a.batch), b1 = min(b0 + P.each, a.batch);
    // whatever the ring holds, no index leaves it
    const int64_t ring_head = a.ring[0], tail = a.ring[1];
    const int64_t avail = min(max(tail - ring_head, static_cast<int64_t>(0)), a.pages);
    const int64_t head = wrap(ring_head, a.pages);
    auto free_page = [&](int64_t i) -> int32_t {          // i < avail <= pages
        const int64_t at = head + i;
        return a.free_pages[at >= a.pages ? at - a.pages : at];
    };

    // tokens and pages given back
    Scan3 mine{0, 0, 0}, total;
    for (int b = b0; b < b1; ++b) {
        const int add = a.add[b];
        if (add < 0) mine.back += min(max(a.held[b], 0), a.max_pages);
        else mine.tok += add;
    }
    const Scan3 at = block_scan(mine, part, &total);
    const int64_t tokens = total.tok, given = total.back;
    __syncthreads();
    // pages taken by the requests that fit the table and the maps
    auto need_of = [&](int b, int64_t end) -> int64_t {   // -1: does not fit
        const int64_t want = (static_cast<int64_t>(max(a.lens[b], 0)) + a.add[b] + a.page_size - 1) >> P.shift;
        if (want > a.max_pages || end > a.capacity) return -1;
        return max(want - min(max(a.held[b], 0), a.max_pages), static_cast<int64_t>(0));
    };
    Scan3 need{0, 0, 0};
    int64_t tok = at.tok;
    for (int b = b0; b < b1; ++b) {
        if (a.add[b] < 0) continue;
        tok += a.add[b];
        need.need += max(need_of(b, tok), static_cast<int64_t>(0));
    }
    const Scan3 before = block_scan(need, part, &total);
    tok = at.tok;
    int64_t taken = before.need, back = at.back;
    int refused = 0;
    int64_t served_need = 0;
    const bool writer = blockIdx.x == 0;
    for (int b = b0; b < b1; ++b) {
        const int add = a.add[b];
        const int start = static_cast<int>(min(tok, static_cast<int64_t>(INT32_MAX)));
        starts[b] = start;
        const int held = min(max(a.held[b], 0), a.max_pages), len = max(a.lens[b], 0);
        int lens_out = 0, held_out = 0;
        if (add < 0) {
            first[b] = static_cast<int>(-2 - back);
            back += held;
        } else {
            tok += add;
            const int64_t n = need_of(b, tok);
            const bool ok = n == 0 || (n > 0 && taken + n <= avail);
            first[b] = ok ? static_cast<int>(taken) : -1;
            taken += max(n, static_cast<int64_t>(0));
            served_need += ok ? n : 0;
            refused += !ok;
            lens_out = ok ? len + add : len;
            held_out = held + (ok ? static_cast<int>(n) : 0);
        }
        if (writer) {
            a.starts[b] = start;
            a.lens_out[b] = lens_out;
            a.held_out[b] = held_out;
        }
    }
    __syncthreads();                           // part is free again; starts and first are complete
    if (tid == 0) starts[a.batch] = static_cast<int>(min(tokens, static_cast<int64_t>(INT32_MAX)));
    const Scan3 unused = block_scan(Scan3{refused, served_need, 0}, part, &total);
    (void)unused;
    if (writer && tid == 0) {
        a.starts[a.batch] = starts[a.batch];
        a.ring_out[0] = ring_head + total.need;
        a.ring_out[1] = tail + given;
        a.refused[0] = static_cast<int>(total.tok);
    }

    // table entries and returned pages: one warp per request
    const int warps = blockDim.x >> 5;
    for (int b = blockIdx.x * warps + (tid >> 5); b < a.batch; b += gridDim.x * warps) {
        const int f = first[b];
        if (f == -1) continue;
        const int held = min(max(a.held[b], 0), a.max_pages);
        int32_t* row = a.table + static_cast<int64_t>(b) * a.table_stride;
        if (f >= 0) {
            const int64_t want = (static_cast<int64_t>(max(a.lens[b], 0)) + a.add[b] + a.page_size - 1) >> P.shift;
            for (int64_t i = held + (tid & 31); i < want; i += 32) row[i] = free_page(f + i - held);
        } else {
            const int64_t to = tail + (-2 - static_cast<int64_t>(f));
            for (int i = tid & 31; i < held; i += 32) a.free_pages[wrap(to + i, a.pages)] = row[i];
        }
    }

    // slot maps: the request of a token by binary search in starts
    const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + tid; t < a.capacity; t += stride) {
        int64_t slot = -1;
        int pos = -1, req = -1;
        if (t < tokens) {
            int lo = 0, hi = a.batch - 1;      // the last request whose start is <= t (those that add nothing share the next one's)
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (starts[mid] <= t) lo = mid;
                else hi = mid - 1;
            }
            req = lo;
            if (first[lo] >= 0) {
                pos = max(a.lens[lo], 0) + static_cast<int>(t - starts[lo]);
                const int held = min(max(a.held[lo], 0), a.max_pages);
                const int pg = pos >> P.shift;
                const int32_t page = pg < held ? a.table[lo * a.table_stride + pg]
                                               : free_page(static_cast<int64_t>(first[lo]) + pg - held);
                slot = (static_cast<int64_t>(page) << P.shift) + (pos & (a.page_size - 1));
            }
        }
        a.slots[t] = slot;
        a.positions[t] = pos;
        a.requests[t] = req;
    }
}

// ----------------------------------------------------------------- append --
//
// One warp per head row.  Lane l owns the D / 32 consecutive values from
// l * D / 32.  The arithmetic is fixed, every operation rounded by itself, so
// codes are the same whatever computes them: squares added pairwise (the upper
// half of the row to the lower, until one sum is left: lane exchanges 16 .. 1,
// then within the lane), times 1 / D, plus eps, 1 / sqrt; x * that * weight;
// rotation with separate products and sums; pn4t's rule per group of 64.
// Bound by memory: each value is read once and written once.

template <int E>
__device__ __forceinline__ void load_row(const void* p, int64_t at, bool f16, bool wide, float (&x)[E]) {
    if (f16) {
        const __half* h = static_cast<const __half*>(p) + at;
        if (wide) {
            uint32_t w[E / 2];
            if constexpr (E == 2) w[0] = __ldcs(reinterpret_cast<const unsigned int*>(h));
            if constexpr (E == 4) {
                const uint2 v = __ldcs(reinterpret_cast<const uint2*>(h));
                w[0] = v.x; w[1] = v.y;
            }
            if constexpr (E == 8) {
                const uint4 v = __ldcs(reinterpret_cast<const uint4*>(h));
                w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
            }
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                x[2 * i] = half_bits_to_float(w[i] & 0xFFFFu);
                x[2 * i + 1] = half_bits_to_float(w[i] >> 16);
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) x[i] = __half2float(h[i]);
        }
    } else {
        const float* f = static_cast<const float*>(p) + at;
        if (wide) {
            if constexpr (E == 2) {
                const float2 v = __ldcs(reinterpret_cast<const float2*>(f));
                x[0] = v.x; x[1] = v.y;
            } else {
#pragma unroll
                for (int i = 0; i < E / 4; ++i) {
                    const float4 v = __ldcs(reinterpret_cast<const float4*>(f) + i);
                    x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) x[i] = f[i];
        }
    }
}

template <int E>
__device__ __forceinline__ void norm_row(float (&x)[E], const float* weight, float eps, int lane) {
    float p[E];
#pragma unroll
    for (int i = 0; i < E; ++i) p[i] = __fmul_rn(x[i], x[i]);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1)
#pragma unroll
        for (int i = 0; i < E; ++i) p[i] = __fadd_rn(p[i], __shfl_xor_sync(0xFFFFFFFFu, p[i], d));
#pragma unroll
    for (int h = E / 2; h >= 1; h >>= 1)
#pragma unroll
        for (int i = 0; i < h; ++i) p[i] = __fadd_rn(p[i], p[i + h]);
    const float inv = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fmul_rn(p[0], 1.0f / (32 * E)), eps)));
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = __fmul_rn(__fmul_rn(x[i], inv), weight[lane * E + i]);
}

// Rotates values 0 .. 2 half - 1 of the row; `row` is the warp's D floats of
// shared memory (the partner of value i lies half values away).
template <int E>
__device__ __forceinline__ void rotate_row(float (&x)[E], const float* cos, const float* sin, int half, bool interleaved,
                                           float* row, int lane) {
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < E; i += 2) {
            const int pair = (lane * E + i) >> 1;
            if (pair < half) {
                const float c = cos[pair], s = sin[pair], u = x[i], v = x[i + 1];
                x[i] = __fsub_rn(__fmul_rn(u, c), __fmul_rn(v, s));
                x[i + 1] = __fadd_rn(__fmul_rn(v, c), __fmul_rn(u, s));
            }
        }
    } else {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < E; ++i) row[lane * E + i] = x[i];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int at = lane * E + i;
            if (at < half) x[i] = __fsub_rn(__fmul_rn(x[i], cos[at]), __fmul_rn(row[at + half], sin[at]));
            else if (at < 2 * half) x[i] = __fadd_rn(__fmul_rn(x[i], cos[at - half]), __fmul_rn(row[at - half], sin[at - half]));
        }
    }
}

// pn4t's rule on the row's groups of 64 (2048 / D lanes each): d = fp16 of the
// first largest-magnitude value / -8, codes clamp(rint(x / d), -8, 7) + 8.
// Returns the group's scale bits; codes in n.
template <int E>
__device__ __forceinline__ uint32_t quantise_row(const float (&x)[E], int (&n)[E], int lane) {
    constexpr int kLanes = 64 / E;             // lanes of a group
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < E; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    uint32_t best = top;
#pragma unroll
    for (int d = kLanes / 2; d >= 1; d >>= 1) best = max(best, __shfl_xor_sync(0xFFFFFFFFu, best, d));
    float v = 0.0f;                            // the lane's first value of that size
#pragma unroll
    for (int i = E - 1; i >= 0; --i)
        if ((__float_as_uint(x[i]) & 0x7FFFFFFFu) == best) v = x[i];
    const uint32_t has = __ballot_sync(0xFFFFFFFFu, top == best);
    const uint32_t group = kLanes == 32 ? 0xFFFFFFFFu : ((1u << (kLanes & 31)) - 1u) << (lane / kLanes * kLanes);
    v = __shfl_sync(0xFFFFFFFFu, v, __ffs(has & group) - 1);
    const float q = fminf(fmaxf(__fmul_rn(v, -0.125f), -65504.0f), 65504.0f);
    uint32_t bits = __half_as_ushort(__float2half_rn(q));
    const bool zero = (bits & 0x7FFFu) == 0;
    if (zero) bits = 0;
    const float d = half_bits_to_float(bits);
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const float r = zero ? 0.0f : fminf(fmaxf(rintf(__fdiv_rn(x[i], d)), -8.0f), 7.0f);
        n[i] = static_cast<int>(r) + 8;
    }
    return bits;
}

struct AppendParams {
    KvAppendArgs a;
    KvCache cache;
    int64_t rows;              // tokens * (heads + 2 kv heads)
    bool wide_q, wide_k, wide_v;
};

constexpr int kAppendWarps = 8;

template <int D>
__global__ void __launch_bounds__(kAppendWarps * 32) append_kernel(const AppendParams P) {
    constexpr int E = D / 32;
    __shared__ float rows[kAppendWarps][D];
    const KvAppendArgs& a = P.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = a.heads + 2 * P.cache.heads;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * kAppendWarps + warp; row < P.rows;
         row += static_cast<int64_t>(gridDim.x) * kAppendWarps) {
        const int64_t t = row / per;
        const int r = static_cast<int>(row - t * per);
        const bool is_q = r < a.heads, is_v = r >= a.heads + P.cache.heads;
        const int h = is_q ? r : is_v ? r - a.heads - P.cache.heads : r - a.heads;
        const int64_t slot = is_q ? 0 : a.slots[t];
        if (!is_q && (slot < 0 || slot >= P.cache.slots())) continue;   // the whole warp
        float x[E];
        const void* src = is_q ? a.q : is_v ? a.v : a.k;
        const int64_t stride = is_q ? a.q_stride : is_v ? a.v_stride : a.k_stride;
        load_row<E>(src, t * stride + h * D + lane * E, a.f16, is_q ? P.wide_q : is_v ? P.wide_v : P.wide_k, x);
        if (!is_v) {
            const float* weight = is_q ? a.q_weight : a.k_weight;
            if (weight) norm_row<E>(x, weight, a.eps, lane);
            if (a.half) {
                const int pos = a.positions[t];
                if (pos >= 0 && pos < a.table_rows)
                    rotate_row<E>(x, a.cos + static_cast<int64_t>(pos) * a.half, a.sin + static_cast<int64_t>(pos) * a.half, a.half,
                                  a.interleaved, rows[warp], lane);
            }
        }
        if (is_q) {
            __half2* out = reinterpret_cast<__half2*>(a.q_out + (t * a.heads + h) * D + lane * E);
#pragma unroll
            for (int i = 0; i < E / 2; ++i) out[i] = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
            continue;
        }
        int n[E];
        const uint32_t bits = quantise_row<E>(x, n, lane);
        // code c of a word: half c & 1, bit 4 (c >> 1)
        uint32_t w = 0;
        const int c0 = (lane * E) & 7;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int c = c0 + i;
            w |= static_cast<uint32_t>(n[i]) << (16 * (c & 1) + 4 * (c >> 1));
        }
#pragma unroll
        for (int d = 1; d < 8 / E; d <<= 1) w |= __shfl_xor_sync(0xFFFFFFFFu, w, d);
        uint8_t* rec = P.cache.record(slot, h);
        const int tok = static_cast<int>(slot) & 15, j = lane * E / 64, i = (lane * E % 64) >> 3;
        if (c0 == 0) {
            const int off = is_v ? kv_v_word<D>(tok, j, i) : kv_k_word<D>(tok, j, i);
            *reinterpret_cast<uint32_t*>(rec + off) = w;
        }
        if (lane * E % 64 == 0) {
            const int off = (is_v ? kv_v_scales(D) : kv_k_scales(D)) + (tok * (D / 64) + j) * 2;
            *reinterpret_cast<uint16_t*>(rec + off) = static_cast<uint16_t>(bits);
        }
    }
}

// ------------------------------------------------------------------- read --

struct ReadParams {
    KvCache cache;
    const int64_t* slots;
    int64_t rows;              // tokens * kv heads * 2
    float* k;
    float* v;
};

template <int D>
__global__ void __launch_bounds__(256) read_kernel(const ReadParams P) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); row < P.rows;
         row += static_cast<int64_t>(gridDim.x) * 8) {
        const int64_t th = row >> 1;
        const bool is_v = row & 1;
        const int64_t t = th / P.cache.heads;
        const int h = static_cast<int>(th - t * P.cache.heads);
        const int64_t slot = P.slots[t];
        float x[E];
        if (slot < 0 || slot >= P.cache.slots()) {
#pragma unroll
            for (int i = 0; i < E; ++i) x[i] = 0.0f;
        } else {
            const uint8_t* rec = P.cache.record(slot, h);
            const int tok = static_cast<int>(slot) & 15, j = lane * E / 64, i = (lane * E % 64) >> 3;
            const uint32_t w = *reinterpret_cast<const uint32_t*>(rec + (is_v ? kv_v_word<D>(tok, j, i) : kv_k_word<D>(tok, j, i)));
            const float d = lds_half_as_float(rec + (is_v ? kv_v_scales(D) : kv_k_scales(D)) + (tok * (D / 64) + j) * 2);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int c = ((lane * E) & 7) + e;
                x[e] = __fmul_rn(d, static_cast<float>(static_cast<int>((w >> (16 * (c & 1) + 4 * (c >> 1))) & 15u) - 8));
            }
        }
        float* out = (is_v ? P.v : P.k) + th * D + lane * E;
        if constexpr (E == 2) {
            *reinterpret_cast<float2*>(out) = make_float2(x[0], x[1]);
        } else {
#pragma unroll
            for (int i = 0; i < E / 4; ++i)
                reinterpret_cast<float4*>(out)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
        }
    }
}

int log2_of(int v) {
    int s = 0;
    while ((1 << s) < v) ++s;
    return s;
}

KvCache cache_of(const KvGeometry& g) {
    return KvCache{g.data, g.pages, g.page_size, log2_of(g.page_size), g.heads, g.D};
}

bool rows_aligned(const void* p, int64_t stride, int size, int bytes) {
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && (stride * size) % bytes == 0;
}

}  // namespace

cudaError_t launch_kv_plan(const KvPlanArgs& a, int num_sms, cudaStream_t s) {
    PlanParams P{a, log2_of(a.page_size), 0};
    // a small batch needs few threads, and starts sooner with them
    const int threads = a.batch <= 256 && a.capacity <= 1024 ? 256 : kPlanThreads;
    P.each = (a.batch + threads - 1) / threads;
    const int smem = (2 * a.batch + 1) * 4;
    static std::atomic<uint64_t> smem_set{0};
    if (smem > 40 * 1024)
        if (cudaError_t e = set_smem_limit_once(plan_kernel, (2 * kKvMaxBatch + 1) * 4, smem_set); e != cudaSuccess) return e;
    int64_t blocks = (a.capacity + threads * 4 - 1) / (threads * 4);
    const int64_t by_request = (a.batch + 255) / 256;
    blocks = blocks > by_request ? blocks : by_request;
    if (blocks > num_sms) blocks = num_sms;
    if (blocks < 1) blocks = 1;
    plan_kernel<<<static_cast<int>(blocks), threads, smem, s>>>(P);
    return cudaGetLastError();
}

cudaError_t launch_kv_append(const KvAppendArgs& a, const KvGeometry& g, int num_sms, cudaStream_t s) {
    AppendParams P{a, cache_of(g), a.tokens * (a.heads + 2 * static_cast<int64_t>(g.heads)), false, false, false};
    const int size = a.f16 ? 2 : 4;
    const int bytes = g.D / 32 * size < 16 ? g.D / 32 * size : 16;
    P.wide_q = rows_aligned(a.q, a.q_stride, size, bytes);
    P.wide_k = rows_aligned(a.k, a.k_stride, size, bytes);
    P.wide_v = rows_aligned(a.v, a.v_stride, size, bytes);
    int64_t blocks = (P.rows + kAppendWarps - 1) / kAppendWarps;
    if (blocks > static_cast<int64_t>(num_sms) * 8) blocks = static_cast<int64_t>(num_sms) * 8;
    const int grid = static_cast<int>(blocks);
    if (g.D == 64) append_kernel<64><<<grid, kAppendWarps * 32, 0, s>>>(P);
    else if (g.D == 128) append_kernel<128><<<grid, kAppendWarps * 32, 0, s>>>(P);
    else append_kernel<256><<<grid, kAppendWarps * 32, 0, s>>>(P);
    return cudaGetLastError();
}

cudaError_t launch_kv_read(const KvGeometry& g, const int64_t* slots, int64_t tokens, float* k, float* v, int num_sms,
                           cudaStream_t s) {
    ReadParams P{cache_of(g), slots, tokens * g.heads * 2, k, v};
    int64_t blocks = (P.rows + 7) / 8;
    if (blocks > static_cast<int64_t>(num_sms) * 8) blocks = static_cast<int64_t>(num_sms) * 8;
    const int grid = static_cast<int>(blocks);
    if (g.D == 64) read_kernel<64><<<grid, 256, 0, s>>>(P);
    else if (g.D == 128) read_kernel<128><<<grid, 256, 0, s>>>(P);
    else read_kernel<256><<<grid, 256, 0, s>>>(P);
    return cudaGetLastError();
}

}  // namespace pn
