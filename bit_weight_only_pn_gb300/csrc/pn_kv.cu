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
// then fills its share of the maps, of the table and of the per-request outputs
// (these by block 0 alone cost 2 us).  Nothing is read that any block writes:
// taken pages come from the ring's [head, tail), given ones go behind its tail,
// table entries are read below `held` and written from it on.
//
// 4096 requests, 160000 slots: 7.4 us; 8 requests 3.5 us.  Bound by the chain of
// loads, scans and instructions that every block goes through (about 8000 cycles
// of 14000) and by the slot maps' loads behind it.

constexpr int kPlanThreads = 1024;

// Counts are 32 bits wide and stop at kMost (every block works through all
// requests, and in 64 bits that arithmetic was half its time): what passes it
// passes every capacity and every number of pages, which are below.
constexpr uint32_t kMost = 0x7FFFFFF0u;
__device__ __forceinline__ uint32_t sum_to_most(uint32_t a, uint32_t b) { return min(a + b, kMost); }

// Exclusive prefix over the block's threads of N counts; total gets the sums.
// `part` holds N entries per warp; the caller synchronises before it is reused.
template <int N>
__device__ __forceinline__ void block_scan(uint32_t (&v)[N], uint32_t* part, uint32_t (&total)[N]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    uint32_t in[N];
#pragma unroll
    for (int k = 0; k < N; ++k) in[k] = v[k];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, in[k], d);
            if (lane >= d) in[k] = sum_to_most(in[k], o);
        }
    if (lane == 31)
#pragma unroll
        for (int k = 0; k < N; ++k) part[k * 32 + warp] = in[k];
    __syncthreads();
    if (warp == 0) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            uint32_t w = lane < warps ? part[k * 32 + lane] : 0u;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, w, d);
                if (lane >= d) w = sum_to_most(w, o);
            }
            part[k * 32 + lane] = w;
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        total[k] = part[k * 32 + warps - 1];
        const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, in[k], 1);
        v[k] = sum_to_most(lane ? o : 0u, warp ? part[k * 32 + warp - 1] : 0u);
    }
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

// KEEP: a thread's requests where they stay in registers (read once, all loads on
// their way together), 0 where they are too many and are read in each pass.
template <int KEEP>
__global__ void __launch_bounds__(kPlanThreads, 1) plan_kernel(const PlanParams P) {
    extern __shared__ int plan_smem[];
    __shared__ uint32_t part[2 * 32];
    const KvPlanArgs& a = P.a;
    int* starts = plan_smem;                   // [batch + 1]
    int* first = plan_smem + a.batch + 1;      // [batch]: >= 0 the request's first page of the ring, -1 refused, <= -2 given back
    const int tid = threadIdx.x;
    const int b0 = min(tid * P.each, a.batch), b1 = min(b0 + P.each, a.batch);
    // whatever the ring holds, no index leaves it
    const int64_t ring_head = a.ring[0], tail = a.ring[1];
    const uint32_t avail = static_cast<uint32_t>(min(max(tail - ring_head, static_cast<int64_t>(0)), min(a.pages, static_cast<int64_t>(kMost - 1))));
    const uint32_t pages = static_cast<uint32_t>(a.pages), head = static_cast<uint32_t>(wrap(ring_head, a.pages));
    auto free_page = [&](uint32_t i) -> int32_t {         // i < avail <= pages
        const uint32_t at = head + i;
        return a.free_pages[at >= pages ? at - pages : at];
    };
    struct Item { int add, held, len; };
    auto read = [&](int b) -> Item { return {a.add[b], min(max(a.held[b], 0), a.max_pages), max(a.lens[b], 0)}; };
    Item kept[KEEP ? KEEP : 1];
    if constexpr (KEEP > 0) {
#pragma unroll
        for (int i = 0; i < KEEP; ++i) kept[i] = b0 + i < b1 ? read(b0 + i) : Item{0, 0, 0};
    }
    auto each_request = [&](auto f) {
        if constexpr (KEEP > 0) {
#pragma unroll
            for (int i = 0; i < KEEP; ++i)
                if (b0 + i < b1) f(b0 + i, kept[i]);
        } else {
#pragma unroll 4
            for (int b = b0; b < b1; ++b) f(b, read(b));
        }
    };

    // tokens and pages given back
    uint32_t mine[2] = {0, 0}, total[2];
    each_request([&](int, const Item& q) {
        mine[0] = sum_to_most(mine[0], max(q.add, 0));
        mine[1] = sum_to_most(mine[1], q.add < 0 ? q.held : 0);
    });
    block_scan(mine, part, total);
    const uint32_t tokens = total[0], given = total[1];
    __syncthreads();
    // pages taken by the requests that fit the table and the maps
    auto need_of = [&](const Item& q, uint32_t end) -> int {      // -1: does not fit
        const uint32_t len = static_cast<uint32_t>(q.len) + static_cast<uint32_t>(q.add);
        const uint32_t want = (len >> P.shift) + ((len & (a.page_size - 1)) != 0);
        if (want > static_cast<uint32_t>(a.max_pages) || end > static_cast<uint32_t>(a.capacity)) return -1;
        return max(static_cast<int>(want) - q.held, 0);
    };
    uint32_t need[1] = {0}, all_need[1];
    uint32_t tok = mine[0];
    each_request([&](int, const Item& q) {
        if (q.add < 0) return;
        tok = sum_to_most(tok, q.add);
        need[0] = sum_to_most(need[0], max(need_of(q, tok), 0));
    });
    block_scan(need, part, all_need);
    tok = mine[0];
    uint32_t taken = need[0], back = mine[1];
    uint32_t counts[2] = {0, 0};               // refused requests, pages that the others take
    // every block knows all per-request outputs and writes those of a few of its threads
    const bool writer = static_cast<uint32_t>(tid) * gridDim.x / blockDim.x == blockIdx.x;
    each_request([&](int b, const Item& q) {
        const int start = static_cast<int>(tok);
        starts[b] = start;
        int lens_out = 0, held_out = 0;
        if (q.add < 0) {
            first[b] = -2 - static_cast<int>(back);
            back = sum_to_most(back, q.held);
        } else {
            tok = sum_to_most(tok, q.add);
            const int n = need_of(q, tok);
            const uint32_t upto = sum_to_most(taken, max(n, 0));
            const bool ok = n == 0 || (n > 0 && upto <= avail);
            first[b] = ok ? static_cast<int>(taken) : -1;
            taken = upto;
            counts[0] += !ok;
            counts[1] += ok ? n : 0;
            lens_out = ok ? q.len + q.add : q.len;
            held_out = q.held + (ok ? n : 0);
        }
        if (writer) {
            a.starts[b] = start;
            a.lens_out[b] = lens_out;
            a.held_out[b] = held_out;
        }
    });
    if (tid == 0) starts[a.batch] = static_cast<int>(tokens);
    __syncthreads();                           // part is free again; starts and first are complete

    // table entries and returned pages: one warp per request
    const int warps = blockDim.x >> 5;
    for (int b = blockIdx.x * warps + (tid >> 5); b < a.batch; b += gridDim.x * warps) {
        const int f = first[b];
        if (f == -1) continue;
        const int held = min(max(a.held[b], 0), a.max_pages);
        int32_t* row = a.table + static_cast<int64_t>(b) * a.table_stride;
        if (f >= 0) {
            const int64_t want = (static_cast<int64_t>(max(a.lens[b], 0)) + a.add[b] + a.page_size - 1) >> P.shift;
            for (int64_t i = held + (tid & 31); i < want; i += 32) row[i] = free_page(static_cast<uint32_t>(f + i - held));
        } else {
            const int64_t to = tail + (-2 - static_cast<int64_t>(f));
            for (int i = tid & 31; i < held; i += 32) a.free_pages[wrap(to + i, a.pages)] = row[i];
        }
    }

    // Slot maps.  A warp has 32 tokens in a row: it finds the last request whose
    // start is at most the first token's (those that add nothing share the next
    // one's) with a lane to a probe, and from there each lane its own.
    const uint32_t capacity = static_cast<uint32_t>(a.capacity), stride = gridDim.x * blockDim.x;
    for (uint32_t t0 = blockIdx.x * blockDim.x + (tid & ~31); t0 < capacity; t0 += stride) {
        const uint32_t t = t0 + (tid & 31);
        int req = -1, pos = -1;
        int64_t slot = -1;
        if (t0 < tokens) {                     // (the whole warp)
            int lo = 0;                        // starts[lo] <= t0; none that is has an index of lo + span or above
            for (int span = a.batch; span > 1;) {
                const int step = (span + 31) / 32, at = lo + (tid & 31) * step;
                const uint32_t below = __ballot_sync(0xFFFFFFFFu, at < a.batch && at < lo + span && static_cast<uint32_t>(starts[min(at, a.batch)]) <= t0);
                const int k = 31 - __clz(below);
                span = min(step, lo + span - (lo + k * step));
                lo += k * step;
            }
            int up = 1;                        // doubling steps, then halving ones
            while (lo + up < a.batch && static_cast<uint32_t>(starts[lo + up]) <= t) {
                lo += up;
                up *= 2;
            }
            for (; up >= 1; up /= 2)
                if (lo + up < a.batch && static_cast<uint32_t>(starts[lo + up]) <= t) lo += up;
            if (t < tokens) {
                req = lo;
                const int f = first[lo];
                if (f >= 0) {
                    pos = max(a.lens[lo], 0) + static_cast<int>(t - starts[lo]);
                    const int held = min(max(a.held[lo], 0), a.max_pages), pg = pos >> P.shift;
                    const int32_t page = pg < held ? a.table[lo * a.table_stride + pg] : free_page(static_cast<uint32_t>(f + pg - held));
                    slot = (static_cast<int64_t>(page) << P.shift) + (pos & (a.page_size - 1));
                }
            }
        }
        if (t < capacity) {
            a.slots[t] = slot;
            a.positions[t] = pos;
            a.requests[t] = req;
        }
    }
    // the first block's totals, which no other needs
    if (blockIdx.x != 0) return;
    __syncthreads();
    block_scan(counts, part, total);
    if (tid == 0) {
        a.starts[a.batch] = starts[a.batch];
        a.ring_out[0] = ring_head + total[1];
        a.ring_out[1] = tail + given;
        a.refused[0] = static_cast<int>(total[0]);
    }
}

// ----------------------------------------------------------------- append --
//
// D / 8 lanes to a head row, so a warp takes 32 / (D / 8) heads of a token at
// once: lane l of a row owns values 4 l .. 4 l + 3 and D / 2 + 4 l .. + 3.
// With that ownership the pairwise sum's first level, the rotation of whole
// heads by halves and that of neighbours stay inside a lane, and a row's loads
// are 16 bytes wide.  A warp stays with its token for several groups of heads,
// so the rotation's row and the weights are read once.  For 8192 tokens of
// 48 + 16 heads of 128 in fp32: 85 us, 4.5 TB/s (in fp16 105 us).  It is bound by latency and by
// its instructions before it is by memory: four values to a lane and a warp to
// a row takes 307 us (its exchanges), sixteen to a lane 90 us (half the warps
// to an SM), and rows fetched further ahead than the next change nothing.
//
// The arithmetic is fixed, every operation rounded by itself, so codes are the
// same whatever computes them: squares added pairwise (the upper half of the
// row to the lower, until one sum is left), times 1 / D, plus eps, 1 / sqrt;
// x * that * weight; rotation with separate products and sums; pn4t's rule per
// group of 64.

struct Quads {
    float x[8];                                // values 4 l + i, then D / 2 + 4 l + i
};

// Two fp32 operations in one instruction.  No packed product may meet a packed
// sum: the assembler joins the two (also where the product is written as an
// fma of -0) and the product's own rounding is lost; products that are added
// are scalar ones.
__device__ __forceinline__ void mul2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void add2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

__device__ __forceinline__ void load_quad(const void* p, int64_t at, bool f16, bool wide, float* x) {
    if (f16) {
        const __half* h = static_cast<const __half*>(p) + at;
        if (wide) {
            const uint2 v = __ldcs(reinterpret_cast<const uint2*>(h));
            x[0] = half_bits_to_float(v.x & 0xFFFFu);
            x[1] = half_bits_to_float(v.x >> 16);
            x[2] = half_bits_to_float(v.y & 0xFFFFu);
            x[3] = half_bits_to_float(v.y >> 16);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = __half2float(h[i]);
        }
    } else {
        const float* f = static_cast<const float*>(p) + at;
        if (wide) {
            const float4 v = __ldcs(reinterpret_cast<const float4*>(f));
            x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = f[i];
        }
    }
}

template <int D>
__device__ __forceinline__ void norm_row(Quads& q, const float (&weight)[8], float eps) {
    constexpr int L = D / 8;
    float p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = __fmul_rn(q.x[i], q.x[i]);
#pragma unroll
    for (int i = 0; i < 4; i += 2) add2(p[i], p[i + 1], p[i], p[i + 1], p[4 + i], p[5 + i]);
#pragma unroll
    for (int d = L / 2; d >= 1; d >>= 1)
#pragma unroll
        for (int i = 0; i < 4; i += 2)
            add2(p[i], p[i + 1], p[i], p[i + 1], __shfl_xor_sync(0xFFFFFFFFu, p[i], d), __shfl_xor_sync(0xFFFFFFFFu, p[i + 1], d));
    const float sum = __fadd_rn(__fadd_rn(p[0], p[2]), __fadd_rn(p[1], p[3]));
    const float inv = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(sum, 1.0f / D), eps)));   // correctly rounded, as 1 / x is
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        mul2(q.x[i], q.x[i + 1], q.x[i], q.x[i + 1], inv, inv);
        mul2(q.x[i], q.x[i + 1], q.x[i], q.x[i + 1], weight[i], weight[i + 1]);
    }
}

// How the rotation's pairs lie.
enum { kTurnNone, kTurnHalves /* of the whole head: in a lane */, kTurnNeighbours, kTurnPart /* halves of a part */ };

// What a lane needs of the row of cos and sin, for each of its values: the
// pair's cos, and its sin with the sign of the value's product.
struct Turn {
    float c[8], s[8];
};

template <int D, int TURN>
__device__ __forceinline__ void load_turn(Turn& t, const float* cos, const float* sin, int half, int l) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int at = (i < 4 ? 0 : D / 2) + 4 * l + (i & 3);
        int pair;
        bool second;
        if (TURN == kTurnNeighbours) {
            pair = at >> 1;
            second = at & 1;
        } else {
            second = at >= half;
            pair = second ? at - half : at;
        }
        const bool turns = TURN == kTurnNeighbours ? pair < half : at < 2 * half;
        t.c[i] = turns ? cos[pair] : 1.0f;
        t.s[i] = turns ? (second ? sin[pair] : -sin[pair]) : 0.0f;
    }
}

// (a, b) -> (a c - b s, b c + a s), products and sums rounded one by one;
// a c - b s = a c + b (-s) exactly so.  `row` is D floats of shared memory per
// row (kTurnPart only).  Values outside the rotated part stay as they are.
template <int D, int TURN>
__device__ __forceinline__ void rotate_row(Quads& q, const Turn& t, int half, float* row, int l) {
    float partner[8];
    if (TURN == kTurnHalves) {
#pragma unroll
        for (int i = 0; i < 8; ++i) partner[i] = q.x[i ^ 4];
    } else if (TURN == kTurnNeighbours) {
#pragma unroll
        for (int i = 0; i < 8; ++i) partner[i] = q.x[i ^ 1];
    } else {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) row[(i < 4 ? 0 : D / 2) + 4 * l + (i & 3)] = q.x[i];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int at = (i < 4 ? 0 : D / 2) + 4 * l + (i & 3);
            partner[i] = at < half ? row[at + half] : at < 2 * half ? row[at - half] : 0.0f;
        }
    }
    // (a pair's two values turn or stay together: 2 half is even)
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const int at = (i < 4 ? 0 : D / 2) + 4 * l + (i & 3);
        if (TURN == kTurnHalves || at < 2 * half) {
            add2(q.x[i], q.x[i + 1], __fmul_rn(q.x[i], t.c[i]), __fmul_rn(q.x[i + 1], t.c[i + 1]), __fmul_rn(partner[i], t.s[i]),
                 __fmul_rn(partner[i + 1], t.s[i + 1]));
        }
    }
}

__device__ __forceinline__ float first_of_size(const float* x, uint32_t size) {
    float v = x[3];
#pragma unroll
    for (int i = 2; i >= 0; --i)
        if ((__float_as_uint(x[i]) & 0x7FFFFFFFu) == size) v = x[i];
    return v;
}

// The scale (fp16 bits) of a group whose first largest-magnitude value is v.
__device__ __forceinline__ uint32_t scale_bits(float v) {
    const uint32_t bits = __half_as_ushort(__float2half_rn(fminf(fmaxf(__fmul_rn(v, -0.125f), -65504.0f), 65504.0f)));
    return (bits & 0x7FFFu) ? bits : 0u;
}

// Codes clamp(rint(x / d), -8, 7) + 8 of four values at places c0 .. c0 + 3 of a word.
__device__ __forceinline__ uint32_t half_word(const float* x, uint32_t bits, int c0) {
    const float d = half_bits_to_float(bits);
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float r = bits ? fminf(fmaxf(rintf(__fdiv_rn(x[i], d)), -8.0f), 7.0f) : 0.0f;
        const int c = c0 + i;
        w |= static_cast<uint32_t>(static_cast<int>(r) + 8) << (16 * (c & 1) + 4 * (c >> 1));
    }
    return w;
}

// The lanes' 64-value groups by pn4t's rule.  D >= 128: a group is 16 lanes'
// first or second four values; D = 64: eight lanes' both.
template <int D>
__device__ __forceinline__ void group_scales(const Quads& q, uint32_t (&bits)[2]) {
    constexpr int kSpan = D == 64 ? 8 : 16;
    const int lane = threadIdx.x & 31;
    const uint32_t members = ((1u << kSpan) - 1u) << (lane / kSpan * kSpan);
    uint32_t top[2], best[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        top[k] = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) top[k] = max(top[k], __float_as_uint(q.x[4 * k + i]) & 0x7FFFFFFFu);
        best[k] = top[k];
#pragma unroll
        for (int d = kSpan / 2; d >= 1; d >>= 1) best[k] = max(best[k], __shfl_xor_sync(0xFFFFFFFFu, best[k], d));
    }
    if constexpr (D == 64) best[0] = best[1] = max(best[0], best[1]);
    float v[2];
    uint32_t has[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        has[k] = __ballot_sync(0xFFFFFFFFu, top[k] == best[k]) & members;
        v[k] = __shfl_sync(0xFFFFFFFFu, first_of_size(q.x + 4 * k, best[k]), has[k] ? __ffs(has[k]) - 1 : lane);
    }
    if constexpr (D == 64) v[0] = v[1] = has[0] ? v[0] : v[1];     // values 0 .. 31 come first
    bits[0] = scale_bits(v[0]);
    bits[1] = scale_bits(v[1]);
}

struct AppendParams {
    KvAppendArgs a;
    KvCache cache;
    int q_sets, kv_sets;       // groups of heads (32 / (D / 8) each) per token, of q and of k or v
    int sets;                  // groups that one warp takes, of one kind
    int q_tasks, kv_tasks;     // warps per token, of q and of k or v
    int64_t tasks;             // warps' worth of work
    bool wide_q, wide_k, wide_v;
};

constexpr int kAppendWarps = 8, kAppendBlocks = 4;                // of a block, of an SM

template <int D, bool F16, int TURN>
__global__ void __launch_bounds__(kAppendWarps * 32, kAppendBlocks) append_kernel(const AppendParams P) {
    constexpr int L = D / 8, kRows = 32 / L;   // lanes to a row, rows to a warp
    __shared__ float rows[TURN == kTurnPart ? kAppendWarps : 1][kRows * D];
    const KvAppendArgs& a = P.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % L, sub = lane / L;
    const int per = P.q_tasks + 2 * P.kv_tasks;
    for (int64_t task = static_cast<int64_t>(blockIdx.x) * kAppendWarps + warp; task < P.tasks;
         task += static_cast<int64_t>(gridDim.x) * kAppendWarps) {
        const int64_t t = task / per;
        int kind = static_cast<int>(task - t * per);
        const bool is_q = kind < P.q_tasks, is_v = kind >= P.q_tasks + P.kv_tasks;
        if (!is_q) kind -= is_v ? P.q_tasks + P.kv_tasks : P.q_tasks;
        const int64_t slot = is_q ? 0 : a.slots[t];
        if (!is_q && (slot < 0 || slot >= P.cache.slots())) continue;      // the whole warp
        const int heads = is_q ? a.heads : P.cache.heads;
        const int set0 = kind * P.sets, set1 = min(set0 + P.sets, is_q ? P.q_sets : P.kv_sets);
        const void* src = is_q ? a.q : is_v ? a.v : a.k;
        const bool wide = is_q ? P.wide_q : is_v ? P.wide_v : P.wide_k;
        const int64_t base = t * (is_q ? a.q_stride : is_v ? a.v_stride : a.k_stride);
        auto load = [&](Quads& q, int set) {
            const int h = min(set * kRows + sub, heads - 1);               // rows past the last head repeat it
            load_quad(src, base + h * D + 4 * l, F16, wide, q.x);
            load_quad(src, base + h * D + D / 2 + 4 * l, F16, wide, q.x + 4);
        };
        Quads next;
        load(next, set0);
        const float* weight = is_v ? nullptr : is_q ? a.q_weight : a.k_weight;
        float w[8];
        if (weight) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = weight[(i < 4 ? 0 : D / 2) + 4 * l + (i & 3)];
        }
        bool turns = TURN != kTurnNone && !is_v;
        Turn tn;
        if (turns) {
            const int pos = a.positions[t];
            turns = pos >= 0 && pos < a.table_rows;
            if (turns) load_turn<D, TURN>(tn, a.cos + static_cast<int64_t>(pos) * a.half, a.sin + static_cast<int64_t>(pos) * a.half, a.half, l);
        }
        uint2* to = reinterpret_cast<uint2*>(a.q_out + (t * a.heads + set0 * kRows + sub) * D + 4 * l);
        for (int set = set0; set < set1; ++set) {
            Quads q = next;
            if (set + 1 < set1) load(next, set + 1);
            if (weight) norm_row<D>(q, w, a.eps);
            if (turns) rotate_row<D, TURN>(q, tn, a.half, rows[TURN == kTurnPart ? warp : 0] + sub * D, l);
            const int h = set * kRows + sub;
            if (is_q) {
                if (h < heads) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const __half2 lo = __floats2half2_rn(q.x[4 * k], q.x[4 * k + 1]), hi = __floats2half2_rn(q.x[4 * k + 2], q.x[4 * k + 3]);
                        to[k * (D / 8)] = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
                    }
                }
                to += kRows * (D / 4);
                continue;
            }
            uint32_t bits[2];
            group_scales<D>(q, bits);
            // two lanes to a word: the even one puts the first half's together, the odd one the second's
            const bool odd = l & 1;
            const int c0 = odd ? 4 : 0;
            const uint32_t w0 = half_word(q.x, bits[0], c0), w1 = half_word(q.x + 4, bits[1], c0);
            const uint32_t word = (odd ? w1 : w0) | __shfl_xor_sync(0xFFFFFFFFu, odd ? w0 : w1, 1);
            if (h < heads) {
                uint8_t* rec = P.cache.record(slot, h);
                const int tok = static_cast<int>(slot) & 15;
                const int at = (odd ? D / 2 : 0) + 4 * (l & ~1), j = at / 64, i = (at % 64) / 8;
                *reinterpret_cast<uint32_t*>(rec + (is_v ? kv_v_word<D>(tok, j, i) : kv_k_word<D>(tok, j, i))) = word;
                if (D == 64 ? l == 0 : l % 16 == 0) {
                    uint8_t* sc = rec + (is_v ? kv_v_scales(D) : kv_k_scales(D)) + tok * (D / 64) * 2;
                    *reinterpret_cast<uint16_t*>(sc + 2 * (4 * l / 64)) = static_cast<uint16_t>(bits[0]);
                    if (D > 64) *reinterpret_cast<uint16_t*>(sc + 2 * ((D / 2 + 4 * l) / 64)) = static_cast<uint16_t>(bits[1]);
                }
            }
        }
    }
}

// ------------------------------------------------------------------- read --
//
// A lane to half a code word: four values, a 16-byte store.  28000 tokens, 8 heads of 128:
// 42 us, 6.1 TB/s (a whole word to a lane, whose stores left 16 bytes between lanes: 57).

struct ReadParams {
    KvCache cache;
    const int64_t* slots;
    int64_t parts;             // tokens * kv heads * D / 4
    float* k;
    float* v;
};

template <int D>
__global__ void __launch_bounds__(256) read_kernel(const ReadParams P) {
    constexpr int kParts = D / 4;              // half words of a token's head
    const int64_t stride = static_cast<int64_t>(gridDim.x) * 256;
    for (int64_t n = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; n < P.parts; n += stride) {
        const int64_t th = n / kParts;
        const int at = static_cast<int>(n % kParts), j = at / 16, i = at % 16 / 2, half = at % 2;
        const int64_t t = th / P.cache.heads;
        const int h = static_cast<int>(th - t * P.cache.heads);
        const int64_t slot = P.slots[t];
        const bool real = slot >= 0 && slot < P.cache.slots();
        const uint8_t* rec = P.cache.record(real ? slot : 0, h);
        const int tok = static_cast<int>(slot) & 15;
        uint32_t w[2] = {0, 0};
        float d[2] = {0.0f, 0.0f};
        if (real) {
            w[0] = *reinterpret_cast<const uint32_t*>(rec + kv_k_word<D>(tok, j, i));
            w[1] = *reinterpret_cast<const uint32_t*>(rec + kv_v_word<D>(tok, j, i));
            d[0] = lds_half_as_float(rec + kv_k_scales(D) + (tok * (D / 64) + j) * 2);
            d[1] = lds_half_as_float(rec + kv_v_scales(D) + (tok * (D / 64) + j) * 2);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float x[4];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                x[c] = real ? __fmul_rn(d[k], static_cast<float>(static_cast<int>((w[k] >> (16 * (c & 1) + 4 * (c >> 1) + 8 * half)) & 15u) - 8)) : 0.0f;
            __stcs(reinterpret_cast<float4*>(k ? P.v : P.k) + n, make_float4(x[0], x[1], x[2], x[3]));
        }
    }
}

template <int D, bool F16>
void append(const AppendParams& P, int turn, int grid, cudaStream_t s) {
    const int threads = kAppendWarps * 32;
    if (turn == kTurnNone) append_kernel<D, F16, kTurnNone><<<grid, threads, 0, s>>>(P);
    else if (turn == kTurnHalves) append_kernel<D, F16, kTurnHalves><<<grid, threads, 0, s>>>(P);
    else if (turn == kTurnNeighbours) append_kernel<D, F16, kTurnNeighbours><<<grid, threads, 0, s>>>(P);
    else append_kernel<D, F16, kTurnPart><<<grid, threads, 0, s>>>(P);
}

template <int D>
void append(const AppendParams& P, int turn, int grid, cudaStream_t s) {
    if (P.a.f16) append<D, true>(P, turn, grid, s);
    else append<D, false>(P, turn, grid, s);
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
    // a token to a thread and, for the table, a request to a warp, as far as one wave of blocks goes
    int64_t blocks = (a.capacity + threads - 1) / threads;
    const int64_t by_request = (a.batch + threads / 32 - 1) / (threads / 32);
    blocks = blocks > by_request ? blocks : by_request;
    if (blocks > num_sms) blocks = num_sms;
    if (blocks < 1) blocks = 1;
    auto run = [&](auto keep) {
        constexpr int kKeep = decltype(keep)::value;
        static std::atomic<uint64_t> smem_set{0};
        if (smem > 40 * 1024)
            if (cudaError_t e = set_smem_limit_once(plan_kernel<kKeep>, (2 * kKvMaxBatch + 1) * 4, smem_set); e != cudaSuccess) return e;
        plan_kernel<kKeep><<<static_cast<int>(blocks), threads, smem, s>>>(P);
        return cudaGetLastError();
    };
    if (P.each == 1) return run(std::integral_constant<int, 1>{});
    if (P.each <= 4) return run(std::integral_constant<int, 4>{});
    return run(std::integral_constant<int, 0>{});
}

cudaError_t launch_kv_append(const KvAppendArgs& a, const KvGeometry& g, int num_sms, cudaStream_t s) {
    AppendParams P{a, cache_of(g)};
    const int turn = a.half == 0 ? kTurnNone : a.interleaved ? kTurnNeighbours : a.half == g.D / 2 ? kTurnHalves : kTurnPart;
    const int rows = 32 / (g.D / 8);
    P.q_sets = (a.heads + rows - 1) / rows;
    P.kv_sets = (g.heads + rows - 1) / rows;
    // as many groups of heads to a warp as leave every SM its 32 warps, 8 at most: what a task reads first (its
    // slot or position, the rotation's row, the weights) costs it about four groups' time (1 group: 186 us, 4: 121)
    const int64_t all = a.tokens * (P.q_sets + 2 * static_cast<int64_t>(P.kv_sets));
    P.sets = 1;
    while (P.sets < 8 && all >= static_cast<int64_t>(num_sms) * 32 * P.sets * 2) P.sets *= 2;
    P.q_tasks = (P.q_sets + P.sets - 1) / P.sets;
    P.kv_tasks = (P.kv_sets + P.sets - 1) / P.sets;
    P.tasks = a.tokens * (P.q_tasks + 2 * static_cast<int64_t>(P.kv_tasks));
    const int size = a.f16 ? 2 : 4;
    P.wide_q = rows_aligned(a.q, a.q_stride, size, 4 * size);
    P.wide_k = rows_aligned(a.k, a.k_stride, size, 4 * size);
    P.wide_v = rows_aligned(a.v, a.v_stride, size, 4 * size);
    int64_t blocks = (P.tasks + kAppendWarps - 1) / kAppendWarps;
    // warps that take the next task when they are through with one: 85 us for 8192 tokens of 48 + 16 heads of 128,
    // where a block to every eight tasks (which waits for its longest) takes 89 us
    if (blocks > static_cast<int64_t>(num_sms) * kAppendBlocks) blocks = static_cast<int64_t>(num_sms) * kAppendBlocks;
    const int grid = static_cast<int>(blocks);
    if (g.D == 64) append<64>(P, turn, grid, s);
    else if (g.D == 128) append<128>(P, turn, grid, s);
    else append<256>(P, turn, grid, s);
    return cudaGetLastError();
}

cudaError_t launch_kv_read(const KvGeometry& g, const int64_t* slots, int64_t tokens, float* k, float* v, int num_sms,
                           cudaStream_t s) {
    ReadParams P{cache_of(g), slots, tokens * g.heads * (g.D / 4), k, v};
    int64_t blocks = (P.parts + 255) / 256;
    if (blocks > static_cast<int64_t>(num_sms) * 32) blocks = static_cast<int64_t>(num_sms) * 32;
    const int grid = static_cast<int>(blocks);
    if (g.D == 64) read_kernel<64><<<grid, 256, 0, s>>>(P);
    else if (g.D == 128) read_kernel<128><<<grid, 256, 0, s>>>(P);
    else read_kernel<256><<<grid, 256, 0, s>>>(P);
    return cudaGetLastError();
}

}  // namespace pn
