// pn_logprobs.cu -- log probabilities of given tokens, entropy and the top
// alternatives of rows of logits.
//
// With m the row's largest logit, d = logit - m and e = exp(scale d):
//   R = sum of e over all tokens but one of the largest, S = 1 + R, T = sum e d
//   ln p(token) = scale d - ln S,   entropy = ln S - scale T / S
// R goes without the largest token's 1, so ln S = log1p(R) keeps its bits where one
// token has nearly all of the probability; both terms of the entropy are positive or
// zero, so nothing cancels.
//
// Roundings (u = 2^-24): a thread adds 16 (fp16: 32) values by themselves, 8 (16) to a
// chain, and one such sum in each of a row's vocab / 4096 (8192) turns; a turn whose largest
// logit is a new one moves the sum so far, two additions, an ex2 (4 u) and a product.
// That makes 8 u a turn at most; then 6 additions, and 3 joins of warps and 3 of blocks
// of 8 u each; what the arguments of ex2 err by is at most 34 u, as a term moved by more than
// 2^24 does not count.
//
// One pass over memory.  A cluster of 1 to 8 thread blocks has a row, each block a
// contiguous part of it.  A warp takes 512 (fp16: 1024) values at a time under one
// reference m, the next ones on their way; only where one of them passes it (a few
// times in a row) are the sums moved and the new largest value left out of R.
//
// 2000 rows of 151936 fp16 logits: 123 us, 4.9 TB/s, with 74% of the issue slots in use and
// a last wave of one block to an SM (two blocks to every row: 130 us).  64 rows of fp32:
// 17.8 us, one wave; about 10 of them read.  One row of 32000: 7.1 us.
//
// Top k (at most 32).  The k-th largest of a block's 256 thread maxima is a lower
// bound of the k-th largest value of the row, and so is what all p blocks have (k / p)
// of, rounded up; the best of them is taken.  Only threads, and turns (a warp's 512 or
// 1024 values at a time), whose largest value reaches the bound can hold one of the top
// k: these are read again, and what reaches the bound goes to the row's
// first block, which ranks it by the 64-bit number (order of the logit, ~index): there
// are no ties in that order and the lowest index wins.  Where a block finds more than
// fits (a row of equal values, say), each warp keeps the k first of it in a sorted list,
// a lane to an entry.
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
constexpr int kUnroll = 4;                     // vectors of a thread at a time
constexpr int kMostFound = kWarps * 32;        // values of a block that may be in the top k
constexpr int kMostEntries = kMostCluster * kMostFound;
constexpr float kHuge = 1.7e38f;               // differences of numbers up to it are finite
constexpr float kLeast = -1e30f;               // exponents' least (exp2 of it is 0, and 0 times it is)

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

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Two fp32 numbers in a register pair, and operations on both at once.
using Two = unsigned long long;
__device__ __forceinline__ Two two(float a, float b) {
    Two d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float2 apart(Two v) {
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(v));
    return d;
}
__device__ __forceinline__ Two mul2(Two a, Two b) {
    Two d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ Two add2(Two a, Two b) {
    Two d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
    Two d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// Sums relative to a largest logit m, whose own 1 is not in r (m = -kHuge: no token
// yet); t is sum e y with y = scale log2 e (logit - m).
struct Sums {
    float m, r, t;
    __device__ __forceinline__ bool any() const { return m > -kHuge; }
    // what `o`, with a smaller or the same m, adds
    __device__ __forceinline__ void take(const Sums& o, float c) {
        const float by = (o.m - m) * c, f = exp2_fast(by), s = o.r + (o.any() ? 1.0f : 0.0f);
        r = fmaf(f, s, r);
        t += f == 0.0f ? 0.0f : f * fmaf(s, by, o.t);
    }
    __device__ __forceinline__ void join(const Sums& o, float c) {
        if (o.m > m) {
            const Sums mine = *this;
            *this = o;
            take(mine, c);
        } else {
            take(o, c);
        }
    }
};

// Lane i's for i < n (a power of two up to 32; others' do not count), joined in a fixed order, in all lanes.
__device__ __forceinline__ Sums join_lanes(Sums s, int n, float c) {
    for (int d = 1; d < n; d *= 2) s.join(Sums{__shfl_xor_sync(0xFFFFFFFFu, s.m, d), __shfl_xor_sync(0xFFFFFFFFu, s.r, d), __shfl_xor_sync(0xFFFFFFFFu, s.t, d)}, c);
    return Sums{__shfl_sync(0xFFFFFFFFu, s.m, 0), __shfl_sync(0xFFFFFFFFu, s.r, 0), __shfl_sync(0xFFFFFFFFu, s.t, 0)};
}

// 16 bytes of a row: value i of vector v is the row's element v * kVec - skew + i.
template <typename T>
struct RowOf {
    static constexpr int kVec = 16 / sizeof(T);
    const T* p;                // aligned to 16 bytes, `skew` elements before the row
    int skew, vocab;
    // Vector v as it lies there; -inf in place of what is outside the row, which is not read.
    __device__ __forceinline__ uint4 load(int v) const {
        const int at = v * kVec - skew;
        if (at >= 0 && at + kVec <= vocab) return __ldcg(reinterpret_cast<const uint4*>(p) + v);
        return edge(p, at, v, vocab);
    }
    static __device__ __noinline__ uint4 edge(const T* p, int at, int v, int vocab) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (kVec == 4) {
                w[i] = at + i >= 0 && at + i < vocab ? reinterpret_cast<const uint32_t*>(p)[v * 4 + i] : 0xFF800000u;
            } else {
                const uint16_t* h = reinterpret_cast<const uint16_t*>(p) + v * 8 + 2 * i;
                const uint32_t lo = at + 2 * i >= 0 && at + 2 * i < vocab ? h[0] : 0xFC00u, hi = at + 2 * i + 1 >= 0 && at + 2 * i + 1 < vocab ? h[1] : 0xFC00u;
                w[i] = lo | hi << 16;
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ uint4 nothing() {
        constexpr uint32_t w = kVec == 4 ? 0xFF800000u : 0xFC00FC00u;
        return make_uint4(w, w, w, w);
    }
    static __device__ __forceinline__ void values(const uint4& raw, float (&x)[kVec]) {
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (kVec == 4) {
                x[i] = __uint_as_float(w[i]);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                x[2 * i] = f.x;
                x[2 * i + 1] = f.y;
            }
        }
    }
    // -inf in place of the first value that is `high`.
    template <int N>
    static __device__ __forceinline__ void drop(uint4 (&raw)[N], float high) {
        bool done = false;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (kVec == 4) {
                    const bool hit = !done && __uint_as_float(w[i]) == high;
                    w[i] = hit ? 0xFF800000u : w[i];
                    done |= hit;
                } else {
                    const bool lo = !done && half_bits_to_float(w[i] & 0xFFFFu) == high;
                    w[i] = lo ? (w[i] & 0xFFFF0000u) | 0xFC00u : w[i];
                    done |= lo;
                    const bool hi = !done && half_bits_to_float(w[i] >> 16) == high;
                    w[i] = hi ? (w[i] & 0xFFFFu) | 0xFC000000u : w[i];
                    done |= hi;
                }
            }
            raw[j] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    // -inf in place of all values of kHuge and above (fp16: of infinity); how many there were.
    template <int N>
    static __device__ __forceinline__ float drop_huge(uint4 (&raw)[N]) {
        float n = 0.0f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (kVec == 4) {
                    const bool hit = __uint_as_float(w[i]) >= kHuge;
                    w[i] = hit ? 0xFF800000u : w[i];
                    n += hit;
                } else {
                    const bool lo = (w[i] & 0xFFFFu) == 0x7C00u, hi = w[i] >> 16 == 0x7C00u;
                    w[i] = lo ? (w[i] & 0xFFFF0000u) | 0xFC00u : w[i];
                    w[i] = hi ? (w[i] & 0xFFFFu) | 0xFC000000u : w[i];
                    n += lo + hi;
                }
            }
            raw[j] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        return n;
    }
    // The largest of N vectors (-inf where all are NaN).
    template <int N>
    static __device__ __forceinline__ float largest(const uint4 (&raw)[N]) {
        if constexpr (kVec == 4) {
            float most = -INFINITY;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                most = max3(most, __uint_as_float(raw[j].x), __uint_as_float(raw[j].y));
                most = max3(most, __uint_as_float(raw[j].z), __uint_as_float(raw[j].w));
            }
            return most;
        } else {
            __half2 most = __half2half2(__ushort_as_half(0xFC00));
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) most = __hmax2(most, *reinterpret_cast<const __half2*>(&w[i]));
            }
            return fmaxf(__low2float(most), __high2float(most));
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

// The order of floats that are no NaN as that of signed whole numbers, and back.
__device__ __forceinline__ int order_of(float x) {
    const int i = __float_as_int(x);
    return i < 0 ? i ^ 0x7FFFFFFF : i;
}
__device__ __forceinline__ float float_of(int i) { return __int_as_float(i < 0 ? i ^ 0x7FFFFFFF : i); }

template <typename T, bool kTop>
__global__ void __launch_bounds__(kThreads, 4) logprobs_kernel(const LogprobsArgs a) {
    using Row = RowOf<T>;
    constexpr int kVec = Row::kVec;
    cg::cluster_group cluster = cg::this_cluster();
    __shared__ Sums warp_sums[kWarps], block_sums;
    __shared__ int lists[kTop ? kWarps * 32 : 1];      // the warps' thread maxima in order
    extern __shared__ float highs[];                   // [turns][kWarps]: the largest value of each warp's turns
    __shared__ float bound, share;                     // the k-th and the (k / parts)-th of them
    __shared__ uint32_t found_count, entries, entry_base;
    __shared__ Key found[kTop ? kMostFound : 1];       // the block's
    __shared__ Key entry[kTop ? kMostEntries : 1];     // the row's (first block of a cluster)
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
    const Two c2 = two(c, c);

    const bool by_turns = kTop && parts == 1 && a.top > 1;     // how values are looked at again
    if (kTop && threadIdx.x == 0) {
        bound = share = -INFINITY;
        found_count = entries = 0;
    }
    int turn = 0;
    float m = -kHuge, best = -INFINITY;        // the warp's reference, the thread's maximum
    Two r2 = two(0.0f, 0.0f), t2 = r2;
    uint4 raw[kUnroll];
    auto fetch = [&](int v) {
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) raw[j] = v + lane + j * kThreads < v1 ? row.load(v + lane + j * kThreads) : Row::nothing();
    };
    fetch(v0 + warp * 32);
    for (int v = v0 + warp * 32; v < v1; v += kThreads * kUnroll) {    // the same for the whole warp
        uint4 now[kUnroll];
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) now[j] = raw[j];
        fetch(v + kThreads * kUnroll);         // the next ones are on their way meanwhile
        const float most = Row::largest(now);
        const float high = float_of(__reduce_max_sync(0xFFFFFFFFu, order_of(most)));
        if constexpr (kTop) {
            best = fmaxf(best, most);
            if (by_turns && lane == 0) highs[turn * kWarps + warp] = high;
            ++turn;
        }
        if (high > m || high >= kHuge) {
            const float to = fminf(fmaxf(high, m), kHuge), by = (m - to) * c, f = exp2_fast(by);
            const float2 r1 = apart(r2), t1 = apart(t2);
            const float sum = r1.x + r1.y + (lane == 0 && m > -kHuge ? 1.0f : 0.0f);
            if (to > m) {
                r2 = two(f * sum, 0.0f);
                t2 = two(f == 0.0f ? 0.0f : f * fmaf(sum, by, t1.x + t1.y), 0.0f);
                m = to;
                // the first value of that size, of the first lane that has one, is left out
                if (lane == __ffs(__ballot_sync(0xFFFFFFFFu, most == high)) - 1) Row::drop(now, high);
            }
            if (high >= kHuge) r2 = add2(r2, two(Row::drop_huge(now), 0.0f));      // each adds 1
        }
        // summed by themselves first: the chain of a row's sum is as long as it has turns, not values
        const Two less = two(-m, -m);
        Two r_turn, t_turn;
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
            float x[kVec];
            Row::values(now[j], x);
#pragma unroll
            for (int i = 0; i < kVec; i += 2) {
                const float2 d = apart(mul2(add2(two(x[i], x[i + 1]), less), c2));
                const float y0 = fmaxf(d.x, kLeast), y1 = fmaxf(d.y, kLeast);          // (NaN too)
                const Two e = two(exp2_fast(y0), exp2_fast(y1)), y = two(y0, y1);
                r_turn = j || i ? add2(r_turn, e) : e;
                t_turn = j || i ? fma2(e, y, t_turn) : mul2(e, y);
            }
        }
        r2 = add2(r2, r_turn);
        t2 = add2(t2, t_turn);
    }
    float2 pair = apart(r2);
    Sums all{m, pair.x + pair.y, 0.0f};
    pair = apart(t2);
    all.t = pair.x + pair.y;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) {
        all.r += __shfl_xor_sync(0xFFFFFFFFu, all.r, d);
        all.t += __shfl_xor_sync(0xFFFFFFFFu, all.t, d);
    }
    if (lane == 0) warp_sums[warp] = all;
    int key = order_of(best);
    if constexpr (kTop) {
        // the warp's thread maxima in order, the largest in lane 0
        if (a.top == 1) {
            key = __reduce_max_sync(0xFFFFFFFFu, key);
        } else {
#pragma unroll
            for (int size = 2; size <= 32; size *= 2)
#pragma unroll
                for (int d = size / 2; d >= 1; d /= 2) {
                    const int o = __shfl_xor_sync(0xFFFFFFFFu, key, d);
                    key = ((lane & size) == 0) == ((lane & d) == 0) ? max(key, o) : min(key, o);
                }
        }
        lists[warp * 32 + lane] = key;
    }
    __syncthreads();
    if (warp == 0) {
        all = join_lanes(warp_sums[lane % kWarps], kWarps, c);
        if (lane == 0) block_sums = all;
    }
    if constexpr (kTop) {
        // its place among the block's: how many of each other warp's list go before it (of equal ones, the lower warp's)
        if (a.top == 1) {
            if (threadIdx.x == 32) {
                for (int w = 0; w < kWarps; ++w) key = max(key, lists[w * 32]);
                bound = share = float_of(key);
            }
        } else if (lane < a.top) {
            int place = lane;
#pragma unroll
            for (int o = 1; o < kWarps; ++o) {
                const int other = (warp + o) % kWarps, than = other < warp ? key - (key > INT32_MIN) : key;
                const int* list = lists + other * 32;
                int n = 0;
#pragma unroll
                for (int step = 16; step >= 1; step /= 2) n += list[n + step - 1] > than ? step : 0;
                place += n + (n == 31 && list[31] > than);
            }
            if (place == a.top - 1) bound = float_of(key);
            if (place == (a.top - 1) / parts) share = float_of(key);
        }
    }
    cluster.sync();
    // the row's sums, in the blocks' order, and its bound
    float least = -kHuge;
    all = join_lanes(*cluster.map_shared_rank(&block_sums, lane % parts), parts, c);
    const bool none = !all.any();              // no token at all
    const float log_sum = log1pf(all.r);
    if constexpr (kTop) {
        const int most = __reduce_max_sync(0xFFFFFFFFu, order_of(*cluster.map_shared_rank(&bound, lane % parts)));
        const int all_have = __reduce_min_sync(0xFFFFFFFFu, order_of(*cluster.map_shared_rank(&share, lane % parts)));
        least = fmaxf(least, float_of(max(most, all_have)));
    }
    auto log_p = [&](float logit) {
        return none || !(logit > -kHuge) ? -INFINITY : fmaf(fminf(logit, kHuge) - all.m, a.scale, -log_sum);
    };
    if (rank == 0) {
        for (int i = threadIdx.x; i < a.count; i += kThreads) {
            const int token = a.tokens[r * a.count + i];
            a.logprobs[r * a.count + i] = token >= 0 && token < a.vocab ? log_p(static_cast<float>(begin[token])) : -INFINITY;
        }
        if (threadIdx.x == 0 && a.entropy) a.entropy[r] = none ? 0.0f : fmaxf(fmaf(-0.693147181f, all.t / (1.0f + all.r), log_sum), 0.0f);
    }
    if constexpr (kTop) {
        // f(16 bytes of each lane, whose vector) of the warp's values that may be some of the top k.  Of several in a row
        // of a block's own: the turns that may hold some, 2 KB in one piece each.  Of one, or a part of a row: the threads
        // that may, whose values, 4 KB apart, are few.  (64 rows of 151936 in eight parts, 20 wanted: 18.2 us by turns,
        // 17.2 by threads; 600 rows of a block each: 66 and 85; 2000 rows, one wanted: 125 and 122.)
        auto look_again = [&](auto f) {
            if (!by_turns) {
                for (uint32_t who = __ballot_sync(0xFFFFFFFFu, best >= least && best > -kHuge); who;) {
                    int first[kUnroll];        // of threads' vectors, whose loads are on their way together
#pragma unroll
                    for (int n = 0; n < kUnroll; ++n) {
                        first[n] = who ? v0 + warp * 32 + __ffs(who) - 1 + lane * kThreads : v1;
                        who &= who - 1;
                    }
                    for (int go = 0; go < v1 - v0; go += 32 * kThreads) {
                        uint4 raw[kUnroll][1];
#pragma unroll
                        for (int n = 0; n < kUnroll; ++n) raw[n][0] = first[n] + go < v1 ? row.load(first[n] + go) : Row::nothing();
#pragma unroll
                        for (int n = 0; n < kUnroll; ++n) f(raw[n], first[n] + go);
                    }
                }
                return;
            }
            for (int t0 = 0; t0 < turn; t0 += 32) {
                const float high = t0 + lane < turn ? highs[(t0 + lane) * kWarps + warp] : -INFINITY;
                for (uint32_t which = __ballot_sync(0xFFFFFFFFu, high >= least && high > -kHuge); which; which &= which - 1) {
                    const int first = warp * 32 + lane + (t0 + __ffs(which) - 1) * (kThreads * kUnroll);
                    uint4 raw[kUnroll][1];
#pragma unroll
                    for (int j = 0; j < kUnroll; ++j) raw[j][0] = first + j * kThreads < v1 ? row.load(first + j * kThreads) : Row::nothing();
#pragma unroll
                    for (int j = 0; j < kUnroll; ++j) f(raw[j], first + j * kThreads);
                }
            }
        };
        look_again([&](const uint4 (&raw)[1], int v) {
            if (!(Row::largest(raw) >= least)) return;
            float x[kVec];
            Row::values(raw[0], x);
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const Key k = x[i] >= least ? key_of(x[i], static_cast<uint32_t>(v * kVec - row.skew + i)) : 0;
                if (k == 0) continue;
                const uint32_t at = atomicAdd(&found_count, 1u);
                if (at < kMostFound) found[at] = k;
            }
        });
        __syncthreads();
        uint32_t* counter = cluster.map_shared_rank(&entries, 0);
        Key* to = cluster.map_shared_rank(entry, 0);
        const uint32_t count = found_count;
        if (count <= kMostFound) {
            if (threadIdx.x == 0) entry_base = count ? atomicAdd(counter, count) : 0;
            __syncthreads();
            if (threadIdx.x < count) to[entry_base + threadIdx.x] = found[threadIdx.x];
        } else {
            // many equal values or many large ones in one place: each warp keeps the k first in a sorted list
            Key list = 0, floor = 0;           // floor: the list's k-th
            look_again([&](const uint4 (&raw)[1], int v) {
                if (!__any_sync(0xFFFFFFFFu, Row::largest(raw) >= least)) return;
                float x[kVec];
                Row::values(raw[0], x);
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    const Key k = x[i] >= least ? key_of(x[i], static_cast<uint32_t>(v * kVec - row.skew + i)) : 0;
                    for (uint32_t in = __ballot_sync(0xFFFFFFFFu, k > floor); in; in &= in - 1) {
                        list = insert(list, __shfl_sync(0xFFFFFFFFu, k, __ffs(in) - 1));
                        floor = __shfl_sync(0xFFFFFFFFu, list, a.top - 1);
                        in &= __ballot_sync(0xFFFFFFFFu, k > floor) | (in & -in);
                    }
                }
            });
            if (lane >= a.top) list = 0;
            const int have = __popc(__ballot_sync(0xFFFFFFFFu, list != 0));
            uint32_t at = 0;
            if (lane == 0 && have) at = atomicAdd(counter, static_cast<uint32_t>(have));
            at = __shfl_sync(0xFFFFFFFFu, at, 0);
            if (lane < have) to[at + lane] = list;
        }
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
    if (kTop && parts == 1 && a.top > 1) {     // (one vector more where a row begins inside one)
        const int vectors = a.vocab / RowOf<T>::kVec + 2;
        cfg.dynamicSmemBytes = (vectors + kThreads * kUnroll - 1) / (kThreads * kUnroll) * kWarps * sizeof(float);
    }
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
