// pn_weigh_tc.cu -- the attention weight that cached tokens gather, for many query
// rows to a key/value head (prompts): the same function as pn_weigh.cu, on the
// fifth-generation tensor cores.
//
// A unit of work is (request, key/value head, 128 cached tokens).  The tokens are the
// M of the products and the query rows their N, so that a token's probabilities lie
// in one lane of tensor memory and are summed by one thread: nothing is exchanged
// between lanes.  S_j = K_j Q_j^T for each group j of 64 values, with K's codes as
// fp16 whole numbers n - 8 (exact) and the queries as they are; x = sum_j d_j S_j in
// fp32, so scores are as exact as in the kernels for few rows.  A row's log sum is one
// number here instead of two (less_of), whose rounding is in all of the row's
// probabilities; with that and thousands of rows to a sum, 2048 queries' weights err by
// 2.6e-7 of themselves, single queries' in the other kernel by 3e-8.  In a block of 25 warps
//   warps 16-19 decode the unit's codes into [token][64 values] tiles with the 128-byte
//     swizzle, once for all rows, and the scales as fp32;
//   warp 20 brings the query rows, a chunk at a time, by TMA: a box of 64 values, the
//     heads of the group and as many tokens as fit (64 rows of 256 values, 128 of
//     fewer); warps 21 and 23 make their lse ready and their positions;
//   warp 22 issues the products of a chunk into one of two places in tensor memory;
//   warps 0-15 take scores, exponentials and sums: of each chunk eight, four quarters
//     of the tokens by two halves of the columns;
//   warp 24 looks the units up, 32 at a time.
// A unit's chunks may be shared by a cluster of two blocks.  A token's sums (even and odd
// chunks, halves, blocks) are added at the unit's end in one order and written; results
// depend on neither timing nor what else is in the batch.
//
// 2048 queries of a prompt of 8192 tokens, 24 + 4 heads of 256: 253 us, 0.71 PFLOP/s of
// products.  60 rows of a unit take 1600 cycles: shared memory gives the N = 64 products
// their operands in 768, takes the next queries in 256 and gives the rows' constants in
// 256; tensor memory gives 128 KB in 1050.  (Two constants for a row took 119 us instead
// of 110 for 1024 queries with heads of 128; all 16 warps on one chunk, the next columns
// loaded while these are summed, and 32 columns at a time were no faster; codes converted
// under a branch and units looked up by every warp for itself had cost four and two times
// as much.)
//
// Every wait is bounded; a unit whose wait gave up gets NaN for its weights, and the call's
// status word, where it has one, PN_ETIMEOUT.
#include <atomic>
#include <cstdint>

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "pn_tcgen05.cuh"
#include "pn_weigh.cuh"

namespace pn {
namespace {

constexpr int kSumWarps = 16;                  // two places of S, two halves of the columns, four quarters of the tokens
constexpr int kThreads = (kSumWarps + 9) * 32; // 72 registers each
constexpr int kList = 32;                      // units looked up at a time
constexpr int kUnit = 128;                     // tokens of a unit, MMA M
constexpr int kPlaces = 2;                     // of S in tensor memory
constexpr int kRowStages = 4;                  // of the rows' constants
constexpr int kDecodeWarps = 4;
constexpr uint32_t kNap = 100;                 // nanoseconds between polls

struct Params {
    CUtensorMap qmap;          // queries [tokens][heads][D]; box 64 values x group x per
    WeighParams w;
    int per;                   // tokens of a chunk
    int split;                 // blocks to a unit, in a cluster: 1 or 2
};

template <int D>
struct Shape {
    static constexpr int kGroups = D / 64;
    static constexpr int kCols = D == 256 ? 64 : 128;          // rows of a chunk at most, MMA N
    static constexpr int kABufs = 2;           // decoded units
    static constexpr int kQStages = D == 256 ? 2 : D == 128 ? 4 : 6;
    static constexpr int kABytes = kGroups * kUnit * 128;
    static constexpr int kQBytes = kGroups * kCols * 128;
    static constexpr uint32_t kTmemCols = kPlaces * kGroups * kCols;       // 256 or 512
    static constexpr int kA = 0;
    static constexpr int kQ = kA + kABufs * kABytes;
    static constexpr int kScales = kQ + kQStages * kQBytes;                // [buffer][group][token] floats
    static constexpr int kRowData = kScales + kABufs * kGroups * kUnit * 4;    // [stage][less, pos][column]
    static constexpr int kParts = kRowData + kRowStages * 2 * kCols * 4;    // [2][4][token] parts of the sums
    static constexpr int kOther = kParts + 2 * 4 * kUnit * 4;               // [2][token] sums of the cluster's second block (in the first)
    static constexpr int kUnits = kOther + 2 * kUnit * 4;                  // [2][32] units
    static constexpr int kScan = kUnits + 2 * kList * 80;                  // [threads + 1] units before each thread's requests
    static constexpr int kWarpSums = kScan + (kThreads + 1) * 8;
    static constexpr int kBars = kWarpSums + kThreads / 32 * 8;
    static constexpr int kNumBars = 2 * kQStages + 3 * kABufs + 2 * kPlaces + 2 * kRowStages + 1 + 4 + 4;
    static constexpr int kMisc = kBars + kNumBars * 8;                     // TMEM base, abort, [stage] some row gives nothing (bytes)
    static_assert(kRowStages <= 8, "a byte to each behind two words");
    static constexpr int kBytes = kMisc + 16 + 1024;                       // slack to align to 1024 bytes
    static_assert(kBytes <= 227 * 1024, "fits one SM's shared memory");
    static_assert(kQ % 1024 == 0 && kQBytes % 1024 == 0 && kScales % 16 == 0 && kBars % 8 == 0, "alignment");
    static_assert(kTmemCols == 256 || kTmemCols == 512, "a size tensor memory is allocated in");
};

// fp32 accumulators, fp16 operands, both K-major, M = 128.
__host__ __device__ constexpr uint32_t desc_of(int cols) { return (1u << 4) | (static_cast<uint32_t>(cols >> 3) << 17) | (static_cast<uint32_t>(kUnit >> 4) << 24); }

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %3, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %4, p;\n\t}"
        :: "r"(d), "l"(a), "l"(b), "r"(static_cast<uint32_t>(accumulate)), "r"(desc) : "memory");
}
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        :: "r"(dst), "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// A float to, and an arrival at a barrier of, the same place of block `rank` of the cluster.
__device__ __forceinline__ void store_to_block(uint32_t addr, uint32_t rank, float v) {
    asm volatile("{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %0, %1;\n\tst.shared::cluster.f32 [r], %2;\n\t}" :: "r"(addr), "r"(rank), "f"(v) : "memory");
}
__device__ __forceinline__ void arrive_at_block(uint32_t bar, uint32_t rank) {
    asm volatile("{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %0, %1;\n\tmbarrier.arrive.release.cluster.shared::cluster.b64 _, [r];\n\t}" :: "r"(bar), "r"(rank) : "memory");
}
// A wait for arrivals from another block, whose writes before them are then seen.
__device__ __forceinline__ bool wait_cluster(uint32_t bar, uint32_t parity, uint64_t limit_ns, volatile uint32_t* abort) {
    const int64_t end = clock64() + cycles_of(limit_ns);
    for (;;) {
        uint32_t done;
        asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(done) : "r"(bar), "r"(parity) : "memory");
        if (done) return true;
        if (*abort || clock64() > end) return false;
        __nanosleep(20);
    }
}

// Two fp32 numbers in a register pair, and operations on both at once.
using Two = unsigned long long;
__device__ __forceinline__ Two two(float a, float b) {
    Two d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ Two two(uint32_t a, uint32_t b) {
    Two d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(a), "r"(b));
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

// Of the warps that sum: a barrier, and whether v holds for all of them.
__device__ __forceinline__ void sums_sync() { asm volatile("bar.sync 1, %0;" :: "n"(kSumWarps * 32) : "memory"); }
__device__ __forceinline__ bool all_sums(bool v) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbarrier.cta.red.and.pred q, 2, %1, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r) : "n"(kSumWarps * 32), "r"(static_cast<uint32_t>(v)) : "memory");
    return r != 0;
}

// A unit: the chunks of query rows that see any of its tokens, and the pages of its
// records (-1: none).  b < 0: there is no further one.
struct alignas(16) Unit {
    int b, h, tok0;
    int q0, n, pos0, len;
    int c0, chunks;
    int page[kUnit / kKvTokens];
    int unused[3];
};
static_assert(sizeof(Unit) == 80, "the list's place in shared memory");

// A request's units are numbered tile by tile, all heads of a tile after each other: in
// a prompt a tile costs no more than the one before.  Teams of blocks (of one or two)
// take units in turns, in every second one in reverse order, so the dear ones and the
// cheap ones of a prompt are shared out evenly (in plain turns, head by head, the
// busiest SM had 1.5 times the average).
__device__ __forceinline__ uint64_t unit_of_turn(uint64_t turn, uint32_t team, uint32_t teams) { return turn * teams + (turn & 1u ? teams - 1 - team : team); }

__device__ __noinline__ void look_up(const Params& P, const uint64_t* scan, int each, uint64_t u, Unit* to) {
    const WeighArgs& a = P.w.a;
    const KvCache& cache = P.w.cache;
    WeighRequest r;
    Unit w{};
    int of_head;
    locate<kUnit, kThreads>(P.w, scan, each, u, r, w.b, w.h, of_head);
    // (its number among the request's units, tile by tile)
    const uint64_t index = static_cast<uint64_t>(w.h) * units_of<kUnit>(r) + of_head;
    const uint64_t tile = index / static_cast<uint64_t>(cache.heads);
    w.h = static_cast<int>(index - tile * cache.heads);
    w.tok0 = static_cast<int>(tile) * kUnit;
    w.q0 = r.q0; w.n = r.n; w.pos0 = r.pos0; w.len = r.len;
    const int i0 = max(w.tok0 - r.pos0, 0), last = min(w.tok0 + kUnit, r.len) - 1;
    int i1 = r.n;
    if (a.window && w.tok0 >= a.sinks)
        i1 = static_cast<int>(min(static_cast<int64_t>(i1), max(static_cast<int64_t>(last) + a.window - r.pos0, static_cast<int64_t>(0))));
    w.c0 = i0 / P.per;
    w.chunks = i0 < i1 ? (i1 + P.per - 1) / P.per - w.c0 : 0;
#pragma unroll
    for (int i = 0; i < kUnit / kKvTokens; ++i) {
        const int tok = w.tok0 + i * kKvTokens;
        const int page = tok < r.len ? a.table[w.b * a.table_stride + (tok >> cache.page_shift)] : -1;
        w.page[i] = page >= 0 && page < cache.pages ? page : -1;
    }
    *to = w;
}

// A place in a ring and how often it went round.
template <int N>
struct Ring {
    uint32_t at = 0, turn = 0;
    __device__ __forceinline__ void step() {
        if (++at == N) {
            at = 0;
            ++turn;
        }
    }
    __device__ __forceinline__ uint32_t full() const { return turn & 1u; }             // phase of the turn's filling
    __device__ __forceinline__ uint32_t emptied() const { return (turn - 1u) & 1u; }   // of the emptying before it (turn > 0)
};

// A thread's share of a chunk: S of its token at ts, kCols columns by group.
// Columns c0 .. c1 - 1, multiples of 16, are its warp's.
template <int D, bool kMasked>
__device__ __forceinline__ Two chunk_sum(Two sum, uint32_t ts, const Two (&d)[D / 64], float scale, const float* rows, int c0, int c1, int tok, int window, int sinks) {
    constexpr int NG = D / 64, kCols = Shape<D>::kCols;
    const Two f = two(scale, scale);
    constexpr int kBlock = D == 256 ? 8 : 16;
#pragma unroll 1
    for (int c = c0; c < c1; c += kBlock) {
        uint32_t s[NG][kBlock];
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            if constexpr (kBlock == 16) tmem_ld16(ts + kCols * j + c, s[j]);
            else tmem_ld8(ts + kCols * j + c, s[j]);
        }
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < kBlock; i += 4) {
            const ulonglong2 less = *reinterpret_cast<const ulonglong2*>(rows + c + i);
            const Two l2[2] = {less.x, less.y};
            int pos[4];
            if constexpr (kMasked) {
                const int4 v = *reinterpret_cast<const int4*>(rows + kCols + c + i);
                pos[0] = v.x; pos[1] = v.y; pos[2] = v.z; pos[3] = v.w;
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                Two x = mul2(d[0], two(s[0][i + 2 * k], s[0][i + 2 * k + 1]));
#pragma unroll
                for (int j = 1; j < NG; ++j) x = fma2(d[j], two(s[j][i + 2 * k], s[j][i + 2 * k + 1]), x);
                const float2 y = apart(fma2(x, f, l2[k]));
                float p0 = ex2(y.x), p1 = ex2(y.y);
                if constexpr (kMasked) {
                    const int q0 = pos[2 * k], q1 = pos[2 * k + 1];
                    p0 = tok <= q0 && (tok > q0 - window || tok < sinks) ? p0 : 0.0f;
                    p1 = tok <= q1 && (tok > q1 - window || tok < sinks) ? p1 : 0.0f;
                }
                sum = add2(sum, two(p0, p1));
            }
        }
    }
    return sum;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) weigh_tc_kernel(const __grid_constant__ Params P) {
    using S = Shape<D>;
    constexpr int NG = S::kGroups, kCols = S::kCols, kABufs = S::kABufs, kQStages = S::kQStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = smem_addr(smem_raw), base = (raw_base + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw_base);
    uint32_t bar = base + S::kBars;
    auto take = [&](int n) { const uint32_t b = bar; bar += 8u * n; return b; };
    const uint32_t q_full = take(kQStages), q_empty = take(kQStages), a_full = take(kABufs), a_empty = take(kABufs), d_empty = take(kABufs);
    const uint32_t s_full = take(kPlaces), s_empty = take(kPlaces), rows_full = take(kRowStages), rows_empty = take(kRowStages), drain = take(1);
    const uint32_t list_full = take(2), list_empty = take(2);
    const uint32_t x_full = take(2), x_empty = take(2);        // of the second block's sums: in the first block, in the second
    volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + S::kMisc);
    volatile uint32_t* abort = misc + 1;
    volatile uint8_t* some_none = reinterpret_cast<volatile uint8_t*>(misc + 2);
    uint64_t* scan = reinterpret_cast<uint64_t*>(smem + S::kScan);
    const WeighArgs& a = P.w.a;
    const KvCache& cache = P.w.cache;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = P.w.group;
    const uint64_t limit = P.w.timeout_ns;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kQStages; ++s) {
            mbar_init(q_full + 8 * s, 1);
            mbar_init(q_empty + 8 * s, 1);
        }
        for (int s = 0; s < kABufs; ++s) {
            mbar_init(a_full + 8 * s, kDecodeWarps);
            mbar_init(a_empty + 8 * s, 1);
            mbar_init(d_empty + 8 * s, kSumWarps);
        }
        for (int s = 0; s < kPlaces; ++s) {
            mbar_init(s_full + 8 * s, 1);
            mbar_init(s_empty + 8 * s, kSumWarps / 2);
        }
        for (int s = 0; s < kRowStages; ++s) {
            mbar_init(rows_full + 8 * s, 1);
            mbar_init(rows_empty + 8 * s, kSumWarps / 2);
        }
        mbar_init(drain, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(list_full + 8 * s, 1);
            mbar_init(list_empty + 8 * s, kSumWarps + kDecodeWarps + 4);       // of every warp but the list's
            mbar_init(x_full + 8 * s, 4);
            mbar_init(x_empty + 8 * s, 4);
        }
        *abort = 0u;
        fence_mbar_init();
    }
    if (warp == kThreads / 32 - 1) {
        tmem_alloc(base + S::kMisc, S::kTmemCols);
        tmem_relinquish();
    }
    // rows that no box fills stay zero: their products are finite
    for (int i = threadIdx.x; i < kQStages * S::kQBytes / 16; i += kThreads) reinterpret_cast<uint4*>(smem + S::kQ)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    const int each = scan_units<kUnit, kThreads>(P.w, scan, reinterpret_cast<uint64_t*>(smem + S::kWarpSums));
    tc_fence_before_sync();
    __syncthreads();
    if (P.split > 1) cluster_sync();           // both blocks' barriers are there
    tc_fence_after_sync();
    const uint32_t tmem = misc[0];
    // nap: of the warps that work ahead, whose polling would take the others' issue slots
    auto wait = [&](uint32_t b, uint32_t parity, uint32_t nap = 0) { return mbar_try_wait(b, parity) || wait_phase(b, parity, limit, abort, nap); };
    const int split = P.split, rank = static_cast<int>(blockIdx.x) % split;    // the block's chunks: rank, rank + split, ...
    Unit* list = reinterpret_cast<Unit*>(smem + S::kUnits);
    // The team's unit of a turn, from the list; false behind the last one (or where a wait gave up).
    auto unit_at = [&](uint32_t turn, const Unit*& w, bool& ok) {
        const uint32_t half = (turn / kList) & 1u;
        if (turn % kList == 0) ok = ok && wait(list_full + 8 * half, (turn / (2 * kList)) & 1u);
        w = list + half * kList + turn % kList;
        return ok && w->b >= 0;
    };
    // The same by a whole warp, whose lanes poll each for itself: one answer for all of them.
    auto unit_of_warp = [&](uint32_t turn, const Unit*& w, bool& ok) {
        const bool more = unit_at(turn, w, ok);
        ok = __all_sync(0xFFFFFFFFu, ok);
        return __all_sync(0xFFFFFFFFu, more);
    };
    auto done_with = [&](uint32_t turn) {      // by one thread of each warp
        if (turn % kList == kList - 1) mbar_arrive(list_empty + 8 * ((turn / kList) & 1u));
    };

    if (warp == kSumWarps + 8) {
        // ------------------------------------------------------ unit list --
        // a lane to a unit: found one by one in every role, a unit took each of them some
        // thousand cycles (24 requests with 64 rows of 128 over 4096 tokens: 180 us)
        const uint64_t total = scan[kThreads];
        const uint32_t team = blockIdx.x / split, teams = gridDim.x / split;
        for (uint32_t first = 0;; first += kList) {
            const uint32_t half = (first / kList) & 1u;
            if (first >= 2 * kList && !__all_sync(0xFFFFFFFFu, wait(list_empty + 8 * half, (first / (2 * kList) - 1) & 1u, kNap))) break;
            const uint64_t u = unit_of_turn(static_cast<uint64_t>(first) + lane, team, teams);
            Unit* to = list + half * kList + lane;
            if (u < total) look_up(P, scan, each, u, to);
            else to->b = -1;
            __syncwarp();
            if (lane == 0) mbar_arrive(list_full + 8 * half);
            if (!__all_sync(0xFFFFFFFFu, u < total)) break;
        }
    } else if (warp == kSumWarps + 4) {
        // ------------------------------------------------------- queries --
        if (lane == 0) {
            Ring<kQStages> q;
            bool ok = true, stalled = false;
            uint32_t issued = 0;
            const Unit* w;
            for (uint32_t turn = 0; unit_at(turn, w, ok); ++turn) {
                for (int c = rank; c < w->chunks; c += split) {
                    if (q.turn > 0 && !wait(q_empty + 8 * q.at, q.emptied(), kNap)) {
                        ok = false;
                        break;
                    }
                    // (testing aid: with stall the first chunk's bytes are announced but never
                    // copied; its wait can only time out)
                    stalled |= P.w.stall != 0;
                    const uint32_t dst = base + S::kQ + q.at * S::kQBytes, full = q_full + 8 * q.at;
                    mbar_arrive_expect_tx(full, static_cast<uint32_t>(NG * P.per * group * 128));
                    if (stalled) {
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int j = 0; j < NG; ++j) tma_load_3d(dst + j * kCols * 128, &P.qmap, 64 * j, w->h * group, w->q0 + (w->c0 + c) * P.per, full);
                    ++issued;
                    q.step();
                }
                if (!ok) break;
                done_with(turn);
            }
            if (!ok && !stalled) *abort = 1u;
            // the last copies into the stages land before the block ends, also after an abort
            for (uint32_t s = 0; s < kQStages && s < issued; ++s) wait_phase(q_full + 8 * s, ((issued - 1 - s) / kQStages) & 1u, kAttnDrainNs, nullptr);
        }
        __syncwarp();
    } else if (warp == kSumWarps + 5 || warp == kSumWarps + 7) {
        // ------------------------------------------------ the rows' constants --
        // (a load of lse waited for in every chunk took 3500 cycles a chunk, where its products take 800)
        constexpr int kEach = kCols / 32;      // rows of a lane
        Ring<kRowStages> s;
        int of_token[kEach], of_head[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            of_token[k] = (lane + 32 * k) / group;
            of_head[k] = lane + 32 * k - of_token[k] * group;
        }
        bool ok = true;
        const Unit* w;
        for (uint32_t turn = 0; unit_of_warp(turn, w, ok); ++turn) {
            float lse[kEach];
            auto fetch = [&](int c) {          // of the unit's chunk c; any of the request's where there is no such row
#pragma unroll
                for (int k = 0; k < kEach; ++k) {
                    const int i = min((w->c0 + c) * P.per + of_token[k], w->n - 1);
                    lse[k] = a.lse[(static_cast<int64_t>(w->q0) + i) * a.heads + w->h * group + of_head[k]];
                }
            };
            // the two warps take the block's chunks in turn
            const int mine = rank + (((s.at & 1u) != 0) != (warp == kSumWarps + 7) ? split : 0);
            if (mine < w->chunks) fetch(mine);
            for (int c = rank; c < w->chunks; c += split) {
                if (((s.at & 1u) != 0) != (warp == kSumWarps + 7)) {
                    s.step();
                    continue;
                }
                float now[kEach];
#pragma unroll
                for (int k = 0; k < kEach; ++k) now[k] = lse[k];
                if (c + 2 * split < w->chunks) fetch(c + 2 * split);
                if (s.turn > 0 && !__all_sync(0xFFFFFFFFu, wait(rows_empty + 8 * s.at, s.emptied(), kNap))) {
                    ok = false;
                    break;
                }
                float* to = reinterpret_cast<float*>(smem + S::kRowData) + s.at * 2 * kCols;
                bool none = false;             // (a row that gives nothing sees no token: its products may be NaN)
#pragma unroll
                for (int k = 0; k < kEach; ++k) {
                    const int row = lane + 32 * k, i = (w->c0 + c) * P.per + of_token[k];
                    const bool real = of_token[k] < P.per && i < w->n, gives = real && fabsf(now[k]) != INFINITY;
                    none |= real && !gives;
                    to[row] = less_of(gives ? now[k] : -INFINITY, P.w.scale_rest);
                    reinterpret_cast<int*>(to)[kCols + row] = gives ? w->pos0 + i : INT32_MIN;
                }
                none = __any_sync(0xFFFFFFFFu, none);
                if (lane == 0) some_none[s.at] = none;
                __syncwarp();
                if (lane == 0) mbar_arrive(rows_full + 8 * s.at);
                s.step();
            }
            if (!ok) break;
            __syncwarp();
            if (lane == 0) done_with(turn);
        }
        if (!ok) *abort = 1u;
    } else if (warp == kSumWarps + 6) {
        // ------------------------------------------------------ MMA issue --
        if (elect_one()) {
            Ring<kQStages> q;
            Ring<kABufs> k;
            Ring<kPlaces> t;
            bool ok = true;
            const Unit* w;
            for (uint32_t turn = 0; unit_at(turn, w, ok); ++turn) {
                ok = wait(a_full + 8 * k.at, k.full(), 20);
                if (!ok) break;
                const int chunks = w->chunks, n = w->n, first = w->c0;
                for (int c = rank; c < chunks; c += split) {
                    ok = (t.turn == 0 || wait(s_empty + 8 * t.at, t.emptied(), 20)) && wait(q_full + 8 * q.at, q.full(), 20);
                    if (!ok) break;
                    tc_fence_after_sync();
                    const uint32_t desc = desc_of((min(P.per, n - (first + c) * P.per) * group + 15) / 16 * 16);
                    const uint32_t ka = base + S::kA + k.at * S::kABytes, qa = base + S::kQ + q.at * S::kQBytes, d = tmem + t.at * (NG * kCols);
#pragma unroll
                    for (int j = 0; j < NG; ++j)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_ss(d + kCols * j, smem_desc_sw128(ka + j * (kUnit * 128) + kk * 32), smem_desc_sw128(qa + j * (kCols * 128) + kk * 32), desc, kk != 0);
                    mma_commit(q_empty + 8 * q.at);
                    mma_commit(s_full + 8 * t.at);
                    q.step();
                    t.step();
                }
                if (!ok) break;
                mma_commit(a_empty + 8 * k.at);
                k.step();
                done_with(turn);
            }
            if (!ok) *abort = 1u;
            mma_commit(drain);                 // every product of this block finished (also after an abort)
            wait_phase(drain, 0u, kAttnDrainNs, nullptr);
        }
        __syncwarp();
    } else if (warp >= kSumWarps && warp < kSumWarps + kDecodeWarps) {
        // --------------------------------------------------------- decode --
        constexpr int GP = kv_plane_groups(D), PL = kv_planes(D), kRecords = kUnit / kKvTokens / kDecodeWarps;
        const int g = lane >> 2, t = lane & 3;
        Ring<kABufs> k;
        bool ok = true;
        // a unit's words are on their way while the one before is decoded, as registers allow
        constexpr bool kAhead = D < 256;
        struct Words {
            uint32_t k[kRecords][2][D / 32];
            uint16_t scale[kRecords][2];       // fp16 bits, of tokens lane % 8 and 8 more, group lane / 8
        };
        auto load = [&](const Unit& w, Words& to) {
#pragma unroll
            for (int i = 0; i < kRecords; ++i) {
                const int rec = (warp - kSumWarps) + i * kDecodeWarps, page = w.page[rec];
                const uint8_t* record = page < 0 ? nullptr :
                    cache.record((static_cast<int64_t>(page) << cache.page_shift) + ((w.tok0 + rec * kKvTokens) & (cache.page_size - 1)), w.h);
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
#pragma unroll
                    for (int q = 0; q < D / 32; ++q) to.k[i][hh][q] = 0x88888888u;      // (zero)
                    to.scale[i][hh] = 0;
                    if (!record) continue;
#pragma unroll
                    for (int pl = 0; pl < PL; ++pl) {
                        const uint8_t* p = record + ((hh * PL + pl) * 32 + lane) * 8 * GP;
                        if constexpr (GP == 2) {
                            const uint4 v = *reinterpret_cast<const uint4*>(p);
                            to.k[i][hh][4 * pl] = v.x; to.k[i][hh][4 * pl + 1] = v.y; to.k[i][hh][4 * pl + 2] = v.z; to.k[i][hh][4 * pl + 3] = v.w;
                        } else {
                            const uint2 v = *reinterpret_cast<const uint2*>(p);
                            to.k[i][hh][0] = v.x; to.k[i][hh][1] = v.y;
                        }
                    }
                    // (converted later: a value made of a load under a branch waits for it there)
                    to.scale[i][hh] = *reinterpret_cast<const uint16_t*>(record + kv_k_scales(D) + ((hh * 8 + (lane & 7)) * NG + min(lane >> 3, NG - 1)) * 2);
                }
            }
        };
        const Unit* w;
        Words now, next;
        bool more = unit_of_warp(0, w, ok);
        if (kAhead && more) load(*w, next);
        for (uint32_t turn = 0; more; ++turn) {
            if constexpr (kAhead) now = next;
            else load(*w, now);
            __syncwarp();
            if (lane == 0) done_with(turn);    // its entry is not looked at again
            more = unit_of_warp(turn + 1, w, ok);
            if (kAhead && more) load(*w, next);
            if (k.turn > 0) ok = ok && wait(a_empty + 8 * k.at, k.emptied(), kNap) && wait(d_empty + 8 * k.at, k.emptied(), kNap);
            if (!__all_sync(0xFFFFFFFFu, ok)) {
                ok = false;
                break;
            }
            uint8_t* tile = smem + S::kA + k.at * S::kABytes;
            float* d = reinterpret_cast<float*>(smem + S::kScales) + k.at * NG * kUnit;
            auto put = [&](int token, int j, int i, uint32_t word) {   // 16-byte chunk `i` of a token's row in a group's tile
                const uint32_t sh = word >> 8;
                *reinterpret_cast<uint4*>(tile + j * (kUnit * 128) + token * 128 + ((i ^ (token & 7)) << 4)) =
                    make_uint4(decode_pair<kPn4t, 0>(word, sh), decode_pair<kPn4t, 1>(word, sh), decode_pair<kPn4t, 2>(word, sh), decode_pair<kPn4t, 3>(word, sh));
            };
#pragma unroll
            for (int i = 0; i < kRecords; ++i) {
                const int first = ((warp - kSumWarps) + i * kDecodeWarps) * kKvTokens;
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
#pragma unroll
                    for (int j = 0; j < NG; ++j) {
                        put(first + hh * 8 + g, j, 2 * t, now.k[i][hh][2 * j]);
                        put(first + hh * 8 + g, j, 2 * t + 1, now.k[i][hh][2 * j + 1]);
                    }
                    if ((lane >> 3) < NG) d[(lane >> 3) * kUnit + first + hh * 8 + (lane & 7)] = half_bits_to_float(now.scale[i][hh]);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(a_full + 8 * k.at);
            k.step();
        }
        if (!ok) *abort = 1u;
    } else if (warp < kSumWarps) {
        // ----------------------------------------------- scores and sums --
        const int mine = warp >> 2, place = mine & 1, token = threadIdx.x & (kUnit - 1);
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        float* parts = reinterpret_cast<float*>(smem + S::kParts);
        const int window = a.window ? a.window : INT32_MAX;
        Ring<kABufs> k;
        Ring<kPlaces> t;
        Ring<kRowStages> rows;
        bool ok = true, listed = true;         // listed: the units can be told, whatever else has given up
        const Unit* unit;
        uint32_t n = 0;
        for (;; ++n) {
            const bool more = unit_of_warp(n, unit, listed);
            // Every unit has a barrier of all these warps, so all of them go on or none does: what one
            // has waited for in vain another may find a moment later.
            if (n % kList == 0) listed = all_sums(listed);
            if (!listed || !more) break;
            const Unit w = *unit;
            const int tok = w.tok0 + token;
            // where the token's weight is, and what it was
            int64_t to = -1;
            float before = 0.0f;
            if (tok < w.len) {
                const int page = unit->page[token / kKvTokens];
                if (page >= 0) to = ((static_cast<int64_t>(page) * cache.heads + w.h) << cache.page_shift) + (tok & (cache.page_size - 1));
            }
            __syncwarp();
            if (lane == 0) done_with(n);
            if (mine == 0 && to >= 0 && a.weights && tok < w.pos0) before = a.decay * a.weights[to];
            ok = ok && __all_sync(0xFFFFFFFFu, wait(a_full + 8 * k.at, k.full()));
            Two d[NG];
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                const float v = reinterpret_cast<const float*>(smem + S::kScales)[(k.at * NG + j) * kUnit + token];
                d[j] = two(v, v);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(d_empty + 8 * k.at);
            k.step();
            Two sum = two(0.0f, 0.0f);
            for (int c = rank; c < w.chunks; c += split) {
                if (static_cast<int>(t.at) == place && ok) {
                    ok = wait(rows_full + 8 * rows.at, rows.full(), 20) && wait(s_full + 8 * t.at, t.full(), 20);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    tc_fence_after_sync();
                    if (ok) {
                        const int i0 = (w.c0 + c) * P.per, pos_lo = w.pos0 + i0, pos_hi = pos_lo + P.per - 1;
                        // columns with rows; whether all of them are the request's (others may hold anything)
                        const int real = min(P.per, w.n - i0) * group, end = (real + 15) / 16 * 16;
                        const bool plain = !some_none[rows.at] && (i0 + P.per <= w.n || real == end) && w.tok0 + kUnit - 1 <= pos_lo && (w.tok0 > pos_hi - window || w.tok0 + kUnit <= a.sinks);
                        const int cut = (end / 2 + 15) / 16 * 16, c0 = mine >> 1 ? cut : 0, c1 = mine >> 1 ? end : cut;        // the warp's columns
                        const float* data = reinterpret_cast<const float*>(smem + S::kRowData) + rows.at * 2 * kCols;
                        const uint32_t ts = tmem + t.at * (NG * kCols) + lanes;
                        if (plain) sum = chunk_sum<D, false>(sum, ts, d, P.w.scale_log2, data, c0, c1, tok, window, a.sinks);
                        else sum = chunk_sum<D, true>(sum, ts, d, P.w.scale_log2, data, c0, c1, tok, window, a.sinks);
                    }
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(s_empty + 8 * t.at);
                        mbar_arrive(rows_empty + 8 * rows.at);
                    }
                }
                t.step();
                rows.step();
            }
            if (!ok) *abort = 1u;
            const float2 both = apart(sum);
            // a token's four sums: two places in turn, so that one barrier a unit is enough; the
            // order does not depend on which place of S the unit's first chunk had
            float* part = parts + (n & 1) * 4 * kUnit + token;
            part[mine * kUnit] = ok ? both.x + both.y : __int_as_float(0x7FFFFFFF);
            sums_sync();
            if (mine != 0) continue;
            float all = (part[0] + part[2 * kUnit]) + (part[kUnit] + part[3 * kUnit]);
            if (split > 1) {
                // the second block's goes to the first, in two places in turn
                const uint32_t at = n & 1u, turn = n >> 1;
                const uint32_t slot = base + S::kOther + (at * kUnit + token) * 4;
                if (rank == 1) {
                    if (turn > 0 && ok) ok = __all_sync(0xFFFFFFFFu, wait_cluster(x_empty + 8 * at, (turn - 1) & 1u, limit, abort));
                    store_to_block(slot, 0, ok ? all : __int_as_float(0x7FFFFFFF));
                    __syncwarp();
                    if (lane == 0) arrive_at_block(x_full + 8 * at, 0);
                } else {
                    if (ok) ok = __all_sync(0xFFFFFFFFu, wait_cluster(x_full + 8 * at, turn & 1u, limit, abort));
                    all = ok ? all + *reinterpret_cast<const float*>(smem + S::kOther + (at * kUnit + token) * 4) : __int_as_float(0x7FFFFFFF);
                    __syncwarp();
                    if (lane == 0) arrive_at_block(x_empty + 8 * at, 1);
                }
                if (!ok) *abort = 1u;
            }
            if (rank == 0 && to >= 0) a.out[to] = before + all;
        }
        if (!listed) *abort = 1u;
        // where the list gave up: NaN for the units behind
        if (!listed && mine == 0 && rank == 0)
            for (; unit_of_turn(n, blockIdx.x / split, gridDim.x / split) < scan[kThreads]; ++n) {
                Unit w;
                look_up(P, scan, each, unit_of_turn(n, blockIdx.x / split, gridDim.x / split), &w);
                const int tok = w.tok0 + token, page = w.page[token / kKvTokens];
                if (tok < w.len && page >= 0)
                    a.out[((static_cast<int64_t>(page) * cache.heads + w.h) << cache.page_shift) + (tok & (cache.page_size - 1))] = __int_as_float(0x7FFFFFFF);
            }
    }
    // ------------------------------------------------------------ teardown --
    tc_fence_before_sync();
    __syncthreads();
    if (threadIdx.x == 0 && P.w.status && *abort) atomicCAS(P.w.status, 0u, static_cast<uint32_t>(PN_ETIMEOUT));
    if (warp == kThreads / 32 - 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, S::kTmemCols);
    }
    if (split > 1) cluster_sync();             // no block leaves while the other may still write to it
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
    static EncodeTiledFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess || q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiledFn>(p);
    }();
    return fn;
}

template <int D>
cudaError_t launch(const WeighParams& W, int num_sms, cudaStream_t s) {
    using S = Shape<D>;
    Params P{};
    P.w = W;
    P.per = S::kCols / W.group;
    // queries as [tokens][heads][D], rows at q_stride; what lies behind the last token reads as zero
    EncodeTiledFn fn = encode_tiled();
    const cuuint64_t dims[3] = {D, static_cast<cuuint64_t>(W.a.heads), static_cast<cuuint64_t>(W.a.tokens)};
    const cuuint64_t strides[2] = {D * 2, static_cast<cuuint64_t>(W.a.q_stride) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(W.group), static_cast<cuuint32_t>(P.per)}, element[3] = {1, 1, 1};
    if (!fn || fn(&P.qmap, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<__half*>(W.a.q), dims, strides, box, element, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> smem_set{0};
    if (cudaError_t e = set_smem_limit_once(weigh_tc_kernel<D>, S::kBytes, smem_set); e != cudaSuccess) return e;
    // two blocks to a unit where each has some chunks of it
    const int64_t rows = static_cast<int64_t>(W.a.max_queries) * W.group;
    P.split = rows >= 8 * S::kCols && num_sms > 1 ? 2 : 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(num_sms / P.split * P.split);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::kBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = P.split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, weigh_tc_kernel<D>, P);
}

}  // namespace

// By the rows of a call, as if every request had max_queries queries.
bool weigh_tc_takes(const WeighArgs& a, const KvGeometry& g) {
    const int group = a.heads / g.heads, cols = g.D == 256 ? Shape<256>::kCols : Shape<128>::kCols;
    const int64_t rows = static_cast<int64_t>(a.max_queries) * group;
    return group <= cols && rows > weigh_few_rows(g.D);
}

cudaError_t launch_weigh_tc(const WeighParams& P, int num_sms, cudaStream_t s) {
    if (P.cache.D == 64) return launch<64>(P, num_sms, s);
    return P.cache.D == 128 ? launch<128>(P, num_sms, s) : launch<256>(P, num_sms, s);
}

}  // namespace pn
