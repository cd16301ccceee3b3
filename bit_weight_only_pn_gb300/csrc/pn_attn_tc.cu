// pn_attn_tc.cu -- attention over the 4-bit cache for many query rows to a
// key/value head (prompts, long drafts): the same function as pn_attn.cu, on
// the fifth-generation tensor cores.
//
// A segment is (request, row tile, key/value head): 128 rows, the query heads
// that share the head times as many whole tokens as fit.  Its visible cached
// tokens are taken 64 at a time (32 for heads of 256).  In a thread block of 16
// warps
//   warp 14 copies records into a raw ring (bulk copies, a lane to a stage);
//   warps 8-13 decode them into fp16 whole numbers n - 8, exact, K and V as
//     [token][64 values] tiles with the 128-byte swizzle, and the scales as
//     fp32; a tile's codes are decoded once for 128 rows;
//   warp 15 issues the products: S_j = Q_j K_j^T for each group j of 64 values
//     (fp32 in tensor memory, M = 128, N = 64 or 32), O_j += P_j V_j with P_j
//     from tensor memory and V as its token-major tile;
//   warps 0-7 take the tiles, half a tile's tokens of a row to a thread: x =
//     sum_j d_j S_j, the online softmax, P_j = p d_j rounded once to fp16,
//     written over S.  For heads of 64 and 128 the halves keep references, sums
//     and O's of their own, so they never wait for each other, and are joined at
//     the end of a segment; two O's of 256 columns do not fit tensor memory beside
//     S, so there the two warps that share rows agree on a reference, by a vote
//     per tile and maxima through shared memory when it moves.  S has two places,
//     so one tile's scores are made while the other's probabilities are worked out.
// The scales of K and V never touch the operands, so scores and values are as
// exact as in the kernel for few rows; P_j takes the place of one P because V's
// scale differs by group.
//
// The reference of a row is its maximum of x + log2 of the tile's largest V
// scale (of each token's own where some are hidden), less 7, and stays until that
// maximum lies 15 above it: p d < 2^15, and O is hardly ever rescaled.
//
// What it is bound by (heads of 128, 4096 queries over 8192 tokens, 32 heads: 691
// us): a softmax warp's chain of 1900 cycles a tile, of which 490 are waits and
// set-up, 1070 scores, exponentials and P, the rest stores and the segment's end;
// the 16 products of a tile take 640 (S reads 6 KB of shared memory each, 48
// cycles; O 32), and the decode warps wait three quarters of the time.  16
// softmax warps of 16 tokens took 774 us: what a warp does once a tile is then
// done twice as often.
//
// Work split: as in pn_attn.cu, units (segment, tile) in order, a contiguous
// range to each of one thread block per SM (of fewer where the joins would cost
// more than they save); what crosses block boundaries is joined by the last block
// to arrive, in block order, by all its warps: 16 loads of 16 bytes on their way
// in every thread (with half the warps and 8 loads, 512 rows in 8192 tokens took
// 88 us, now 60).
#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "pn_attn.cuh"
#include "pn_tcgen05.cuh"

namespace pn {
namespace {

constexpr int kRows = 128;                     // MMA M
constexpr int kThreads = 16 * 32;              // 128 registers each
constexpr int kPlaces = 2;                     // of S in tensor memory, 128 columns each
constexpr int kDecodeWarps = 6;
constexpr int kSoftmaxThreads = 256;
constexpr int kRawStages = 4;
constexpr uint32_t kNap = 100;                 // nanoseconds between polls of the warps that work ahead: polling took a third of all instructions
constexpr uint32_t kTmemCols = 512;            // two places of S (P over it), O of either half
constexpr uint32_t kTmemO = kPlaces * 128;
constexpr float kMargin = 7.0f, kSlack = 15.0f;
constexpr uint32_t kIssued = 1u << 8, kOddTurn = 1u << 9;   // marks beside a raw stage's records

// What differs by head size: tensor memory holds two places of S and the O's, so
// heads of 256 have tiles of 32 tokens and one reference and O to a row, of which
// two warps have 16 tokens each.
template <int D>
struct Shape {
    static constexpr int kGroups = D / 64;
    static constexpr int kTile = D == 256 ? 32 : 64;                       // tokens per unit, MMA N of S
    static constexpr int kRecords = kTile / kKvTokens;
    static constexpr int kPart = kTile / 2;                                // tokens of a softmax thread
    static constexpr int kStates = D == 256 ? 1 : 2;                       // references and O's of a row
    static constexpr int kBufs = D == 256 ? 3 : 4;                         // decoded tiles
    static constexpr uint32_t kAll = (1u << kRecords) - 1;
};

// fp32 accumulators, fp16 operands, M = 128; S: N = a tile's tokens, B K-major; O: N = 64, B MN-major (bit 16).
__host__ __device__ constexpr uint32_t desc_s(int tile) { return (1u << 4) | (static_cast<uint32_t>(tile >> 3) << 17) | (static_cast<uint32_t>(kRows >> 4) << 24); }
constexpr uint32_t kDescO = (1u << 4) | (1u << 16) | (8u << 17) | (static_cast<uint32_t>(kRows >> 4) << 24);

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %3, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %4, p;\n\t}"
        :: "r"(d), "l"(a), "l"(b), "r"(static_cast<uint32_t>(accumulate)), "r"(desc) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t desc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %3, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %4, p;\n\t}"
        :: "r"(d), "r"(a), "l"(b), "r"(static_cast<uint32_t>(accumulate)), "r"(desc) : "memory");
}
// One lane of the converged warp: products issued under it keep their operands
// in uniform registers (issued by a lone diverged lane they took 47 cycles each
// where the tensor cores take 40).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// The two warps that share rows (barriers 3 - 6, by quadrant): has either a reason?
// Scores that either has loaded before may be written over behind it.
__device__ __forceinline__ bool pair_any(int pair, bool v) {
    uint32_t r;
    tc_fence_before_sync();
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbarrier.cta.red.or.pred q, %1, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r) : "r"(3 + pair), "r"(static_cast<uint32_t>(v)) : "memory");
    tc_fence_after_sync();
    return r != 0;
}
__device__ __forceinline__ void pair_sync(int pair) { asm volatile("bar.sync %0, 64;" :: "r"(3 + pair) : "memory"); }

__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 2, %0;" :: "n"(kSoftmaxThreads) : "memory"); }
// A request, one of its row tiles, and walking over them.
template <int kTile>
struct Walk {
    int b, qt, h, idx;         // request, row tile, head, tile of the segment
    int n, q0, pos0, len;      // the request's queries, their first row and position, cached tokens
    int qtiles;
    int t0, nt;                // the row tile's tokens
    int pos_lo, pos_hi;
    int lo_tile, sink_tiles, tiles;

    __device__ __forceinline__ void request(const AttnParams& P, int per) {
        const AttnArgs& a = P.a;
        const int T = static_cast<int>(a.tokens);
        q0 = min(max(a.starts[b], 0), T);
        n = min(min(max(a.starts[b + 1], q0), T) - q0, a.max_queries);
        const int64_t room = static_cast<int64_t>(a.max_pages) << P.cache.page_shift;
        len = static_cast<int>(min(static_cast<int64_t>(max(a.lens[b], 0)), room));
        pos0 = len - n;
        qtiles = (n + per - 1) / per;
    }
    __device__ __forceinline__ void row_tile(const AttnParams& P, int per) {
        t0 = qt * per;
        nt = min(per, n - t0);
        pos_lo = pos0 + t0;
        pos_hi = pos_lo + nt - 1;
        const int end_tile = (max(pos_hi + 1, 0) + kTile - 1) / kTile;
        const int lo = P.a.window ? window_first(pos_lo, P.a.window) : 0;
        lo_tile = lo / kTile;
        sink_tiles = P.a.window ? min((P.a.sinks + kTile - 1) / kTile, lo_tile) : 0;
        tiles = max(end_tile - lo_tile + sink_tiles, 1);
    }
    // units of the request
    __device__ __forceinline__ uint32_t units(const AttnParams& P, int per) {
        uint32_t u = 0;
        for (qt = 0; qt < qtiles; ++qt) {
            row_tile(P, per);
            u += static_cast<uint32_t>(tiles);
        }
        return u * P.cache.heads;
    }
    __device__ __forceinline__ int first_token() const { return (idx < sink_tiles ? idx : lo_tile + idx - sink_tiles) * kTile; }
    // the next segment; one follows
    __device__ __forceinline__ void next(const AttnParams& P, int per) {
        idx = 0;
        if (++h < P.cache.heads) return;
        h = 0;
        if (++qt >= qtiles) {
            qt = 0;
            do {
                ++b;
                request(P, per);
            } while (qtiles == 0);
        }
        row_tile(P, per);
    }
};

// The segment and tile of unit u; scan: units before each thread's `each` requests.
template <int kTile>
__device__ __noinline__ Walk<kTile> locate_unit(const AttnParams& P, int per, const uint32_t* scan, int each, uint32_t u) {
    Walk<kTile> w;
    int lo = 0, hi = kThreads - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (scan[mid] <= u) lo = mid;
        else hi = mid - 1;
    }
    uint32_t at = scan[lo];
    w.b = lo * each;
    w.request(P, per);
    for (w.qt = 0;; ++w.qt) {
        while (w.qt >= w.qtiles) {
            w.qt = 0;
            ++w.b;
            w.request(P, per);
        }
        w.row_tile(P, per);
        const uint32_t units = static_cast<uint32_t>(w.tiles) * P.cache.heads;
        if (u < at + units) break;
        at += units;
    }
    w.h = static_cast<int>((u - at) / static_cast<uint32_t>(w.tiles));
    w.idx = static_cast<int>(u - at - static_cast<uint32_t>(w.h) * w.tiles);
    return w;
}

template <int D>
struct Smem : Shape<D> {
    using S = Shape<D>;
    static constexpr int kGroups = S::kGroups, kTile = S::kTile, kBufs = S::kBufs;
    static constexpr int kQ = 0;                                           // [group][128 rows][128 bytes]
    static constexpr int kKv = kQ + kGroups * kRows * 128;                 // [buffer][K, V][group][64 tokens][128 bytes]
    static constexpr int kKvBytes = 2 * kGroups * kTile * 128;
    static constexpr int kScales = kKv + kBufs * kKvBytes;                 // [buffer][K scales of each group, V scales][64 tokens] floats
    static constexpr int kScaleBytes = kTile * 2 * kGroups * 4;
    static constexpr int kRaw = kScales + kBufs * kScaleBytes;             // [stage][4 records]
    static constexpr int kRawBytes = S::kRecords * kv_record_bytes(D);
    static constexpr int kSums = kRaw + kRawStages * kRawBytes;            // [2][rows] (reference, sum)
    static constexpr int kMax = kSums + 2 * kRows * 8;                     // [quadrant][2][32] maxima of warps that share rows
    static constexpr int kTop = kMax + 4 * 2 * 32 * 4;                     // [buffer][record] largest V scale (bits)
    static constexpr int kHave = kTop + kBufs * S::kRecords * 4;                    // [buffer] records that a page holds
    static constexpr int kValid = kHave + kBufs * 4;                       // [raw stage] the same, marks of its last copy
    static constexpr int kBars = (kValid + kRawStages * 4 + 7) / 8 * 8;
    static constexpr int kNumBars = 2 * kRawStages + 2 * kBufs + 1 + 3 * kPlaces + 1 + 1;
    static constexpr int kMisc = kBars + kNumBars * 8;                     // TMEM base, abort, last-block flags, shared segments
    static constexpr int kScan = kMisc + 32;                               // [threads + 1] units before each thread's requests
    static constexpr int kUsed = kScan + (kThreads + 1) * 4;
    static constexpr int kBytes = kUsed + 1024;                            // slack to align to 1024 bytes
    static_assert(kBytes <= 227 * 1024, "fits one SM's shared memory");
    static_assert(kScales % 16 == 0 && kRaw % 16 == 0 && kSums % 16 == 0 && kTop % 16 == 0, "alignment");
};

// Floats of a piece: [D / 4][rows] fours, then (reference, sum) per row.
template <int D>
constexpr int kPiece = kRows * (D + 2);

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

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// log2 of a scale's size, from fp16's least (which stands for zero too) to its largest.
__device__ __forceinline__ float log2_scale(float v) { return lg2(fminf(fmaxf(v, 5.9604645e-8f), 65504.0f)); }

// Half a tile's scores of a row, from tensor memory at ts.  sc: the tile's
// scales from the half's first token on, [K by group, V by group][a tile's
// tokens].  Hidden tokens (bits of seen that are 0) score -inf.  Returns the largest.
template <int D, bool kMasked>
__device__ __forceinline__ float half_scores(Two (&x)[Shape<D>::kPart / 2], uint32_t ts, const float* sc, uint32_t seen) {
    constexpr int NG = D / 64, kTile = Shape<D>::kTile, kWide = Shape<D>::kPart / 16;
    float top[2] = {-INFINITY, -INFINITY};
    uint32_t s[kWide][NG][16];
#pragma unroll
    for (int c = 0; c < kWide; ++c)
#pragma unroll
        for (int j = 0; j < NG; ++j) tmem_ld16(ts + kTile * j + 16 * c, s[c][j]);
    tmem_wait_ld();
#pragma unroll
    for (int c = 0; c < kWide; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) {                  // four tokens
            Two a, b;
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                const ulonglong2 d = *reinterpret_cast<const ulonglong2*>(sc + j * kTile + 16 * c + 4 * i);
                const Two s0 = two(s[c][j][4 * i], s[c][j][4 * i + 1]), s1 = two(s[c][j][4 * i + 2], s[c][j][4 * i + 3]);
                a = j ? fma2(d.x, s0, a) : mul2(d.x, s0);
                b = j ? fma2(d.y, s1, b) : mul2(d.y, s1);
            }
            float2 u = apart(a), v = apart(b);
            if constexpr (kMasked) {
                const uint32_t m = seen >> (16 * c + 4 * i);
                u.x = m & 1u ? u.x : -INFINITY;
                u.y = m & 2u ? u.y : -INFINITY;
                v.x = m & 4u ? v.x : -INFINITY;
                v.y = m & 8u ? v.y : -INFINITY;
                a = two(u.x, u.y);
                b = two(v.x, v.y);
            }
            top[0] = max3(top[0], u.x, u.y);
            top[1] = max3(top[1], v.x, v.y);
            x[8 * c + 2 * i] = a;
            x[8 * c + 2 * i + 1] = b;
        }
    return fmaxf(top[0], top[1]);
}

// The largest score with the log2 of its token's largest V scale added: for tiles
// with hidden tokens, whose scales may be anything and must not set a reference.
template <int D>
__device__ __forceinline__ float top_with_scale(const Two (&x)[Shape<D>::kPart / 2], const float* sc) {
    constexpr int NG = D / 64, kTile = Shape<D>::kTile;
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < Shape<D>::kPart / 2; ++i) {
        float2 most = make_float2(0.0f, 0.0f);         // (NaN: none)
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const float2 d = *reinterpret_cast<const float2*>(sc + (NG + j) * kTile + 2 * i);
            most = make_float2(fmaxf(most.x, fabsf(d.x)), fmaxf(most.y, fabsf(d.y)));
        }
        const float2 v = apart(x[i]);
        top = max3(top, v.x + log2_scale(most.x), v.y + log2_scale(most.y));
    }
    return top;
}

// The probabilities of the same tokens by group, to tensor memory at tp; their
// sum (before V's scales) is added to sum.
template <int D, bool kMasked>
__device__ __forceinline__ void half_probabilities(const Two (&x)[Shape<D>::kPart / 2], uint32_t tp, const float* sc, uint32_t seen, float ref,
                                                   float& sum) {
    constexpr int NG = D / 64, kTile = Shape<D>::kTile, kPart = Shape<D>::kPart;
    const float less = ref == -INFINITY ? 0.0f : -ref;
    const Two less2 = two(less, less);
    Two part[2] = {two(sum, 0.0f), two(0.0f, 0.0f)};
    uint32_t p[NG][kPart / 2];
#pragma unroll
    for (int i = 0; i < kPart / 4; ++i) {              // four tokens
        Two e[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float2 v = apart(add2(x[2 * i + k], less2));
            e[k] = two(ex2(v.x), ex2(v.y));
            part[k] = add2(part[k], e[k]);
        }
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const ulonglong2 d = *reinterpret_cast<const ulonglong2*>(sc + (NG + j) * kTile + 4 * i);
            float2 a = apart(mul2(d.x, e[0])), b = apart(mul2(d.y, e[1]));
            if constexpr (kMasked) {                   // a hidden token's scale may be anything, NaN too
                const uint32_t m = seen >> (4 * i);
                a.x = m & 1u ? a.x : 0.0f;
                a.y = m & 2u ? a.y : 0.0f;
                b.x = m & 4u ? b.x : 0.0f;
                b.y = m & 8u ? b.y : 0.0f;
            }
            p[j][2 * i] = pack_half2(a.x, a.y);
            p[j][2 * i + 1] = pack_half2(b.x, b.y);
        }
    }
#pragma unroll
    for (int j = 0; j < NG; ++j) {
        if constexpr (kPart == 32) tmem_st16(tp + 16 * j, p[j]);
        else tmem_st8(tp + 16 * j, p[j]);
    }
    const float2 both = apart(add2(part[0], part[1]));
    sum = both.x + both.y;
}

struct RowState {
    float ref, sum;
    bool ok;                   // no wait has run out
};

// Half a tile of a row: S at ts, P to tp, O (of one state: the warp's share of it)
// at to.  most: the pair's place for maxima.  before, parity: the barrier phase by
// which the last product into O is done (0: O holds nothing yet).
template <int D, bool kMasked>
__device__ __forceinline__ RowState half_tile(RowState st, uint32_t ts, uint32_t tp, uint32_t to, const float* sc, float big, uint32_t seen,
                                              float* most, uint32_t before, uint32_t parity, uint64_t limit_ns, volatile uint32_t* abort) {
    using S = Shape<D>;
    Two x[S::kPart / 2];
    float top = half_scores<D, kMasked>(x, ts, sc, seen);
    if constexpr (kMasked) top = top_with_scale<D>(x, sc);
    else top += big;
    // the reference moves when it is passed by far
    auto far = [&]() { return top > st.ref + kSlack || (st.ref == -INFINITY && top > -INFINITY); };
    const int lane = threadIdx.x & 31, half = (threadIdx.x >> 7) & 1, pair = (threadIdx.x >> 5) & 3;
    if (S::kStates == 2 ? __any_sync(0xFFFFFFFFu, far()) : pair_any(pair, far())) {
        if constexpr (S::kStates == 1) {
            most[half * 32 + lane] = top;
            pair_sync(pair);
            top = fmaxf(top, most[(half ^ 1) * 32 + lane]);
        }
        const float ref = far() ? top - kMargin : st.ref;
        const float f = st.ref == -INFINITY ? 0.0f : ex2(st.ref - ref);
        st.ref = ref;
        st.sum *= f;
        if (before) {
            if (st.ok) st.ok = __all_sync(0xFFFFFFFFu, wait_phase(before, parity, limit_ns, abort));
            tc_fence_after_sync();
#pragma unroll 1
            for (int c = 0; c < D * S::kStates / 2; c += 16) {
                uint32_t o[16];
                tmem_ld16(to + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                tmem_st16(to + c, o);
            }
        }
    }
    half_probabilities<D, kMasked>(x, tp, sc, seen, st.ref, st.sum);
    return st;
}

// The same for tiles with hidden tokens, a call of its own: few tiles are, and
// with its code beside the other's in the loop every tile took a fifth longer.
template <int D>
__device__ __noinline__ RowState half_tile_masked(RowState st, uint32_t ts, uint32_t tp, uint32_t to, const float* sc, float big, int tok,
                                                  uint32_t have, int pos, int window, int sinks, float* most, uint32_t before,
                                                  uint32_t parity, uint64_t limit_ns, volatile uint32_t* abort) {
    uint32_t seen = 0;
#pragma unroll
    for (int c = 0; c < Shape<D>::kPart; ++c) {
        const bool s = ((have >> (c / 16)) & 1u) && tok + c <= pos && (tok + c > pos - window || tok + c < sinks);
        seen |= static_cast<uint32_t>(s) << c;
    }
    return half_tile<D, true>(st, ts, tp, to, sc, big, seen, most, before, parity, limit_ns, abort);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_tc_kernel(const __grid_constant__ AttnParams P) {
    using M = Smem<D>;
    constexpr int NG = M::kGroups, kTile = M::kTile, kTileRecords = M::kRecords, kBufs = M::kBufs, kPart = M::kPart, kStates = M::kStates;
    using Walk = Walk<kTile>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = smem_addr(smem_raw), base = (raw_base + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw_base);
    uint32_t bar = base + M::kBars;
    auto take = [&](int n) { const uint32_t b = bar; bar += 8u * n; return b; };
    const uint32_t raw_full = take(kRawStages), raw_empty = take(kRawStages), kv_full = take(kBufs), kv_empty = take(kBufs);
    const uint32_t q_full = take(1), s_full = take(kPlaces), p_ready = take(2 * kPlaces), o_full = take(1), drain = take(1);
    volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + M::kMisc);
    volatile uint32_t* abort = misc + 1;
    volatile uint32_t* last_flag = misc + 2;           // [2]
    volatile uint32_t* shared = misc + 4;              // [2] first units of segments of other blocks too, [2] their tiles
    volatile uint32_t* valid = reinterpret_cast<volatile uint32_t*>(smem + M::kValid);
    volatile uint32_t* have_of = reinterpret_cast<volatile uint32_t*>(smem + M::kHave);
    uint32_t* scan = reinterpret_cast<uint32_t*>(smem + M::kScan);
    const AttnArgs& a = P.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = kRows / P.group;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kRawStages; ++s) {
            mbar_init(raw_full + 8 * s, 1);
            mbar_init(raw_empty + 8 * s, kTileRecords);
            valid[s] = 0u;
        }
        for (int s = 0; s < kBufs; ++s) {
            mbar_init(kv_full + 8 * s, kTileRecords);
            mbar_init(kv_empty + 8 * s, 1);
        }
        mbar_init(q_full, kSoftmaxThreads / 32);
        for (int w = 0; w < kPlaces; ++w) {
            mbar_init(s_full + 8 * w, 1);
            mbar_init(p_ready + 16 * w, 8 / kStates);      // of either state
            mbar_init(p_ready + 16 * w + 8, 8 / kStates);
        }
        mbar_init(o_full, 1);
        mbar_init(drain, 1);
        *abort = 0u;
        fence_mbar_init();
    }
    if (warp == 15) {
        tmem_alloc(base + M::kMisc, kTmemCols);
        tmem_relinquish();
    }
    // units before each thread's share of the requests
    const int each = (a.batch + kThreads - 1) / kThreads;
    uint32_t segments = 0;
    {
        uint32_t* warp_sums = reinterpret_cast<uint32_t*>(smem + M::kSums);
        const int b0 = min(static_cast<int>(threadIdx.x) * each, a.batch), b1 = min(b0 + each, a.batch);
        Walk w{};
        uint32_t mine = 0, segs = 0;
        for (w.b = b0; w.b < b1; ++w.b) {
            w.request(P, per);
            mine = add_units(mine, w.units(P, per));
            segs += static_cast<uint32_t>(w.qtiles) * P.cache.heads;
        }
        uint32_t in = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, in, d);
            if (lane >= d) in = add_units(in, o);
        }
        segs = __reduce_add_sync(0xFFFFFFFFu, segs);
        if (lane == 31) {
            warp_sums[warp] = in;
            warp_sums[kThreads / 32 + warp] = segs;
        }
        __syncthreads();
        uint32_t at = in - mine;
        for (int i = 0; i < warp; ++i) at = add_units(at, warp_sums[i]);
        for (int i = 0; i < kThreads / 32; ++i) segments += warp_sums[kThreads / 32 + i];
        scan[threadIdx.x] = at;
        if (threadIdx.x == kThreads - 1) scan[kThreads] = all_units(P, add_units(at, mine));
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = misc[0];
    const uint32_t total = scan[kThreads];
    // A block shares a segment of T tiles for no less than sqrt(T D / 256) of them:
    // a tile takes about a microsecond, and so does the join of a part for every 256
    // values of a head, which one block does for all parts.
    const float tiles = static_cast<float>(total) / static_cast<float>(max(segments, 1u));
    const uint32_t least = max(static_cast<uint32_t>(sqrtf(tiles * (D / 256.0f))), 1u);
    const uint32_t blocks = min(gridDim.x, max(total / least, 1u));
    const bool idle = blockIdx.x >= min(blocks, total);
    const uint32_t u0 = idle ? 0 : static_cast<uint32_t>(static_cast<uint64_t>(total) * blockIdx.x / blocks);
    const uint32_t u1 = idle ? 0 : static_cast<uint32_t>(static_cast<uint64_t>(total) * (blockIdx.x + 1) / blocks);
    auto locate = [&](uint32_t u, Walk& w) { w = locate_unit<kTile>(P, per, scan, each, u); };
    auto block_slot = [&](uint32_t c, bool begins) { return P.block_slots + (2 * static_cast<int64_t>(c) + begins) * kPiece<D>; };
    auto give_up = [&]() {
        *abort = 1u;
        atomicCAS(P.status, 0u, kAttnTimeout);
    };

    if (warp == 14) {
        // ------------------------------------------------------- producer --
        const uint32_t count = u1 - u0;
        if (lane < kRawStages && static_cast<uint32_t>(lane) < count) {
            Walk w;
            locate(u0 + lane, w);
            int tok0 = 0, page[kTileRecords];
            auto look = [&]() {                // the current unit's pages
                tok0 = w.first_token();
                const int records = min(max((w.len - tok0 + kKvTokens - 1) / kKvTokens, 0), kTileRecords);
                const int32_t* row = a.table + static_cast<int64_t>(w.b) * a.table_stride;
#pragma unroll
                for (int i = 0; i < kTileRecords; ++i) page[i] = i < records ? row[(tok0 + i * kKvTokens) >> P.cache.page_shift] : -1;
            };
            look();
            uint32_t turn = 0, n = lane;
            int64_t t0 = 0;
            // Every lane polls its own stage and copies as soon as it is free: lanes
            // that left a wait one by one would meet again behind it, and four
            // stages be filled when the last of them is empty.
            for (uint32_t polls = 0; n < count; ++polls) {
                if (turn > 0 && !mbar_try_wait(raw_empty + 8 * lane, (turn - 1) & 1u)) {
                    if (polls % 64 == 63) {
                        const int64_t now = clock64();
                        if (t0 == 0) t0 = now;
                        if (*abort || now - t0 > cycles_of(P.timeout_ns)) {
                            give_up();
                            break;
                        }
                    }
                    __nanosleep(kNap);
                    continue;
                }
                uint32_t have = 0;
#pragma unroll
                for (int i = 0; i < kTileRecords; ++i) have |= static_cast<uint32_t>(page[i] >= 0 && page[i] < P.cache.pages) << i;
                // (testing aid: with stall the first unit's bytes are announced but
                // never copied; its wait can only time out)
                const bool copied = !(P.stall && n == 0);
                valid[lane] = have | (copied ? kIssued : 0u) | ((turn & 1u) ? kOddTurn : 0u);
                mbar_arrive_expect_tx(raw_full + 8 * lane, __popc(have) * kv_record_bytes(D));
                if (copied) {
                    const uint32_t dst = base + M::kRaw + lane * M::kRawBytes;
                    if (P.cache.page_size >= kTile) {  // one page holds the tile: its records follow each other
                        if (have)
                            bulk_g2s(dst, P.cache.record((static_cast<int64_t>(page[0]) << P.cache.page_shift) + (tok0 & (P.cache.page_size - 1)), w.h),
                                     __popc(have) * kv_record_bytes(D), raw_full + 8 * lane);
                    } else {
#pragma unroll
                        for (int i = 0; i < kTileRecords; ++i) {
                            if (!((have >> i) & 1)) continue;
                            const int tok = tok0 + i * kKvTokens;
                            bulk_g2s(dst + i * kv_record_bytes(D),
                                     P.cache.record((static_cast<int64_t>(page[i]) << P.cache.page_shift) + (tok & (P.cache.page_size - 1)), w.h),
                                     kv_record_bytes(D), raw_full + 8 * lane);
                        }
                    }
                }
                ++turn;
                t0 = 0;
                n += kRawStages;
                if (n < count) {
                    int idx = w.idx + kRawStages;
                    while (idx >= w.tiles) {
                        idx -= w.tiles;
                        w.next(P, per);
                    }
                    w.idx = idx;
                    look();
                }
            }
            // the last copy into the stage lands before the block ends, also after an abort
            if (valid[lane] & kIssued) wait_phase(raw_full + 8 * lane, valid[lane] & kOddTurn ? 1u : 0u, kAttnDrainNs, nullptr);
        }
        __syncwarp();
    } else if (warp == 15) {
        // ------------------------------------------------------ MMA issue --
        if (elect_one()) {
            bool ok = u0 < u1;
            uint32_t segs = 0;
            Walk w;
            if (ok) locate(u0, w);
            auto wait = [&](uint32_t b, uint32_t parity) {
                return mbar_try_wait(b, parity) || wait_phase(b, parity, P.timeout_ns, abort);
            };
            // Descriptors: the upper words are constants (stride byte offset 1024, version
            // 1, 128-byte swizzle), the lower ones address and leading byte offset.  K
            // and Q: rows of 128 bytes, K-major, 8 rows to 1024 bytes.  V the same
            // bytes as an MN-major tile, 64 values by tokens, 8 tokens to 1024; one
            // atom wide, so its leading offset is not used (set to 1024).
            constexpr uint32_t kHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
            constexpr uint32_t kStep = M::kKvBytes >> 4;
            auto desc = [](uint32_t low) { return (static_cast<uint64_t>(kHigh) << 32) | low; };
            const uint32_t q_low = ((base + M::kQ) >> 4) | (1u << 16);
            const uint32_t k_low0 = ((base + M::kKv) >> 4) | (1u << 16);
            const uint32_t v_low0 = ((base + M::kKv + NG * (kTile * 128)) >> 4) | ((1024u >> 4) << 16);
            auto scores = [&](uint32_t k, uint32_t d) {        // S = Q K^T of the tile at k
#pragma unroll
                for (int j = 0; j < NG; ++j)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_ss(d + kTile * j, desc(q_low + ((j * (kRows * 128) + kk * 32) >> 4)),
                               desc(k + ((j * (kTile * 128) + kk * 32) >> 4)), desc_s(kTile), kk != 0);
            };
            // the decoded tiles in turn: kb, kp the next S's buffer and parity, kt its
            // place; vb, vt, vp the next O's buffer, place of P and parity
            uint32_t kb = 0, kp = 0, kt = 0, vb = 0, vt = 0, vp = 0;
            auto next_scores = [&]() {
                if (!wait(kv_full + 8 * kb, kp)) return false;
                tc_fence_after_sync();
                scores(k_low0 + kb * kStep, tmem + kt * 128);
                mma_commit(s_full + 8 * kt);
                if (++kb == kBufs) { kb = 0; kp ^= 1u; }
                if (++kt == kPlaces) kt = 0;
                return true;
            };
            for (uint32_t u = u0; u < u1 && ok;) {
                const uint32_t count = min(static_cast<uint32_t>(w.tiles - w.idx), u1 - u);
                ok = wait(q_full, segs & 1u);
                tc_fence_after_sync();
                for (uint32_t i = 0; i < min(count, static_cast<uint32_t>(kPlaces)) && ok; ++i) ok = next_scores();
                for (uint32_t i = 0; i < count && ok; ++i) {
                    const uint32_t t = tmem + vt * 128, v = v_low0 + vb * kStep;
#pragma unroll
                    for (int h = 0; h < kStates; ++h) {
                        ok = wait(p_ready + 16 * vt + 8 * h, vp);
                        if (!ok) break;
                        tc_fence_after_sync();
#pragma unroll
                        for (int j = 0; j < NG; ++j)
#pragma unroll
                            for (int kk = 0; kk < 2; ++kk)
                                mma_ts(tmem + kTmemO + 128 * h + 64 * j, t + 32 * h + 16 * j + 8 * kk,
                                       desc(v + ((j * (kTile * 128) + (2 * h + kk) * 2048) >> 4)), kDescO, i > 0 || kk != 0);
                    }
                    if (!ok) break;
                    mma_commit(kv_empty + 8 * vb);
                    if (i + 1 == count) mma_commit(o_full);
                    if (++vb == kBufs) vb = 0;
                    if (++vt == kPlaces) { vt = 0; vp ^= 1u; }
                    if (i + kPlaces < count) ok = next_scores();
                }
                ++segs;
                u += count;
                if (u < u1) w.next(P, per);
            }
            if (!ok && u0 < u1) give_up();
            mma_commit(drain);                             // every product of this block finished (also after an abort)
            wait_phase(drain, 0u, kAttnDrainNs, nullptr);
        }
        __syncwarp();
    } else if (warp >= 8) {
        // --------------------------------------------------------- decode --
        // the block's records in turn, both halves of 8 tokens at once
        const int g = lane >> 2, t = lane & 3;
        constexpr int kKinds = (2 * NG + 3) / 4;           // kinds of scale (K, V by group) to a lane: lane / 8 and every fourth
        bool ok = true;
        for (uint32_t task = warp - 8; task / kTileRecords < u1 - u0; task += kDecodeWarps) {
            const uint32_t n = task / kTileRecords, rec = task % kTileRecords;
            const uint32_t s = n % kRawStages, buf = n % kBufs;
            ok = wait_phase(raw_full + 8 * s, (n / kRawStages) & 1u, P.timeout_ns, abort);
            if (ok && n >= kBufs) ok = wait_phase(kv_empty + 8 * buf, (n / kBufs - 1) & 1u, P.timeout_ns, abort, kNap);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            const uint8_t* from = smem + M::kRaw + s * M::kRawBytes + rec * kv_record_bytes(D);
            uint8_t* kt = smem + M::kKv + buf * M::kKvBytes;
            uint8_t* vt = kt + NG * (kTile * 128);
            const uint32_t have = valid[s];
            // 16-byte chunk `i` of a token's row in a group's tile, swizzled
            auto put = [&](uint8_t* tile, int token, int j, int i, uint32_t word) {
                const uint32_t sh = word >> 8;
                *reinterpret_cast<uint4*>(tile + j * (kTile * 128) + token * 128 + ((i ^ (token & 7)) << 4)) =
                    make_uint4(decode_pair<kPn4t, 0>(word, sh), decode_pair<kPn4t, 1>(word, sh), decode_pair<kPn4t, 2>(word, sh),
                               decode_pair<kPn4t, 3>(word, sh));
            };
            // every load before the first store, which might be taken to alias
            const bool real = (have >> rec) & 1;
            float scale[2][kKinds];            // the lane's, of tokens lane % 8 and 8 more
            uint32_t kw[2][2 * NG], vw[2][2 * NG];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int q = 0; q < kKinds; ++q) {
                    const int kind = (lane >> 3) + 4 * q;
                    scale[h][q] = kind < 2 * NG ? lds_half_as_float(from + (kind < NG ? kv_k_scales(D) : kv_v_scales(D)) +
                                                                    ((h * 8 + (lane & 7)) * NG + kind % NG) * 2) : 0.0f;
                }
                if constexpr (NG >= 2) {
#pragma unroll
                    for (int pl = 0; pl < NG / 2; ++pl) {
                        const uint8_t* p = from + (h * (NG / 2) + pl) * 512 + lane * 16;
                        const uint4 k4 = lds_u128(p), v4 = lds_u128(p + kv_v_codes(D));
                        kw[h][4 * pl] = k4.x; kw[h][4 * pl + 1] = k4.y; kw[h][4 * pl + 2] = k4.z; kw[h][4 * pl + 3] = k4.w;
                        vw[h][4 * pl] = v4.x; vw[h][4 * pl + 1] = v4.y; vw[h][4 * pl + 2] = v4.z; vw[h][4 * pl + 3] = v4.w;
                    }
                } else {
                    const uint8_t* p = from + h * 256 + lane * 8;
                    const uint2 k2 = lds_u64(p), v2 = lds_u64(p + kv_v_codes(D));
                    kw[h][0] = k2.x; kw[h][1] = k2.y;
                    vw[h][0] = v2.x; vw[h][1] = v2.y;
                }
            }
            // words of K: (group, which of two); of V: (group's plane, token of two, group in the plane)
            constexpr int GP = NG >= 2 ? 2 : 1;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k0 = rec * 16 + h * 8 + g, v0 = rec * 16 + h * 8 + 2 * t;
#pragma unroll
                for (int j = 0; j < NG; ++j) {
                    put(kt, k0, j, 2 * t, kw[h][2 * j]);
                    put(kt, k0, j, 2 * t + 1, kw[h][2 * j + 1]);
                    put(vt, v0, j, g, vw[h][j / GP * 2 * GP + j % GP]);
                    put(vt, v0 + 1, j, g, vw[h][j / GP * 2 * GP + GP + j % GP]);
                }
            }
            // scales: K by scale * log2 e, V; none where no page holds the record
            float* sc = reinterpret_cast<float*>(smem + M::kScales + buf * M::kScaleBytes) + rec * 16 + (lane & 7);
            uint32_t top = 0u;                 // (NaN: none)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int q = 0; q < kKinds; ++q) {
                    const int kind = (lane >> 3) + 4 * q;
                    if (kind < 2 * NG) sc[kind * kTile + 8 * h] = !real ? 0.0f : kind < NG ? scale[h][q] * P.scale_log2 : scale[h][q];
                    if (real && kind >= NG) top = max(top, __float_as_uint(fmaxf(fabsf(scale[h][q]), 0.0f)));
                }
            const uint32_t most = __reduce_max_sync(0xFFFFFFFFu, top);
            if (lane == 0) {
                reinterpret_cast<uint32_t*>(smem + M::kTop)[buf * kTileRecords + rec] = most;
                if (rec == 0) have_of[buf] = have & M::kAll;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(kv_full + 8 * buf);
                mbar_arrive(raw_empty + 8 * s);
            }
        }
        if (!ok) give_up();
    } else {
        // -------------------------------------------------------- softmax --
        const int half = warp >> 2, row = threadIdx.x & 127;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        float* pair_most = reinterpret_cast<float*>(smem + M::kMax) + (warp & 3) * 64;
        const uint32_t to_o = tmem + kTmemO + half * 128 + lanes;              // the half's O, or its columns of the one O
        float2* sums = reinterpret_cast<float2*>(smem + M::kSums);         // [2][rows] (reference, sum)
        bool ok = true;
        uint32_t segs = 0, n = 0, buf = 0, place = 0, s_turn = 0;         // n: units done; its buffer, its place of S and how often that went round
        uint32_t shared_seg[2] = {0xFFFFFFFFu, 0xFFFFFFFFu}, shared_tiles[2] = {0, 0};   // pieces of segments of other blocks too
        // a row tile's queries, swizzled; rows past them are zero
        auto load_queries = [&](const Walk& w) {
            const int rows = w.nt * P.group;
            constexpr int kEach = kRows * (D / 8) / kSoftmaxThreads;
            uint4 v[kEach];
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                const int i = threadIdx.x + k * kSoftmaxThreads, r = i / (D / 8), c = i % (D / 8);
                v[k] = make_uint4(0, 0, 0, 0);
                if (r < rows) {
                    const int tq = r / P.group;
                    v[k] = *reinterpret_cast<const uint4*>(a.q + (static_cast<int64_t>(w.q0) + w.t0 + tq) * a.q_stride +
                                                           (w.h * P.group + r - tq * P.group) * D + 8 * c);
                }
            }
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                const int i = threadIdx.x + k * kSoftmaxThreads, r = i / (D / 8), c = i % (D / 8);
                *reinterpret_cast<uint4*>(smem + M::kQ + (c >> 3) * (kRows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = v[k];
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
        };
        Walk w;
        if (u0 < u1) {
            locate(u0, w);
            load_queries(w);
        }
        for (uint32_t u = u0; u < u1;) {
            const int first = w.idx;
            const uint32_t count = min(static_cast<uint32_t>(w.tiles - first), u1 - u);
            const int rows = w.nt * P.group;
            const int lo_tile = w.lo_tile, sink_tiles = w.sink_tiles, pos_lo = w.pos_lo, pos_hi = w.pos_hi;
            const int pos = pos_lo + min(row, max(rows - 1, 0)) / P.group;
            const int window = a.window ? a.window : INT32_MAX;
            RowState st{-INFINITY, 0.0f, ok};
            uint32_t written = 0;              // barrier of the P whose stores are on their way; told when the next tile is looked at
            auto tell = [&]() {
                tmem_wait_st();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(written);
            };
            for (uint32_t i = 0; i < count; ++i) {
                bool there = st.ok && wait_phase(kv_full + 8 * buf, (n / kBufs) & 1u, P.timeout_ns, abort);
                const int idx = first + static_cast<int>(i), tok0 = (idx < sink_tiles ? idx : lo_tile + idx - sink_tiles) * kTile;
                const uint32_t ts = tmem + place * 128 + lanes;
                const float* sc = reinterpret_cast<const float*>(smem + M::kScales + buf * M::kScaleBytes) + half * kPart;
                const uint32_t* tops = reinterpret_cast<const uint32_t*>(smem + M::kTop) + buf * kTileRecords;
                float most;
                if constexpr (kTileRecords == 4) {
                    const uint4 v = *reinterpret_cast<const uint4*>(tops);
                    most = __uint_as_float(max(max(v.x, v.y), max(v.z, v.w)));
                } else {
                    const uint2 v = *reinterpret_cast<const uint2*>(tops);
                    most = __uint_as_float(max(v.x, v.y));
                }
                const float big = log2_scale(most);
                const uint32_t have = have_of[buf];
                const bool plain = have == M::kAll && tok0 + kTile - 1 <= pos_lo && (tok0 > pos_hi - window || tok0 + kTile <= a.sinks);
                if (i > 0) tell();
                there = there && wait_phase(s_full + 8 * place, s_turn & 1u, P.timeout_ns, abort);
                st.ok = __all_sync(0xFFFFFFFFu, there);
                tc_fence_after_sync();
                const uint32_t before = i > 0 ? kv_empty + 8 * ((buf + kBufs - 1) % kBufs) : 0u, parity = ((n - 1) / kBufs) & 1u;
                const uint32_t tp = ts + half * (kStates == 2 ? 32 : 8);
                if (plain)
                    st = half_tile<D, false>(st, ts + half * kPart, tp, to_o, sc, big, ~0u, pair_most, before, parity, P.timeout_ns, abort);
                else
                    st = half_tile_masked<D>(st, ts + half * kPart, tp, to_o, sc, big, tok0 + half * kPart, have >> (half * kPart / kKvTokens), pos,
                                             window, a.sinks, pair_most, before, parity, P.timeout_ns, abort);
                written = p_ready + 16 * place + (kStates == 2 ? 8 * half : 0);
                ++n;
                if (++buf == kBufs) buf = 0;
                if (++place == kPlaces) { place = 0; ++s_turn; }
            }
            tell();
            ok = st.ok;
            // every score of the segment is there, so Q may be replaced
            const Walk done = w;
            if (u + count < u1) {
                w.next(P, per);
                load_queries(w);
            }
            sums[half * kRows + row] = make_float2(st.ref, st.sum);
            if (ok) ok = wait_phase(o_full, segs & 1u, P.timeout_ns, abort);
            if (!ok) give_up();
            ++segs;
            tc_fence_after_sync();
            softmax_sync();
            // the halves' common reference and sum
            const float2 e0 = sums[row], e1 = sums[kRows + row];
            const float m = fmaxf(e0.x, e1.x);
            const float f0 = e0.x == -INFINITY ? 0.0f : ex2(e0.x - m), f1 = e1.x == -INFINITY ? 0.0f : ex2(e1.x - m);
            const float l = f0 * e0.y + f1 * e1.y;
            const bool whole = count == static_cast<uint32_t>(done.tiles);
            const int tq = row / P.group;
            const int64_t at = row < rows ? (static_cast<int64_t>(done.q0) + done.t0 + tq) * a.heads + done.h * P.group + row - tq * P.group : -1;
            float* slot = nullptr;
            if (!whole) {
                const int kind = first == 0;
                slot = block_slot(blockIdx.x, kind);
                shared_seg[kind] = u - first;
                shared_tiles[kind] = done.tiles;
                if (half == 0) reinterpret_cast<float2*>(slot + kRows * D)[row] = make_float2(m, l);
            }
            const float inv = whole ? (l == 0.0f ? 0.0f : 1.0f / l) : 1.0f;
            const float g0 = f0 * inv, g1 = f1 * inv;
            if (whole && half == 0 && a.lse && at >= 0) a.lse[at] = log_sum(m, l);
#pragma unroll 2
            for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 16) {
                uint32_t o0[16], o1[16];
                tmem_ld16(tmem + kTmemO + lanes + c, o0);
                if constexpr (kStates == 2) tmem_ld16(tmem + kTmemO + 128 + lanes + c, o1);
                tmem_wait_ld();
                float o[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    o[k] = g0 * __uint_as_float(o0[k]);
                    if constexpr (kStates == 2) o[k] = fmaf(g1, __uint_as_float(o1[k]), o[k]);
                }
                if (!whole) {
                    if (row < rows)
#pragma unroll
                        for (int k = 0; k < 16; k += 4)
                            reinterpret_cast<float4*>(slot)[((c + k) / 4) * kRows + row] = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
                } else if (at >= 0) {
                    uint4* out = reinterpret_cast<uint4*>(a.out + at * D + c);
                    out[0] = make_uint4(pack_half2(o[0], o[1]), pack_half2(o[2], o[3]), pack_half2(o[4], o[5]), pack_half2(o[6], o[7]));
                    out[1] = make_uint4(pack_half2(o[8], o[9]), pack_half2(o[10], o[11]), pack_half2(o[12], o[13]), pack_half2(o[14], o[15]));
                }
            }
            tc_fence_before_sync();                    // O has been read before the next segment's first P is told
            softmax_sync();                            // sums are written again
            u += count;
        }

        if (threadIdx.x < 2) {
            shared[threadIdx.x] = shared_seg[threadIdx.x];
            shared[2 + threadIdx.x] = shared_tiles[threadIdx.x];
        }
    }

    // ------------------------------------------- segments of several blocks --
    // Their joins by all warps: every role is through, no product or copy is on its way.
    tc_fence_before_sync();
    __syncthreads();
    if (u0 < u1) {
        auto block_of = [&](uint32_t x) {              // the block that holds unit x
            return static_cast<uint32_t>(((static_cast<uint64_t>(x) + 1) * blocks + total - 1) / total - 1);
        };
        if (threadIdx.x < 2) {
            bool last = false;
            const uint32_t seg = shared[threadIdx.x];
            if (seg != 0xFFFFFFFFu) {
                const uint32_t c0 = block_of(seg), c1 = block_of(seg + shared[2 + threadIdx.x] - 1);
                __threadfence();
                last = atomicAdd(&P.counters[c0], 1u) == c1 - c0;
                __threadfence();
                if (last) P.counters[c0] = 0u;
            }
            last_flag[threadIdx.x] = last;
        }
        __syncthreads();
        const int row = threadIdx.x & (kRows - 1), quarter = threadIdx.x / kRows;
        float* quarters = reinterpret_cast<float*>(smem);                  // [4][rows]; no product reads Q or the tiles any more
        float* factors = quarters + 4 * kRows;                             // [parts][rows]
        for (int kind = 0; kind < 2; ++kind) {
            if (!last_flag[kind]) continue;
            const uint32_t seg = shared[kind], c0 = block_of(seg), c1 = block_of(seg + shared[2 + kind] - 1);
            const int parts = static_cast<int>(c1 - c0 + 1);
            Walk w;
            locate(seg, w);
            const int rows = w.nt * P.group, tq = row / P.group;
            const int64_t at = row < rows ? (static_cast<int64_t>(w.q0) + w.t0 + tq) * a.heads + w.h * P.group + row - tq * P.group : -1;
            auto part = [&](int p) { return block_slot(c0 + p, p == 0); };
            auto part_sum = [&](int p) { return __ldcg(reinterpret_cast<const float2*>(part(p) + kRows * D) + row); };
            float m = -INFINITY, l = 0.0f;
#pragma unroll 8
            for (int p = quarter; p < parts; p += 4) m = fmaxf(m, part_sum(p).x);
            quarters[threadIdx.x] = m;
            __syncthreads();
            m = fmaxf(fmaxf(quarters[row], quarters[kRows + row]), fmaxf(quarters[2 * kRows + row], quarters[3 * kRows + row]));
            __syncthreads();
#pragma unroll 8
            for (int p = quarter; p < parts; p += 4) {
                const float2 v = part_sum(p);
                const float f = v.x == -INFINITY ? 0.0f : ex2(v.x - m);
                factors[p * kRows + row] = f;
                l += f * v.y;
            }
            quarters[threadIdx.x] = l;
            __syncthreads();
            l = (quarters[row] + quarters[kRows + row]) + (quarters[2 * kRows + row] + quarters[3 * kRows + row]);
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            if (quarter == 0 && a.lse && at >= 0) a.lse[at] = log_sum(m, l);
            if (at >= 0) {
                constexpr int kFours = D / 16 < 8 ? D / 16 : 8;            // at a time, of two parts: 16 loads on their way
                for (int c = quarter * (D / 4); c < (quarter + 1) * (D / 4); c += 4 * kFours) {
                    float4 o[kFours];
#pragma unroll
                    for (int k = 0; k < kFours; ++k) o[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 2
                    for (int p = 0; p < parts; ++p) {
                        const float4* from = reinterpret_cast<const float4*>(part(p)) + (c / 4) * kRows + row;
                        float4 v[kFours];
#pragma unroll
                        for (int k = 0; k < kFours; ++k) v[k] = __ldcg(from + k * kRows);
                        const float f = factors[p * kRows + row];
#pragma unroll
                        for (int k = 0; k < kFours; ++k) {
                            o[k].x = fmaf(f, v[k].x, o[k].x); o[k].y = fmaf(f, v[k].y, o[k].y);
                            o[k].z = fmaf(f, v[k].z, o[k].z); o[k].w = fmaf(f, v[k].w, o[k].w);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < kFours; ++k)
                        *reinterpret_cast<uint2*>(a.out + at * D + c + 4 * k) = make_uint2(pack_half2(o[k].x * inv, o[k].y * inv),
                                                                                           pack_half2(o[k].z * inv, o[k].w * inv));
                }
            }
            __syncthreads();                           // the factors are written again
        }
    }
    // ------------------------------------------------------------ teardown --
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 15) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int D>
cudaError_t launch(AttnParams P, uint8_t* ws, int num_sms, cudaStream_t s) {
    static std::atomic<uint64_t> smem_set{0};
    if (cudaError_t e = set_smem_limit_once(attn_tc_kernel<D>, Smem<D>::kBytes, smem_set); e != cudaSuccess) return e;
    P.status = reinterpret_cast<uint32_t*>(ws);
    P.counters = reinterpret_cast<uint32_t*>(ws + 256);
    P.block_slots = reinterpret_cast<float*>(ws + 256 + attn_counter_bytes(num_sms));
    constexpr int kMost = (Smem<D>::kScales - 4 * kRows * 4) / (kRows * 4);                  // blocks whose factors fit the place of Q and the tiles
    attn_tc_kernel<D><<<num_sms < kMost ? num_sms : kMost, kThreads, Smem<D>::kBytes, s>>>(P);
    return cudaGetLastError();
}

}  // namespace

// By the rows and the row tiles of the call, as if every request had max_queries
// queries: a tile of up to 128 rows costs this kernel what 62, 37 or 41 rows
// (heads of 64, 128, 256) cost the one for few rows, which takes them 16 or, of
// 256, 8 at a time, and with few tiles it loses what 1200, 600 or 1300 rows cost
// to the joins of segments that several blocks share.  Microseconds there, here:
//   8 heads of 64.  24 requests of 4096 cached tokens: 32 rows 52, 82; 64: 84, 83;
//     70: 100, 84.  One of 8192: 128 rows 28, 29; 512: 61, 46
//   8 heads of 128.  24 of 4096: 32 rows 85, 103; 40: 115, 105; 64: 148, 107.  One
//     of 8192: 64 rows 31, 31; 256: 62, 54; 512: 103, 60.  One of 1024, 128 rows: 23, 25
//   4 heads of 256.  24 of 4096: 32 rows 93, 111; 48: 129, 113; 70: 184, 117.  One
//     of 8192: 256 rows 66, 87; 512: 115, 88.  One of 1024, 256 rows: 27, 58
// It looks at no lengths, so it misses by a little where both are close (128 rows
// of 128 in 1024 tokens run here, 25 for 23; 48 rows with a window, 114 and 116),
// and a batch goes by its longest request: one of 512 queries beside 63 single
// tokens on up to 16384 cached ones, 32 + 8 heads of 128, takes 536 us in one call,
// 78 and 113 as two.
bool attn_tc_takes(const AttnArgs& a, const KvGeometry& g) {
    const int group = a.heads / g.heads;
    if (group > kRows) return false;
    const int per = kRows / group, at_once = g.D == 256 ? 8 : 16;
    const int64_t rows = (static_cast<int64_t>(a.max_queries) * group + at_once - 1) / at_once * at_once;
    const int64_t tiles = (static_cast<int64_t>(a.max_queries) + per - 1) / per;
    const int64_t tile_cost = g.D == 64 ? 62 : g.D == 128 ? 37 : 41, joins = g.D == 64 ? 1200 : g.D == 128 ? 600 : 1300;
    return static_cast<double>(a.batch) * g.heads * static_cast<double>(rows - tile_cost * tiles) > static_cast<double>(joins);
}

double attn_tc_units(const AttnArgs& a, const KvGeometry& g) {
    const int per = kRows / (a.heads / g.heads), tile = g.D == 256 ? Shape<256>::kTile : Shape<128>::kTile;
    static_assert(Shape<64>::kTile == Shape<128>::kTile, "a tile's tokens");
    const double allowed = static_cast<double>(a.batch) * static_cast<double>((static_cast<int64_t>(a.max_queries) + per - 1) / per);
    const double there = static_cast<double>(a.tokens) / per + a.batch;
    const int64_t tiles = (static_cast<int64_t>(a.max_pages) * g.page_size + tile - 1) / tile;
    return (allowed < there ? allowed : there) * g.heads * static_cast<double>(tiles);
}

size_t attn_tc_workspace_bytes(int num_sms) {
    return 256 + attn_counter_bytes(num_sms) + 2 * static_cast<size_t>(num_sms) * kPiece<256> * 4;
}

cudaError_t launch_attention_tc(AttnParams P, uint8_t* ws, int num_sms, cudaStream_t s) {
    if (P.cache.D == 256) return launch<256>(P, ws, num_sms, s);
    return P.cache.D == 64 ? launch<64>(P, ws, num_sms, s) : launch<128>(P, ws, num_sms, s);
}

}  // namespace pn
