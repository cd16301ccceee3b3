// pn_attn.cu -- attention of a step's queries over the 4-bit cache.
//
// For each query row (token, head): x_t = scale * q . k_t over the visible
// cached tokens t, out = sum_t exp(x_t) v_t / sum_t exp(x_t), lse = ln sum_t
// exp(x_t), with k_t, v_t the cache's exact values d (n - 8).
//
// One pass over the cache.  The codes enter the products as they are: four
// bits masked out of a word are the fp16 number n 2^-24 (n 2^-20 for the upper
// four of a byte), a subnormal, which the tensor cores multiply exactly.  So
// two codes cost one LOP3 (and a shift for every other pair), no conversion.
//   S: sum_d q_d (n_d - 8) = sum_d q_d n_d - 8 sum_d q_d: the second sum is
//   taken once per row and group and is the accumulator's first value; each
//   group's sum is multiplied by its scale in fp32.  The queries of a row are
//   multiplied by a power of two so that the largest lies in [2^10, 2^11), and
//   those that meet a lower four bits by 16 more.
//   O: the scales of V go into the probabilities, and 8 is taken off the codes
//   before the product (one HADD2 per pair, exact): with the 8 in the sums a
//   sharp softmax over a token whose value is 0 would leave 2^-20 of its scale
//   in place of the other tokens' share.
// The products run on mma.sync with the cache as the A operand: S^T = K Q^T
// (16 tokens x 8 query rows), O^T += V^T P^T (16 values x 8 query rows).  The
// 8 columns are the query heads that share the key/value head and the step's
// tokens, so a decode step wastes few of them, and the words of a record are
// stored in the order in which the fragments take them (pn_kv.cuh).
//
// Probabilities are rounded to fp16 once, after the scale of V is multiplied
// in: p d with p = 2^(x' - m), x' = x log2 e.  The reference m of a row is the
// running maximum of x' + log2 |d| (d the token's largest V scale) less 14, so
// p |d| stays below 2^15 whatever the scales are and keeps its 11 bits down to
// 2^-28 of the largest.  Sums, maxima and outputs are held in fp32.
//
// Work split: the units (request, key/value head, row group, 32-token tile) of
// a call are numbered in that order and every consumer warp of the grid takes
// one contiguous range of them, so the cache bytes are shared evenly whatever
// the lengths are, and a warp keeps its accumulators for as long as a segment
// (request, head, row group) lasts.  A segment counts one unit more than it has
// tiles: to start one costs a warp about what a tile does.  A producer warp
// fills each warp's own ring of stages by bulk copies.  Segments that one warp
// has to itself go straight to the output; the pieces of the others are joined
// in shared memory when the block is done, and those of several blocks through
// the workspace (L2) by the last block to arrive, in unit order, so results do
// not depend on timing.
//
// One block of 15 consumer warps to an SM.  The schedulers serve older warps
// first: of two blocks of 7 the first was done 10 us of 50 before the second,
// and half the SM idled since.  So a warp that is kLead tiles ahead of the
// block's last one waits for it.
#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "pn_attn.cuh"

namespace pn {
namespace {

constexpr int kTile = 32;                      // tokens per unit
constexpr int kTileRecords = kTile / kKvTokens;
constexpr uint32_t kSegmentUnits = 1;          // of a segment beside its tiles
constexpr int kLead = 6;                       // tiles that a warp may be ahead of its block's last one
constexpr uint32_t kIssued = 1u << 8;          // marks beside a stage's records: its copy was started,
constexpr uint32_t kOddTurn = 1u << 9;         // in an odd turn of the ring
// 8x8 transpose of 16-bit elements across the warp (row lane / 4, columns 2 (lane % 4), + 1).
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
template <int W>
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" :: "n"(W * 32) : "memory"); }

// What a request asks of the cache.
struct Request {
    int n;                     // query tokens
    int q0;                    // first of them
    int pos0;                  // position of the first
    int rows;                  // n * group
    int len;
    int lo_tile;               // first tile of the window
    int sink_tiles;            // tiles before it that hold visible first tokens
    int tiles;                 // units per (head, row group), at least 1
    int row_groups;
    __device__ __forceinline__ uint32_t units(int heads) const { return (static_cast<uint32_t>(tiles) + kSegmentUnits) * row_groups * heads; }
    __device__ __forceinline__ int tile(int idx) const { return idx < sink_tiles ? idx : lo_tile + idx - sink_tiles; }
};

template <int RT>
__device__ __forceinline__ Request request_of(const AttnParams& P, int b) {
    Request r;
    const AttnArgs& a = P.a;
    const int T = static_cast<int>(a.tokens);
    r.q0 = min(max(a.starts[b], 0), T);
    r.n = min(min(max(a.starts[b + 1], r.q0), T) - r.q0, a.max_queries);
    const int64_t room = static_cast<int64_t>(a.max_pages) << P.cache.page_shift;
    r.len = static_cast<int>(min(static_cast<int64_t>(max(a.lens[b], 0)), room));
    r.pos0 = r.len - r.n;
    r.rows = r.n * P.group;
    const int lo = a.window ? window_first(r.pos0, a.window) : 0;
    r.lo_tile = lo / kTile;
    r.sink_tiles = a.window ? min((a.sinks + kTile - 1) / kTile, r.lo_tile) : 0;
    r.tiles = max((r.len + kTile - 1) / kTile - r.lo_tile + r.sink_tiles, 1);
    r.row_groups = (r.rows + RT - 1) / RT;
    return r;
}

// Unit v of a request: (head, row group, place among its tiles; negative: one
// of the units before them).
__device__ __forceinline__ void locate(uint32_t v, const Request& r, int& h, int& rg, int& idx) {
    const uint32_t each = static_cast<uint32_t>(r.tiles) + kSegmentUnits, seg = v / each;
    idx = static_cast<int>(v - seg * each) - static_cast<int>(kSegmentUnits);
    h = static_cast<int>(seg / static_cast<uint32_t>(r.row_groups));
    rg = static_cast<int>(seg - h * r.row_groups);
}

// The segment after (r, b, h, rg), which there is.
template <int RT>
__device__ __forceinline__ void next_segment(const AttnParams& P, Request& r, int& b, int& h, int& rg) {
    if (++rg < r.row_groups) return;
    rg = 0;
    if (++h < P.cache.heads) return;
    h = 0;
    do r = request_of<RT>(P, ++b); while (r.rows == 0);
}

template <int D>
struct Shape {
    static constexpr int kGroups = D / 64;             // groups of 64 values (one scale each)
    static constexpr int kPlanes = kv_planes(D);
    static constexpr int kPlaneGroups = kv_plane_groups(D);
    static constexpr int kRecord = kv_record_bytes(D);
    static constexpr int kStage = kTileRecords * kRecord;
    static constexpr int kPlaneBytes = 256 * kPlaneGroups;     // 8 tokens of a plane
};

// Floats of a piece: rows x D values, then (reference, sum) per row.
template <int D, int NT>
constexpr int kPiece = 8 * NT * (D + 2);

template <int D, int NT>
struct Smem {
    static constexpr int kRT = 8 * NT;
    // consumer warps: with the producer 16 at 128 registers where these suffice (8 rows, D <= 128), 12 at 168 for 16 rows
    // of D = 64 (24 requests of 4096 tokens, 8 heads: 35 us, with 8 warps 40), else 8 (12 do not make 16 rows of 128 faster)
    static constexpr int kWarps = D == 256 ? 7 : NT == 1 ? 15 : D == 64 ? 11 : 7;
    static constexpr int kThreads = (kWarps + 1) * 32;
    static constexpr int kDepth = D == 256 ? 2 : D == 128 && NT == 1 ? 3 : 4;      // stages per warp
    static constexpr int kWarpRing = kDepth * Shape<D>::kStage;
    static constexpr int kRing = kWarps * kWarpRing;
    static constexpr int kPieces = 2 * kWarps;                             // pieces of segments: two to a warp
    static constexpr int kRunsMost = kWarps + 1;                           // a warp's last piece goes on in the next one's first
    static constexpr int kFactors = kRing;                                 // [pieces][rows] floats
    static constexpr int kRowOut = kFactors + kPieces * kRT * 4;           // [runs][rows] where a run's row goes
    static constexpr int kPieceOf = kRowOut + kRunsMost * kRT * 8;         // [pieces] PieceInfo
    static constexpr int kRuns = kPieceOf + kPieces * 24;                  // order [pieces], run starts [runs + 1], number of runs
    static constexpr int kBars = kRuns + (kPieces + kRunsMost + 2 + 1) / 2 * 8;    // full, empty
    static constexpr int kValid = kBars + 2 * kWarps * kDepth * 8;         // per stage: records that hold data, marks of its last copy
    static constexpr int kProgress = kValid + kWarps * kDepth * 4;         // [warps] tiles done
    static constexpr int kMisc = kProgress + kWarps * 4;                   // abort, last-block flags
    static constexpr int kScan = kMisc + 12;                               // the warps' sums, then [batch + 1] prefix sums of units
    static constexpr int kFixed = kScan + (kWarps + 1) * 4;
    static int bytes(int batch) { return kFixed + (batch + 1) * 4; }
    static_assert(kBars % 8 == 0 && kRowOut % 8 == 0 && kPieceOf % 4 == 0, "alignment");
    static_assert(2 * kPiece<D, NT> * 4 <= 2 * Shape<D>::kStage || 2 * kPiece<D, NT> * 4 <= kWarpRing, "a warp's pieces fit its stages");
    static_assert(kPieces <= 32, "a lane to a piece");
};

// A piece of a segment: the segment's first unit with a tile (kNone: no piece),
// its tiles, and whose it is.
struct PieceInfo {
    uint32_t seg;
    int tiles, q0, rows, h, rg;
};
constexpr uint32_t kNone = 0xFFFFFFFFu;

// Halves (code of token a, code of token b) of two tokens' words: the even
// codes 0, 2, 4, 6 at bits 0, 4, 8, 12 of each half, or the odd ones.
__device__ __forceinline__ uint32_t token_pair(uint32_t a, uint32_t b, bool odd) {
    return __byte_perm(a, b, odd ? 0x7632 : 0x5410);
}

// Pair I (0 .. 3) of four code pairs at bits 0, 4, 8, 12 of a word's halves, as
// fp16 numbers: n 2^-24 for I even, n 2^-20 for I odd.  `shifted` = word >> 8.
template <int I>
__device__ __forceinline__ uint32_t raw_pair(uint32_t word, uint32_t shifted) {
    return (I >= 2 ? shifted : word) & (I & 1 ? 0x00F000F0u : 0x000F000Fu);
}

// The same less 8: (n - 8) 2^-24 or (n - 8) 2^-20.
template <int I>
__device__ __forceinline__ uint32_t value_pair(uint32_t word, uint32_t shifted) {
    uint32_t d;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(raw_pair<I>(word, shifted)), "r"(I & 1 ? 0x80808080u : 0x80088008u));
    return d;
}

// D = C + A * B, m16n8k16, fp16 inputs, fp32 accumulate.
__device__ __forceinline__ void mma_from(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1, float c0, float c1, float c2, float c3) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

template <int N>
__device__ __forceinline__ void load_scales(const uint8_t* p, float (&d)[N]) {
    uint32_t w[(N + 1) / 2];
    if constexpr (N == 1) w[0] = *reinterpret_cast<const uint16_t*>(p);
    if constexpr (N == 2) w[0] = lds_u32(p);
    if constexpr (N == 4) {
        const uint2 v = lds_u64(p);
        w[0] = v.x; w[1] = v.y;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = half_bits_to_float(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu);
}

// Running state of a warp's share of a segment.  Lane (g, t) holds, for query
// columns 8 nt + 2t + c, the reference and its part of the sum, and of O the
// values 64 j + 8 g + 2 i (o[..][c]) and + 1 (o[..][2 + c]) for i = 0 .. 3.
// o is in units of 2^-24 (i even) and 2^-20 (i odd).
template <int D, int NT>
struct State {
    float ref[NT][2];
    float sum[NT][2];
    float o[NT][D / 16][4];

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            ref[n][0] = ref[n][1] = -INFINITY;
            sum[n][0] = sum[n][1] = 0.0f;
#pragma unroll
            for (int m = 0; m < D / 16; ++m) o[n][m][0] = o[n][m][1] = o[n][m][2] = o[n][m][3] = 0.0f;
        }
    }
    // the columns' whole sums, and o in units of 1
    __device__ __forceinline__ void finish() {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int d = 4; d <= 16; d <<= 1) sum[n][c] += __shfl_xor_sync(0xFFFFFFFFu, sum[n][c], d);
#pragma unroll
            for (int m = 0; m < D / 16; ++m)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[n][m][c] *= m & 1 ? 0x1p20f : 0x1p24f;
        }
    }
    __device__ __forceinline__ void scale_by(int n, float f0, float f1) {
#pragma unroll
        for (int m = 0; m < D / 16; ++m) {
            o[n][m][0] *= f0;
            o[n][m][1] *= f1;
            o[n][m][2] *= f0;
            o[n][m][3] *= f1;
        }
    }
};

// A row group's queries: lane (g, t) holds the B fragments of row 8 nt + g, and
// for its columns' rows 8 nt + 2t + c what the products start from and the
// factor from a product to the score times log2 e.
template <int D, int NT>
struct Queries {
    uint2 q[NT][D / 64][2][2];                 // [group][word of the lane's pair][MMA]
    float start[NT][D / 64][2];
    float factor[NT][2];
    int pos[NT][2];

    __device__ __forceinline__ void load(const AttnParams& P, const Request& r, int h, int row0) {
        constexpr int NG = D / 64;
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int row = min(row0 + 8 * n + g, r.rows - 1);
            const int qi = row / P.group;
            const __half* src = P.a.q + (r.q0 + qi) * P.a.q_stride + (h * P.group + row - qi * P.group) * D;
            uint4 f[NG][2];
            uint32_t top = 0;                  // the row's largest |q|, as bits: both halves of a register at once
#pragma unroll
            for (int j = 0; j < NG; ++j)
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    f[j][w] = *reinterpret_cast<const uint4*>(src + 64 * j + 16 * t + 8 * w);
                    const uint32_t v[4] = {f[j][w].x, f[j][w].y, f[j][w].z, f[j][w].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) top = __vmaxu2(top, v[i] & 0x7FFF7FFFu);
                }
            top = max(top & 0xFFFFu, top >> 16);
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            const int e = 25 - static_cast<int>(max(top >> 10, 1u));             // the largest |q| 2^e lies in [2^10, 2^11)
            const float up = __int_as_float((127 + e) << 23);
            float sum[NG];
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                sum[j] = 0.0f;
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const uint32_t v[4] = {f[j][w].x, f[j][w].y, f[j][w].z, f[j][w].w};
                    uint32_t to[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float a0 = half_bits_to_float(v[i] & 0xFFFFu) * up, a1 = half_bits_to_float(v[i] >> 16) * up;
                        sum[j] += a0 + a1;
                        to[i] = i & 1 ? pack_half2(a0, a1) : pack_half2(16.0f * a0, 16.0f * a1);
                    }
                    q[n][j][w][0] = make_uint2(to[0], to[1]);
                    q[n][j][w][1] = make_uint2(to[2], to[3]);
                }
                sum[j] += __shfl_xor_sync(0xFFFFFFFFu, sum[j], 1);
                sum[j] += __shfl_xor_sync(0xFFFFFFFFu, sum[j], 2);
            }
            const float back = P.scale_log2 * __int_as_float((127 + 20 - e) << 23);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int from = (2 * t + c) << 2;             // the columns' rows are those of lanes (2t + c, .)
#pragma unroll
                for (int j = 0; j < NG; ++j) start[n][j][c] = -0x1p-17f * __shfl_sync(0xFFFFFFFFu, sum[j], from);   // -8 * 2^-20
                factor[n][c] = __shfl_sync(0xFFFFFFFFu, back, from);
                pos[n][c] = r.pos0 + min(row0 + 8 * n + 2 * t + c, r.rows - 1) / P.group;
            }
        }
    }
};

template <int D, int NT, bool kMasked>
__device__ __forceinline__ void take_tile(const uint8_t* stage, int tok0, uint32_t valid, const Queries<D, NT>& Q, int window,
                                          int sinks, State<D, NT>& st) {
    using S = Shape<D>;
    constexpr int NG = S::kGroups, GP = S::kPlaneGroups, PL = S::kPlanes;
    const int lane = threadIdx.x & 31, g = lane >> 2;
    float x[kTileRecords][NT][4];
    float e[kTileRecords][2];                  // log2 of the tokens' largest V scale
    float top[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) top[n][0] = top[n][1] = -INFINITY;
#pragma unroll
    for (int r = 0; r < kTileRecords; ++r) {
        const uint8_t* rec = stage + r * S::kRecord;
        float dk0[NG], dk1[NG];
        load_scales<NG>(rec + kv_k_scales(D) + g * 2 * NG, dk0);
        load_scales<NG>(rec + kv_k_scales(D) + (g + 8) * 2 * NG, dk1);
#pragma unroll
        for (int n = 0; n < NT; ++n) x[r][n][0] = x[r][n][1] = x[r][n][2] = x[r][n][3] = 0.0f;
#pragma unroll
        for (int pl = 0; pl < PL; ++pl) {
            uint32_t w0[2 * GP], w1[2 * GP];   // the lane's words of tokens g and g + 8: [group][2]
            const uint8_t* p0 = rec + pl * S::kPlaneBytes + lane * 8 * GP;
            const uint8_t* p1 = p0 + PL * S::kPlaneBytes;
            if constexpr (GP == 2) {
                const uint4 u = lds_u128(p0), v = lds_u128(p1);
                w0[0] = u.x; w0[1] = u.y; w0[2] = u.z; w0[3] = u.w;
                w1[0] = v.x; w1[1] = v.y; w1[2] = v.z; w1[3] = v.w;
            } else {
                const uint2 u = lds_u64(p0), v = lds_u64(p1);
                w0[0] = u.x; w0[1] = u.y;
                w1[0] = v.x; w1[1] = v.y;
            }
#pragma unroll
            for (int jj = 0; jj < GP; ++jj) {
                const int j = pl * GP + jj;
                float acc[NT][4];
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const uint32_t a = w0[2 * jj + w], b = w1[2 * jj + w], as = a >> 8, bs = b >> 8;
                    const uint32_t a0 = raw_pair<0>(a, as), a1 = raw_pair<0>(b, bs), a2 = raw_pair<1>(a, as), a3 = raw_pair<1>(b, bs);
                    const uint32_t b0 = raw_pair<2>(a, as), b1 = raw_pair<2>(b, bs), b2 = raw_pair<3>(a, as), b3 = raw_pair<3>(b, bs);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float s0 = Q.start[n][j][0], s1 = Q.start[n][j][1];
                        const uint2 u = Q.q[n][j][w][0], v = Q.q[n][j][w][1];
                        if (w == 0) mma_from(acc[n], a0, a1, a2, a3, u.x, u.y, s0, s1, s0, s1);
                        else mma_16816(acc[n], a0, a1, a2, a3, u.x, u.y);
                        mma_16816(acc[n], b0, b1, b2, b3, v.x, v.y);
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    x[r][n][0] = fmaf(dk0[j], acc[n][0], x[r][n][0]);
                    x[r][n][1] = fmaf(dk0[j], acc[n][1], x[r][n][1]);
                    x[r][n][2] = fmaf(dk1[j], acc[n][2], x[r][n][2]);
                    x[r][n][3] = fmaf(dk1[j], acc[n][3], x[r][n][3]);
                }
            }
        }
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            float dv[NG], big = 5.9604645e-8f;      // 2^-24, the least scale: rows of V that are all zero count as it
            load_scales<NG>(rec + kv_v_scales(D) + (g + 8 * hh) * 2 * NG, dv);
#pragma unroll
            for (int j = 0; j < NG; ++j) big = fmaxf(big, fabsf(dv[j]));
            e[r][hh] = lg2(big);
        }
    }
    // which of the lane's scores are seen: bit ((r * 2 + hh) * NT + n) * 2 + c
    uint32_t seen = 0xFFFFFFFFu;
    if constexpr (kMasked) {
        seen = 0;
#pragma unroll
        for (int r = 0; r < kTileRecords; ++r)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int tok = tok0 + r * kKvTokens + hh * 8 + g;
                        const bool s = ((valid >> r) & 1) && tok <= Q.pos[n][c] && (tok > Q.pos[n][c] - window || tok < sinks);
                        seen |= static_cast<uint32_t>(s) << (((r * 2 + hh) * NT + n) * 2 + c);
                    }
    }
    auto sees = [&](int r, int hh, int n, int c) { return !kMasked || ((seen >> (((r * 2 + hh) * NT + n) * 2 + c)) & 1u); };
#pragma unroll
    for (int r = 0; r < kTileRecords; ++r)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float y = fmaf(x[r][n][2 * hh + c], Q.factor[n][c], e[r][hh]);
                    top[n][c] = fmaxf(top[n][c], sees(r, hh, n, c) ? y : -INFINITY);
                }
    bool moved = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int d = 4; d <= 16; d <<= 1) top[n][c] = fmaxf(top[n][c], __shfl_xor_sync(0xFFFFFFFFu, top[n][c], d));
            top[n][c] -= 14.0f;
            moved |= top[n][c] > st.ref[n][c];
        }
    if (__any_sync(0xFFFFFFFFu, moved)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float f[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float to = fmaxf(top[n][c], st.ref[n][c]);
                f[c] = st.ref[n][c] == -INFINITY ? 0.0f : ex2(st.ref[n][c] - to);
                st.ref[n][c] = to;
                st.sum[n][c] *= f[c];
            }
            st.scale_by(n, f[0], f[1]);
        }
    }
#pragma unroll
    for (int r = 0; r < kTileRecords; ++r) {
        const uint8_t* rec = stage + r * S::kRecord;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float p = ex2(fmaf(x[r][n][2 * hh + c], Q.factor[n][c], -st.ref[n][c]));
                    x[r][n][2 * hh + c] = sees(r, hh, n, c) ? p : 0.0f;
                    st.sum[n][c] += x[r][n][2 * hh + c];
                }
        float dv[2][NG];
        load_scales<NG>(rec + kv_v_scales(D) + g * 2 * NG, dv[0]);
        load_scales<NG>(rec + kv_v_scales(D) + (g + 8) * 2 * NG, dv[1]);
#pragma unroll
        for (int pl = 0; pl < PL; ++pl) {
            uint32_t w[2][2 * GP];             // [h][token of the pair][group]
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint8_t* p = rec + kv_v_codes(D) + (h * PL + pl) * S::kPlaneBytes + lane * 8 * GP;
                if constexpr (GP == 2) {
                    const uint4 u = lds_u128(p);
                    w[h][0] = u.x; w[h][1] = u.y; w[h][2] = u.z; w[h][3] = u.w;
                } else {
                    const uint2 u = lds_u64(p);
                    w[h][0] = u.x; w[h][1] = u.y;
                }
            }
#pragma unroll
            for (int jj = 0; jj < GP; ++jj) {
                const int j = pl * GP + jj;
                uint32_t b[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        // a hidden token's scale may be anything, NaN too: it is not multiplied
                        float p0 = x[r][n][2 * hh] * dv[hh][j], p1 = x[r][n][2 * hh + 1] * dv[hh][j];
                        if (kMasked) {
                            p0 = sees(r, hh, n, 0) ? p0 : 0.0f;
                            p1 = sees(r, hh, n, 1) ? p1 : 0.0f;
                        }
                        b[n][hh] = transpose_8x8(pack_half2(p0, p1));
                    }
                const uint32_t e0 = token_pair(w[0][jj], w[0][GP + jj], false), o0 = token_pair(w[0][jj], w[0][GP + jj], true);
                const uint32_t e1 = token_pair(w[1][jj], w[1][GP + jj], false), o1 = token_pair(w[1][jj], w[1][GP + jj], true);
                const uint32_t e0s = e0 >> 8, o0s = o0 >> 8, e1s = e1 >> 8, o1s = o1 >> 8;
                static_for<4>([&](auto ic) {
                    constexpr int I = decltype(ic)::value;
                    const uint32_t a0 = value_pair<I>(e0, e0s), a1 = value_pair<I>(o0, o0s);
                    const uint32_t a2 = value_pair<I>(e1, e1s), a3 = value_pair<I>(o1, o1s);
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma_16816(st.o[n][4 * j + I], a0, a1, a2, a3, b[n][0], b[n][1]);
                });
            }
        }
    }
}

// Where row `row` of row group rg of (request, head h) goes: its index in
// [token][head], or -1 behind the last row.
template <int RT>
__device__ __forceinline__ int64_t row_index(const AttnParams& P, int q0, int rows, int h, int rg, int row) {
    const int i = rg * RT + row;
    if (i >= rows) return -1;
    const int qi = i / P.group;
    return (static_cast<int64_t>(q0) + qi) * P.a.heads + h * P.group + i - qi * P.group;
}

template <int D, int NT>
__global__ void __launch_bounds__(Smem<D, NT>::kThreads, 1) attn_kernel(const __grid_constant__ AttnParams P) {
    using S = Shape<D>;
    using M = Smem<D, NT>;
    constexpr int RT = 8 * NT, NG = S::kGroups, W = M::kWarps;
    extern __shared__ __align__(128) uint8_t smem[];
    const int depth = P.depth, warp_ring = depth * S::kStage;
    uint8_t* behind = smem - P.early;          // with fewer stages what follows them lies that much earlier
    const uint32_t base = smem_addr(smem), bars = base - P.early + M::kBars;
    auto full = [&](uint32_t s) { return bars + 8u * s; };
    auto empty = [&](uint32_t s) { return bars + 8u * (W * M::kDepth + s); };
    volatile uint32_t* valid = reinterpret_cast<volatile uint32_t*>(behind + M::kValid);
    volatile uint32_t* progress = reinterpret_cast<volatile uint32_t*>(behind + M::kProgress);
    volatile uint32_t* abort = reinterpret_cast<volatile uint32_t*>(behind + M::kMisc);
    volatile uint32_t* last_flag = abort + 1;                            // [2]
    uint32_t* warp_sums = reinterpret_cast<uint32_t*>(behind + M::kScan);
    uint32_t* prefix = reinterpret_cast<uint32_t*>(behind + M::kFixed);    // [batch + 1]
    const AttnArgs& a = P.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int heads = P.cache.heads;

    if (static_cast<int>(threadIdx.x) < W * depth) {
        mbar_init(full(threadIdx.x), 1);
        mbar_init(empty(threadIdx.x), 1);
        valid[threadIdx.x] = 0u;
        if (threadIdx.x < W) progress[threadIdx.x] = 0u;
        if (threadIdx.x == 0) *abort = 0u;
        fence_mbar_init();
    }
    // units before each request
    {
        const int each = (a.batch + M::kThreads - 1) / M::kThreads;
        const int b0 = min(static_cast<int>(threadIdx.x) * each, a.batch), b1 = min(b0 + each, a.batch);
        uint32_t mine = 0;
        for (int b = b0; b < b1; ++b) mine = add_units(mine, request_of<RT>(P, b).units(heads));
        uint32_t in = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, in, d);
            if (lane >= d) in = add_units(in, o);
        }
        if (lane == 31) warp_sums[warp] = in;
        __syncthreads();
        uint32_t at = in - mine;
        for (int w = 0; w < warp; ++w) at += warp_sums[w];
        for (int b = b0; b < b1; ++b) {
            prefix[b] = at;
            if (b + 1 < b1) at += request_of<RT>(P, b).units(heads);
        }
        if (threadIdx.x == M::kThreads - 1) {
            uint32_t all = 0;
            for (int w = 0; w <= W; ++w) all = add_units(all, warp_sums[w]);
            prefix[a.batch] = all_units(P, all);
        }
        __syncthreads();
    }
    const uint32_t total = prefix[a.batch];
    uint32_t blocks = min(gridDim.x, (total + W - 1) / W);
    // One request with short segments: a block to a segment, so that nothing is
    // joined over blocks (that takes longer than four tiles to a warp do).
    if (a.batch == 1 && total > 0) {
        const Request r = request_of<RT>(P, 0);
        const uint32_t segments = static_cast<uint32_t>(r.row_groups) * heads;
        if (r.tiles <= 4 * W && segments <= gridDim.x) blocks = segments;
    }
    if (blockIdx.x >= blocks) return;                                    // nothing of this block is in flight
    auto first_unit = [&](uint32_t w) {                                  // of consumer warp w of the grid
        return static_cast<uint32_t>(static_cast<uint64_t>(total) * w / (blocks * W));
    };
    auto request_at = [&](uint32_t u) {                                  // the request that holds unit u
        int lo = 0, hi = a.batch - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (prefix[mid] <= u) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    };
    // A warp's range u .. u1 - 1 from its first unit with a tile on: request,
    // head, row group and tile of u.
    auto begin = [&](uint32_t& u, uint32_t u1, Request& r, int& b, int& h, int& rg, int& idx) {
        if (u >= u1) return;
        b = request_at(u);
        r = request_of<RT>(P, b);
        locate(u - prefix[b], r, h, rg, idx);
        if (idx < 0) {
            u += static_cast<uint32_t>(-idx);
            idx = 0;
        }
    };

    if (warp == W) {
        // ------------------------------------------------------- producer --
        // A lane to each consumer warp: it copies the warp's units into its
        // stages in turn and looks up the next one's pages while it waits.
        if (lane < W) {
            const uint32_t mine = blockIdx.x * W + lane, u1 = first_unit(mine + 1), s0 = lane * depth;
            uint32_t u = first_unit(mine);
            const bool one_page = P.cache.page_size >= kTile;
            int b = 0, h = 0, rg = 0, idx = 0;
            Request r{};
            int tok0 = 0, records = 0, page[kTileRecords];
            auto look = [&]() {                // the current unit's pages
                const int tile = r.tile(idx);
                tok0 = tile * kTile;
                records = min(max((r.len - tok0 + kKvTokens - 1) / kKvTokens, 0), kTileRecords);
                const int32_t* row = a.table + static_cast<int64_t>(b) * a.table_stride;
#pragma unroll
                for (int i = 0; i < kTileRecords; ++i)
                    page[i] = i < records && (i == 0 || !one_page) ? row[(tok0 + i * kKvTokens) >> P.cache.page_shift] : -1;
            };
            begin(u, u1, r, b, h, rg, idx);
            if (u < u1) look();
            uint32_t s = 0, turn = 0;
            int64_t t0 = 0;
            bool first = true;
            for (uint32_t polls = 0; u < u1; ++polls) {
                if (turn > 0 && !mbar_try_wait(empty(s0 + s), (turn - 1) & 1u)) {
                    if (polls % 256 == 255) {
                        const int64_t now = clock64();
                        if (t0 == 0) t0 = now;
                        if (*abort || now - t0 > cycles_of(P.timeout_ns)) {
                            *abort = 1u;
                            atomicCAS(P.status, 0u, kAttnTimeout);
                            break;
                        }
                    }
                    continue;
                }
                // pages outside the cache: their tokens are not seen
                uint32_t have = 0;
#pragma unroll
                for (int i = 0; i < kTileRecords; ++i)
                    if (page[i] >= 0 && page[i] < P.cache.pages) have |= one_page ? (1u << records) - 1 : 1u << i;
                // (testing aid: with stall each warp's first bytes are announced but never
                // copied; its wait can only time out)
                const bool copied = !(P.stall && first);
                first = false;
                const uint32_t dst = base + lane * warp_ring + s * S::kStage;
                valid[s0 + s] = have | (copied ? kIssued : 0u) | ((turn & 1u) ? kOddTurn : 0u);
                mbar_arrive_expect_tx(full(s0 + s), __popc(have) * S::kRecord);
                if (copied) {
#pragma unroll
                    for (int i = 0; i < kTileRecords; ++i) {
                        if (!((have >> i) & 1) || (i > 0 && one_page)) continue;
                        const int tok = tok0 + i * kKvTokens;
                        const uint8_t* src = P.cache.record((static_cast<int64_t>(page[i]) << P.cache.page_shift) + (tok & (P.cache.page_size - 1)), h);
                        bulk_g2s(dst + i * S::kRecord, src, (one_page ? __popc(have) : 1) * S::kRecord, full(s0 + s));
                    }
                }
                if (++s == static_cast<uint32_t>(depth)) {
                    s = 0;
                    ++turn;
                }
                t0 = 0;
                ++u;
                if (++idx == r.tiles) {
                    idx = 0;
                    u += kSegmentUnits;
                    if (u < u1) next_segment<RT>(P, r, b, h, rg);
                }
                if (u < u1) look();
            }
            // the last copies into the stages land before the block ends, also after an abort
            for (int i = 0; i < depth; ++i)
                if (valid[s0 + i] & kIssued) wait_phase(full(s0 + i), valid[s0 + i] & kOddTurn ? 1u : 0u, kAttnDrainNs, nullptr);
        }
        return;
    }

    // ---------------------------------------------------------- consumers --
    const int g = lane >> 2, t = lane & 3;
    const uint32_t mine = blockIdx.x * W + warp;
    const uint32_t u1 = first_unit(mine + 1);
    // a warp's pieces: [0] of a segment that began before it, [1] of one that goes on behind it
    PieceInfo* pieces = reinterpret_cast<PieceInfo*>(behind + M::kPieceOf);
    if (lane < 2) pieces[2 * warp + lane].seg = kNone;
    __syncwarp();
    {
        float* my_pieces = reinterpret_cast<float*>(smem + warp * warp_ring);         // [2] pieces, once the stages are free
        uint32_t stage = warp * depth, parity = 0, done = 0;
        bool alive = true, waiting = false;
        int b = 0, h = 0, rg = 0, first = 0;
        Request r{};
        uint32_t u = first_unit(mine);
        begin(u, u1, r, b, h, rg, first);
        while (u < u1) {
            const int count = static_cast<int>(min(static_cast<uint32_t>(r.tiles - first), u1 - u));
            const int row0 = rg * RT;
            State<D, NT> st;
            st.clear();
            Queries<D, NT> Q;
            Q.load(P, r, h, row0);
            const int pos_lo = r.pos0 + row0 / P.group;
            const int pos_hi = r.pos0 + min(row0 + RT - 1, r.rows - 1) / P.group;
            const int window = a.window ? a.window : INT32_MAX;
            for (int k = 0; k < count; ++k) {
                if (alive) {
                    alive = __all_sync(0xFFFFFFFFu, wait_phase(full(stage), parity, P.timeout_ns, abort));
                    if (!alive && lane == 0) {
                        *abort = 1u;
                        atomicCAS(P.status, 0u, kAttnTimeout);
                    }
                }
                if (!alive) break;
                const int tok0 = r.tile(first + k) * kTile;
                const uint32_t have = valid[stage] & ((1u << kTileRecords) - 1);
                const uint8_t* data = smem + stage * S::kStage;
                if (tok0 > pos_hi) {
                    // no row sees this tile
                } else if (have == (1u << kTileRecords) - 1 && tok0 + kTile - 1 <= pos_lo && (tok0 > pos_hi - window || tok0 + kTile <= a.sinks)) {
                    take_tile<D, NT, false>(data, tok0, have, Q, window, a.sinks, st);
                } else {
                    take_tile<D, NT, true>(data, tok0, have, Q, window, a.sinks, st);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty(stage));
                if (++stage == (warp + 1) * static_cast<uint32_t>(depth)) {
                    stage = warp * depth;
                    parity ^= 1u;
                }
                // not too far ahead of the block's last warp (it goes on by itself, so this ends;
                // bounded all the same)
                if (++done % 4 == 0) {
                    if (lane == 0) progress[warp] = done;
                    for (int tries = 0; tries < 4096; ++tries) {
                        const uint32_t last = __reduce_min_sync(0xFFFFFFFFu, progress[lane < W ? lane : warp]);
                        if (done <= last + kLead || *abort) break;
                        __nanosleep(200);
                    }
                }
            }
            st.finish();
            const bool cut = first + count < r.tiles;
            if (first == 0 && !cut) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int64_t at = row_index<RT>(P, r.q0, r.rows, h, rg, 8 * n + 2 * t + c);
                        if (at < 0) continue;
                        const float inv = st.sum[n][c] == 0.0f ? 0.0f : 1.0f / st.sum[n][c];
#pragma unroll
                        for (int j = 0; j < NG; ++j) {
                            uint32_t w[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) w[i] = pack_half2(st.o[n][4 * j + i][c] * inv, st.o[n][4 * j + i][2 + c] * inv);
                            *reinterpret_cast<uint4*>(a.out + at * D + 64 * j + 8 * g) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                        if (a.lse && g == 0) a.lse[at] = log_sum(st.ref[n][c], st.sum[n][c]);
                    }
            } else {
                const int kind = first == 0 ? 1 : 0;
                // the warp's stages are free behind its last unit; an earlier piece waits in the workspace
                const bool at_end = cut || u + count + kSegmentUnits >= u1;
                float* slot = at_end ? my_pieces + kind * kPiece<D, NT> : P.warp_slots + static_cast<int64_t>(mine) * kPiece<D, NT>;
                waiting |= !at_end;
                __syncwarp();
                if (lane == 0) pieces[2 * warp + kind] = PieceInfo{u - first, r.tiles, r.q0, r.rows, h, rg};
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int row = 8 * n + 2 * t + c;
#pragma unroll
                        for (int j = 0; j < NG; ++j) {
                            float4* to = reinterpret_cast<float4*>(slot + row * D + 64 * j + 8 * g);
                            to[0] = make_float4(st.o[n][4 * j][c], st.o[n][4 * j][2 + c], st.o[n][4 * j + 1][c], st.o[n][4 * j + 1][2 + c]);
                            to[1] = make_float4(st.o[n][4 * j + 2][c], st.o[n][4 * j + 2][2 + c], st.o[n][4 * j + 3][c], st.o[n][4 * j + 3][2 + c]);
                        }
                        if (g == 0) reinterpret_cast<float2*>(slot + RT * D)[row] = make_float2(st.ref[n][c], st.sum[n][c]);
                    }
            }
            u += count;
            first = 0;
            if (!cut) {
                u += kSegmentUnits;
                if (u < u1) next_segment<RT>(P, r, b, h, rg);
            }
        }
        if (lane == 0) progress[warp] = kNone;
        if (waiting && alive) {                        // (after an abort copies may still be on their way into the stages)
            __syncwarp();                              // the warp's own writes
            const float4* from = reinterpret_cast<const float4*>(P.warp_slots + static_cast<int64_t>(mine) * kPiece<D, NT>);
#pragma unroll 8
            for (int i = lane; i < kPiece<D, NT> / 4; i += 32) reinterpret_cast<float4*>(my_pieces)[i] = from[i];
        }
    }

    // -------------------------------------------------- the block's join --
    // Its pieces in unit order form runs of one segment each.
    consumers_sync<W>();
    uint32_t* order = reinterpret_cast<uint32_t*>(behind + M::kRuns);      // [pieces] piece numbers
    uint32_t* run_at = order + M::kPieces;                               // [runs + 1] first piece of a run, then the number of runs
    float* factors = reinterpret_cast<float*>(behind + M::kFactors);       // [pieces][rows]
    if (warp == 0) {
        const uint32_t seg = lane < M::kPieces ? pieces[lane].seg : kNone, lower = (1u << lane) - 1u;
        const uint32_t have = __ballot_sync(0xFFFFFFFFu, seg != kNone);
        const uint32_t before = __shfl_sync(0xFFFFFFFFu, seg, have & lower ? 31 - __clz(have & lower) : lane);
        const bool starts = seg != kNone && (!(have & lower) || before != seg);
        const uint32_t start = __ballot_sync(0xFFFFFFFFu, starts);
        if (seg != kNone) order[__popc(have & lower)] = lane;
        if (starts) run_at[__popc(start & lower)] = __popc(have & lower);
        if (lane == 0) {
            run_at[__popc(start)] = __popc(have);
            run_at[M::kRunsMost + 1] = __popc(start);
        }
    }
    consumers_sync<W>();
    const int runs = static_cast<int>(run_at[M::kRunsMost + 1]);
    if (runs == 0) return;
    // a segment is the block's alone if all its tiles are
    const uint32_t b_u0 = first_unit(blockIdx.x * W), b_u1 = first_unit((blockIdx.x + 1) * W);
    auto inside = [&](const PieceInfo& i) { return i.seg >= b_u0 && i.seg + i.tiles <= b_u1; };
    auto piece_at = [&](int i) {                       // i-th piece of the block
        return reinterpret_cast<const float*>(smem + (order[i] >> 1) * warp_ring) + (order[i] & 1) * kPiece<D, NT>;
    };
    auto block_slot = [&](uint32_t c, bool begins) { return P.block_slots + (2 * static_cast<int64_t>(c) + begins) * kPiece<D, NT>; };
    // A run's row: common reference and sum; each piece's factor to them, for
    // whole segments to the output; the others' (reference, sum) goes to the
    // block's slot.
    int64_t* row_out = reinterpret_cast<int64_t*>(behind + M::kRowOut);    // [runs][rows]: output row, kToNone, kToSlot + begins
    constexpr int64_t kToNone = -1, kToSlot = -3;
    // Four lanes to a row, each with every fourth piece: a run has one of each warp at most.
    static_assert(W <= 16, "pieces of a run");
    for (int i = threadIdx.x / 4; i < runs * RT; i += W * 8) {
        const int run = i / RT, row = i % RT, p0 = run_at[run] + lane % 4, p1 = run_at[run + 1];
        const PieceInfo info = pieces[order[run_at[run]]];
        float2 v[4];
        float m = -INFINITY, l = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[k] = p0 + 4 * k < p1 ? reinterpret_cast<const float2*>(piece_at(p0 + 4 * k) + RT * D)[row] : make_float2(-INFINITY, 0.0f);
            m = fmaxf(m, v[k].x);
        }
        const uint32_t four = 0xFu << (lane & 28);
        m = fmaxf(m, __shfl_xor_sync(four, m, 1));
        m = fmaxf(m, __shfl_xor_sync(four, m, 2));
        float f[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            f[k] = v[k].x == -INFINITY ? 0.0f : ex2(v[k].x - m);
            l += f[k] * v[k].y;
        }
        l += __shfl_xor_sync(four, l, 1);
        l += __shfl_xor_sync(four, l, 2);
        const bool whole = inside(info);
        const float inv = !whole ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (p0 + 4 * k < p1) factors[(p0 + 4 * k) * RT + row] = f[k] * inv;
        if (lane % 4) continue;
        if (whole) {
            const int64_t at = row_index<RT>(P, info.q0, info.rows, info.h, info.rg, row);
            if (a.lse && at >= 0) a.lse[at] = log_sum(m, l);
            row_out[i] = at >= 0 ? at : kToNone;
        } else {
            const bool begins = info.seg >= b_u0;
            reinterpret_cast<float2*>(block_slot(blockIdx.x, begins) + RT * D)[row] = make_float2(m, l);
            row_out[i] = kToSlot + begins;
        }
    }
    consumers_sync<W>();
    for (int i = threadIdx.x; i < runs * (RT * D / 4); i += W * 32) {
        const int run = i / (RT * D / 4), e = (i % (RT * D / 4)) * 4, row = e / D, d = e % D;
        const int64_t at = row_out[run * RT + row];
        if (at == kToNone) continue;
        const int p0 = run_at[run], p1 = run_at[run + 1];
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int p = p0; p < p1; ++p) {
            const float f = factors[p * RT + row];
            const float4 v = *reinterpret_cast<const float4*>(piece_at(p) + e);
            o.x = fmaf(f, v.x, o.x); o.y = fmaf(f, v.y, o.y); o.z = fmaf(f, v.z, o.z); o.w = fmaf(f, v.w, o.w);
        }
        if (at >= 0) *reinterpret_cast<uint2*>(a.out + at * D + d) = make_uint2(pack_half2(o.x, o.y), pack_half2(o.z, o.w));
        else *reinterpret_cast<float4*>(block_slot(blockIdx.x, at != kToSlot) + e) = o;
    }

    // ------------------------------------------- segments of several blocks --
    // The first and the last run may be pieces of such; the last block to
    // arrive joins them, in block order.
    const PieceInfo side_of[2] = {pieces[order[0]], pieces[order[run_at[runs] - 1]]};
    const bool shared[2] = {!inside(side_of[0]), side_of[1].seg != side_of[0].seg && !inside(side_of[1])};
    if (!shared[0] && !shared[1]) return;              // the same for every thread
    auto block_of = [&](uint32_t x) {                  // the block that holds unit x
        return static_cast<uint32_t>(((static_cast<uint64_t>(x) + 1) * blocks + total - 1) / total - 1);
    };
    consumers_sync<W>();                               // the block's slots are written, the pieces read
    if (threadIdx.x < 2) {
        const PieceInfo& info = side_of[threadIdx.x];
        bool last = false;
        if (shared[threadIdx.x]) {
            const uint32_t c0 = block_of(info.seg), c1 = block_of(info.seg + info.tiles - 1);
            uint32_t old;
            asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(old) : "l"(P.counters + c0) : "memory");
            last = old == c1 - c0;
            if (last) P.counters[c0] = 0u;
        }
        last_flag[threadIdx.x] = last;
    }
    consumers_sync<W>();
    // Nothing is in flight into the ring and no piece is read any more: it holds
    // the parts' references and sums, their factors, and each warp's sum of every
    // W-th part.
    float2* part_sums = reinterpret_cast<float2*>(smem);                 // [parts][rows]; the grid's fit (see launch)
    for (int side = 0; side < 2; ++side) {
        if (!last_flag[side]) continue;
        const PieceInfo info = side_of[side];
        const uint32_t c0 = block_of(info.seg), c1 = block_of(info.seg + info.tiles - 1);
        const int parts = static_cast<int>(c1 - c0 + 1);
        float* part_factors = reinterpret_cast<float*>(part_sums + parts * RT);      // [parts][rows]
        float4* share = reinterpret_cast<float4*>(smem + (parts * RT * 12 + 15) / 16 * 16);   // [warps][RT * D / 4]
        for (int i = threadIdx.x; i < parts * RT; i += W * 32) {
            const int p = i / RT, row = i % RT;
            part_sums[i] = __ldcg(reinterpret_cast<const float2*>(block_slot(c0 + p, p == 0) + RT * D) + row);
        }
        consumers_sync<W>();
        for (int row = warp; row < RT; row += W) {
            float m = -INFINITY, l = 0.0f;
            for (int p = lane; p < parts; p += 32) m = fmaxf(m, part_sums[p * RT + row].x);
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
            for (int p = lane; p < parts; p += 32) {
                const float2 v = part_sums[p * RT + row];
                l += v.x == -INFINITY ? 0.0f : ex2(v.x - m) * v.y;
            }
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            for (int p = lane; p < parts; p += 32) {
                const float ref = part_sums[p * RT + row].x;
                part_factors[p * RT + row] = ref == -INFINITY ? 0.0f : ex2(ref - m) * inv;
            }
            const int64_t at = row_index<RT>(P, info.q0, info.rows, info.h, info.rg, row);
            if (a.lse && at >= 0 && lane == 0) a.lse[at] = log_sum(m, l);
        }
        consumers_sync<W>();
        constexpr int kEach = RT * D / 128;            // fours of a lane
        float4 o[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) o[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int p = warp; p < parts; p += W) {
            const float4* from = reinterpret_cast<const float4*>(block_slot(c0 + p, p == 0));
            float4 v[kEach];
#pragma unroll
            for (int k = 0; k < kEach; ++k) v[k] = __ldcg(from + lane + 32 * k);
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                const float f = part_factors[p * RT + (lane + 32 * k) * 4 / D];
                o[k].x = fmaf(f, v[k].x, o[k].x); o[k].y = fmaf(f, v[k].y, o[k].y);
                o[k].z = fmaf(f, v[k].z, o[k].z); o[k].w = fmaf(f, v[k].w, o[k].w);
            }
        }
#pragma unroll
        for (int k = 0; k < kEach; ++k) share[warp * (RT * D / 4) + lane + 32 * k] = o[k];
        consumers_sync<W>();
        for (int i = threadIdx.x; i < RT * D / 4; i += W * 32) {
            const int row = i * 4 / D, d = i * 4 % D;
            const int64_t at = row_index<RT>(P, info.q0, info.rows, info.h, info.rg, row);
            if (at < 0) continue;
            float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int w = 0; w < min(W, parts); ++w) {
                const float4 v = share[w * (RT * D / 4) + i];
                s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
            }
            *reinterpret_cast<uint2*>(a.out + at * D + d) = make_uint2(pack_half2(s.x, s.y), pack_half2(s.z, s.w));
        }
        consumers_sync<W>();                           // the ring is written again
    }
}

// Workspace: status word (256 bytes), one counter and two slots per thread
// block, one slot per consumer warp.
template <int D, int NT>
size_t workspace_bytes(int num_sms) {
    return 256 + attn_counter_bytes(num_sms) + static_cast<size_t>(num_sms) * (2 + Smem<D, NT>::kWarps) * kPiece<D, NT> * 4;
}

template <int D, int NT>
cudaError_t launch(AttnParams P, uint8_t* ws, int num_sms, cudaStream_t s) {
    using M = Smem<D, NT>;
    constexpr int kLimit = 227 * 1024;
    static std::atomic<uint64_t> smem_set{0};
    if (cudaError_t e = set_smem_limit_once(attn_kernel<D, NT>, kLimit, smem_set); e != cudaSuccess) return e;
    const int smem = M::bytes(P.a.batch);
    // a very large batch's prefix sums take the place of a stage per warp
    P.depth = M::kDepth;
    int shift = 0;
    while (smem - shift > kLimit && P.depth > 2) {
        --P.depth;
        shift += M::kWarps * Shape<D>::kStage;
    }
    P.early = shift;
    if (smem - shift > kLimit || 2 * kPiece<D, NT> * 4 > P.depth * Shape<D>::kStage) return cudaErrorInvalidValue;
    // the last block to join keeps the parts' references, sums and factors and its warps' shares in the ring
    int grid = num_sms;
    const int room = M::kWarps * P.depth * Shape<D>::kStage - M::kWarps * M::kRT * D * 4 - 16;
    if (grid > room / (M::kRT * 12)) grid = room / (M::kRT * 12);
    P.status = reinterpret_cast<uint32_t*>(ws);
    P.counters = reinterpret_cast<uint32_t*>(ws + 256);
    P.block_slots = reinterpret_cast<float*>(ws + 256 + attn_counter_bytes(num_sms));
    P.warp_slots = P.block_slots + 2 * static_cast<size_t>(grid) * kPiece<D, NT>;
    attn_kernel<D, NT><<<grid, M::kThreads, smem - shift, s>>>(P);
    return cudaGetLastError();
}

}  // namespace

size_t attn_workspace_bytes(int num_sms) {
    size_t most = 0;
    for (size_t n : {workspace_bytes<64, 1>(num_sms), workspace_bytes<64, 2>(num_sms), workspace_bytes<128, 1>(num_sms),
                     workspace_bytes<128, 2>(num_sms), workspace_bytes<256, 1>(num_sms), attn_tc_workspace_bytes(num_sms)})
        most = n > most ? n : most;
    return most;
}

// Two limits.  Row groups as the arguments alone allow for them, every request
// with max_queries queries, below 2^31, whichever kernel runs.  And the chosen
// kernel's units below 2^32 - 1, where the requests' queries together are no more
// than `tokens`: n queries are at most n / per + 1 row groups (tiles), so a long
// prompt beside many single tokens counts as what it is.  (With max_queries for
// every request there too, 64 requests with one chunk of 8192 queries of 64 + 8
// heads and tables for 131072 tokens would not fit, by a factor of 2.)
bool attn_fits(const AttnArgs& a, const KvGeometry& g) {
    const int group = a.heads / g.heads;
    const int64_t rows = static_cast<int64_t>(a.max_queries) * group, per = g.D < 256 && rows > 8 ? 16 : 8;
    const double batch = a.batch, allowed = batch * static_cast<double>((rows + per - 1) / per);
    if (allowed * g.heads >= 2147483648.0) return false;
    if (attn_tc_takes(a, g)) return attn_tc_units(a, g) < 4294967295.0;
    const double there = static_cast<double>(a.tokens) * group / static_cast<double>(per) + batch;
    const int64_t tiles = (static_cast<int64_t>(a.max_pages) * g.page_size + kTile - 1) / kTile + kSegmentUnits;
    return (allowed < there ? allowed : there) * g.heads * static_cast<double>(tiles) < 4294967295.0;
}

cudaError_t launch_attention(const AttnArgs& a, const KvGeometry& g, void* workspace, int num_sms, uint64_t timeout_ns, int stall,
                             cudaStream_t s) {
    int shift = 0;
    while ((1 << shift) < g.page_size) ++shift;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    AttnParams P{a, KvCache{g.data, g.pages, g.page_size, shift, g.heads, g.D}, a.heads / g.heads, a.scale * 1.4426950408889634f,
                 nullptr, nullptr, nullptr, nullptr, timeout_ns, stall};
    if (attn_tc_takes(a, g)) return launch_attention_tc(P, ws, num_sms, s);
    // 8 or 16 query rows share the decoded codes
    const bool wide = static_cast<int64_t>(a.max_queries) * P.group > 8;
    if (g.D == 64) return wide ? launch<64, 2>(P, ws, num_sms, s) : launch<64, 1>(P, ws, num_sms, s);
    if (g.D == 128) return wide ? launch<128, 2>(P, ws, num_sms, s) : launch<128, 1>(P, ws, num_sms, s);
    return launch<256, 1>(P, ws, num_sms, s);
}

}  // namespace pn
