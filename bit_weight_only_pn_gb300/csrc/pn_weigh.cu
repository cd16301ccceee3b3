// pn_weigh.cu -- the attention weight that cached tokens gather.
//
// For a cached token t of a request and a key/value head: the sum, over the step's
// queries and the query heads that share the head and see t, of exp(scale q . k_t -
// lse), with each row's lse as attention gave it, and decay times what t had before
// (nothing, for the step's own tokens).
//
// Only K is read.  The products run on mma.sync, 16 tokens x 8 query rows, with the
// codes as fp16 whole numbers n - 8 and the queries as they are, so every product is
// exact; each group's sum is multiplied by its scale in fp32.  There is no softmax
// state, so tokens do not wait for each other: a warp has 32 of them, whose codes
// stay in registers while the query rows go by, and each lane sums what its columns
// give.  A token's sum is made by one warp in a fixed order; nothing is joined and
// no result depends on timing.
//
// Three kernels, by the rows (queries of a request, at most, times heads that share a
// key/value head): here that for few of them, and the one for more heads to a key/value
// head than the tensor memory's kernel (pn_weigh_tc.cu) has columns for.
#include <atomic>
#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "pn_weigh.cuh"

namespace pn {
namespace {

using Params = WeighParams;
using Request = WeighRequest;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 32;                      // tokens of a warp
constexpr int kUnit = kWarps * kTile;          // tokens of a block's unit of work
constexpr int kChunk = 8 * kWarps;             // query rows made ready at a time, 8 by a warp

// Code pair I of a word as fp16 whole numbers n - 8.  (Not as subnormals, which attention
// takes as they are: the tensor cores align sums by the operands' exponents, and
// products of subnormals lie some bits below theirs.  Attention's outputs are rounded
// to fp16 and do not show it; weights are not, and erred by 1e-6 instead of 2e-7.)
template <int I>
__device__ __forceinline__ uint32_t codes(uint32_t word, uint32_t shifted) { return decode_pair<kPn4t, I>(word, shifted); }

// Row g of eight as the lane's part of the products' B fragments.
template <int D>
__device__ __forceinline__ void load_fragments(const __half* src, uint4 (&q)[D / 64][2]) {
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int j = 0; j < D / 64; ++j)
#pragma unroll
        for (int w = 0; w < 2; ++w) q[j][w] = *reinterpret_cast<const uint4*>(src + 64 * j + 16 * t + 8 * w);
}

// Queries of a row that gives nothing become zeros: whatever they are, its products are finite, and nothing times its share.
template <int NG>
__device__ __forceinline__ void drop_fragments(uint4 (&q)[NG][2]) {
#pragma unroll
    for (int j = 0; j < NG; ++j) q[j][0] = q[j][1] = make_uint4(0, 0, 0, 0);
}

// The sums of tokens 8 (2 i + hh) + g over a warp's columns, and what the tokens had
// before (of lane (g, t): token 8 t + g), to the weights of a tile whose records are at
// slots `place` (-1: nowhere).
__device__ __forceinline__ void write_sums(const Params& P, const float (&sum)[2][2], const int64_t (&place)[2], int h, int tok0, int len, float before) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float all = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float s = sum[i >> 1][i & 1];
        s += __shfl_xor_sync(0xFFFFFFFFu, s, 1);
        s += __shfl_xor_sync(0xFFFFFFFFu, s, 2);
        if (t == i) all = s;
    }
    const int64_t mine = t < 2 ? place[0] : place[1];
    if (mine >= 0 && tok0 + 8 * t + g < len)
        P.a.out[(((mine >> P.cache.page_shift) * P.cache.heads + h) << P.cache.page_shift) + (mine & (P.cache.page_size - 1)) + ((8 * t + g) & 15)] = before + all;
}

// Eight query rows ready for the products: B fragments by lane, and for each row its
// LogSum (-inf: a row that gives nothing) and its position.
template <int D>
struct Rows {
    uint4 q[D / 64][2][32];
    float less[8], share[8];
    int pos[8];
};

template <int D>
__device__ __forceinline__ void make_ready(const Params& P, const Request& r, int h, int row0, Rows<D>& to) {
    constexpr int NG = D / 64;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int row = min(row0 + g, r.rows - 1), qi = row / P.group, head = h * P.group + row - qi * P.group;
    uint4 q[NG][2];
    load_fragments<D>(P.a.q + (r.q0 + qi) * P.a.q_stride + head * D, q);
    const bool real = row0 + g < r.rows;
    const LogSum l = log_sum_of(real ? P.a.lse[static_cast<int64_t>(r.q0 + qi) * P.a.heads + head] : -INFINITY, P.scale_rest);
    if (l.less == -INFINITY) drop_fragments(q);
#pragma unroll
    for (int j = 0; j < NG; ++j) {
        to.q[j][0][lane] = q[j][0];
        to.q[j][1][lane] = q[j][1];
    }
    if (t == 0) {
        to.less[g] = l.less;
        to.share[g] = l.factor;
        to.pos[g] = r.pos0 + qi;
    }
}

// A warp's tokens: codes of K (words of tokens g and g + 8 of each record) and scales.
template <int D>
struct Keys {
    static constexpr int kWords = D / 64 * 2;  // of a token, to a lane
    uint32_t w[2][2][kWords];
    float d[2][2][D / 64];
};

template <int D>
__device__ __forceinline__ void load_keys(const uint8_t* const (&record)[2], Keys<D>& k) {
    constexpr int NG = D / 64, GP = kv_plane_groups(D), PL = kv_planes(D);
    const int lane = threadIdx.x & 31, g = lane >> 2;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
#pragma unroll
            for (int i = 0; i < Keys<D>::kWords; ++i) k.w[r][hh][i] = 0;
#pragma unroll
            for (int j = 0; j < NG; ++j) k.d[r][hh][j] = 0.0f;
            if (!record[r]) continue;
#pragma unroll
            for (int pl = 0; pl < PL; ++pl) {
                const uint8_t* p = record[r] + ((hh * PL + pl) * 32 + lane) * 8 * GP;
                if constexpr (GP == 2) {
                    const uint4 v = *reinterpret_cast<const uint4*>(p);
                    k.w[r][hh][4 * pl] = v.x; k.w[r][hh][4 * pl + 1] = v.y; k.w[r][hh][4 * pl + 2] = v.z; k.w[r][hh][4 * pl + 3] = v.w;
                } else {
                    const uint2 v = *reinterpret_cast<const uint2*>(p);
                    k.w[r][hh][0] = v.x; k.w[r][hh][1] = v.y;
                }
            }
            const __half* d = reinterpret_cast<const __half*>(record[r] + kv_k_scales(D)) + (g + 8 * hh) * NG;
#pragma unroll
            for (int j = 0; j < NG; ++j) k.d[r][hh][j] = __half2float(d[j]);
        }
}

// The products of the warp's 32 tokens with NT times eight rows, by group scaled and summed.
template <int D, int NT>
__device__ __forceinline__ void products(const Keys<D>& k, const Rows<D>* rows, float (&x)[2][NT][4]) {
    constexpr int NG = D / 64;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < NG; ++j) {
        float acc[2][NT][4];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            uint4 b[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) b[n] = rows[n].q[j][w][lane];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                // word 2t + w of group j of tokens g (a) and g + 8 (c)
                const uint32_t a = k.w[r][0][2 * j + w], c = k.w[r][1][2 * j + w], as = a >> 8, cs = c >> 8;
                const uint32_t a0 = codes<0>(a, as), a1 = codes<0>(c, cs), a2 = codes<1>(a, as), a3 = codes<1>(c, cs);
                const uint32_t b0 = codes<2>(a, as), b1 = codes<2>(c, cs), b2 = codes<3>(a, as), b3 = codes<3>(c, cs);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (w == 0) mma_from(acc[r][n], a0, a1, a2, a3, b[n].x, b[n].y, 0.0f, 0.0f, 0.0f, 0.0f);
                    else mma_16816(acc[r][n], a0, a1, a2, a3, b[n].x, b[n].y);
                    mma_16816(acc[r][n], b0, b1, b2, b3, b[n].z, b[n].w);
                }
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[r][n][i] = j ? fmaf(k.d[r][i >> 1][j], acc[r][n][i], x[r][n][i]) : k.d[r][i >> 1][j] * acc[r][n][i];
    }
}

// More query heads to a key/value head than the kernel for many rows has columns for: a
// block shares its rows among 256 tokens.  64 ragged requests to 16384 tokens, one query each:
// 132 heads of 128 to one 115 us (128 heads, in that kernel: 62), 264 of 64 to two 169.
template <int D>
__global__ void __launch_bounds__(kThreads, 2) weigh_kernel(const __grid_constant__ Params P) {
    constexpr int NT = D == 256 ? 1 : 2;       // row groups at a time, as registers allow
    __shared__ Rows<D> ready[kWarps];
    __shared__ uint64_t scan[kThreads + 1];
    __shared__ uint64_t warp_sums[kWarps];
    const WeighArgs& a = P.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int heads = P.cache.heads, window = a.window ? a.window : INT32_MAX;
    const int each = scan_units<kUnit, kThreads>(P, scan, warp_sums);
    const uint64_t total = scan[kThreads];
    for (uint64_t u = blockIdx.x; u < total; u += gridDim.x) {
        Request r;
        int b, h, unit;
        locate<kUnit, kThreads>(P, scan, each, u, r, b, h, unit);
        const int first = unit * kUnit, tok0 = first + warp * kTile;
        const uint8_t* record[2];
        int64_t place[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int tok = tok0 + i * kKvTokens;
            record[i] = nullptr;
            place[i] = -1;
            if (tok >= r.len) continue;
            const int page = a.table[b * a.table_stride + (tok >> P.cache.page_shift)];
            if (page < 0 || page >= P.cache.pages) continue;
            place[i] = (static_cast<int64_t>(page) << P.cache.page_shift) + (tok & (P.cache.page_size - 1));
            record[i] = P.cache.record(place[i], h);
        }
        Keys<D> keys;
        load_keys<D>(record, keys);
        const int64_t mine = t < 2 ? place[0] : place[1];      // of lane (g, t)'s token, 8 t + g
        float before = 0.0f;
        if (a.weights && mine >= 0 && tok0 + 8 * t + g < r.pos0)
            before = a.decay * a.weights[(((mine >> P.cache.page_shift) * heads + h) << P.cache.page_shift) + (mine & (P.cache.page_size - 1)) + ((8 * t + g) & 15)];
        float sum[2][2] = {};
        // the queries that see any of the unit's tokens
        const int last = min(first + kUnit, r.len) - 1;
        const int i0 = max(first - r.pos0, 0);
        int i1 = r.n;
        if (a.window && first >= a.sinks) i1 = static_cast<int>(min(static_cast<int64_t>(i1), max(static_cast<int64_t>(last) + window - r.pos0, static_cast<int64_t>(0))));
        const int row_end = i1 * P.group;
        for (int row0 = i0 * P.group / 8 * 8; row0 < row_end; row0 += kChunk) {
            __syncthreads();                   // the rows before have been read
            if (row0 + 8 * warp < row_end) make_ready<D>(P, r, h, row0 + 8 * warp, ready[warp]);
            __syncthreads();
            const int groups = min((row_end - row0 + 7) / 8, kWarps);
            for (int n0 = 0; n0 < groups; n0 += NT) {
                const int from = row0 + 8 * n0, upto = min(from + 8 * min(NT, groups - n0), r.rows) - 1;
                const int pos_lo = r.pos0 + from / P.group, pos_hi = r.pos0 + upto / P.group;
                if (tok0 > pos_hi) continue;
                float x[2][NT][4];
                products<D, NT>(keys, ready + n0, x);
                const bool plain = n0 + NT <= groups && record[0] && record[1] && tok0 + kTile - 1 <= pos_lo && (tok0 > pos_hi - window || tok0 + kTile <= a.sinks);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (n0 + n >= groups) break;
                    const Rows<D>& rows = ready[n0 + n];
                    const float2 l = *reinterpret_cast<const float2*>(rows.less + 2 * t),
                                 e = *reinterpret_cast<const float2*>(rows.share + 2 * t);
                    const int2 pos = *reinterpret_cast<const int2*>(rows.pos + 2 * t);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {
                            float p0 = ex2(fmaf(x[i][n][2 * hh], P.scale_log2, l.x)), p1 = ex2(fmaf(x[i][n][2 * hh + 1], P.scale_log2, l.y));
                            if (!plain) {
                                const int k = tok0 + i * kKvTokens + hh * 8 + g;
                                p0 = k <= pos.x && (k > pos.x - window || k < a.sinks) ? p0 : 0.0f;
                                p1 = k <= pos.y && (k > pos.y - window || k < a.sinks) ? p1 : 0.0f;
                            }
                            sum[i][hh] = fmaf(p1, e.y, fmaf(p0, e.x, sum[i][hh]));
                        }
                }
            }
        }
        write_sums(P, sum, place, h, tok0, r.len, before);
    }
}

// ---------------------------------------------------- few rows to a head --
//
// Every warp takes a contiguous range of the call's tiles (request, head, 32 tokens) and
// works alone: the next tile's codes, scales and weights are on their way while it
// multiplies, and the pages of the one behind that are being looked up.  The rows of the
// request and head are ready in the warp's registers, up to 8 (heads of 64: 16), or in its
// own part of shared memory, where 8 NT of them at a time meet the tile's codes.
//
// 64 ragged requests to 16384 tokens, 32 + 8 heads of 128, one query each: 71 us, 4.5 TB/s
// of what it has to read and write.  Bound by memory and the instructions for it: with a
// tile's registers copied, masks worked out for every tile and places in 64 bits
// throughout, a tile took 600 instructions and the call 101 us.  With 5 queries
// each (20 rows) it takes 120 us, with 11 (44) 201, where blocks that share rows and wait
// for each other took 291 and 368: those waited, these are bound by instructions.  Heads of
// 64: 64 us (the forms for 8 rows spill, 80 bytes), of 256: 148 (84 bytes), with 5 queries 92, 348.

template <int D>
struct Tile {
    uint32_t w[2][2][D / 32];                  // as Keys
    uint32_t d[2][2][(D / 64 + 1) / 2];        // scales, two to a word
    float before;
};

// The pages of a tile's two records, -1 for none, and where a head's keys and weights
// of page 0 begin, from where others are so many bytes (entries) on.
struct Place {
    int page[2];
};
struct HeadBase {
    const uint8_t* keys;
    const float* weights;
    float* out;
    int64_t page_bytes, page_entries;
};

template <int D, int NT>
struct FewRows {
    uint4 q[NT][D / 64][2];
    float less[NT][2], share[NT][2];
    int pos[NT][2];
};

template <int D>
__device__ __forceinline__ void load_tile(const HeadBase& base, const Place& place, int tok0, int in_page, bool kept, Tile<D>& k) {
    constexpr int NG = D / 64, GP = kv_plane_groups(D), PL = kv_planes(D);
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        // (of a page that is none the first one is read, and not used)
        const uint8_t* record = base.keys + max(place.page[r], 0) * base.page_bytes + (((tok0 + r * kKvTokens) & in_page) >> 4) * kv_record_bytes(D);
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
#pragma unroll
            for (int pl = 0; pl < PL; ++pl) {
                const uint8_t* p = record + ((hh * PL + pl) * 32 + lane) * 8 * GP;
                if constexpr (GP == 2) {
                    const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p));
                    k.w[r][hh][4 * pl] = v.x; k.w[r][hh][4 * pl + 1] = v.y; k.w[r][hh][4 * pl + 2] = v.z; k.w[r][hh][4 * pl + 3] = v.w;
                } else {
                    const uint2 v = __ldcs(reinterpret_cast<const uint2*>(p));
                    k.w[r][hh][0] = v.x; k.w[r][hh][1] = v.y;
                }
            }
            const uint8_t* d = record + kv_k_scales(D) + (g + 8 * hh) * NG * 2;
            if constexpr (NG == 1) k.d[r][hh][0] = *reinterpret_cast<const uint16_t*>(d);
            if constexpr (NG == 2) k.d[r][hh][0] = *reinterpret_cast<const uint32_t*>(d);
            if constexpr (NG == 4) {
                const uint2 v = *reinterpret_cast<const uint2*>(d);
                k.d[r][hh][0] = v.x; k.d[r][hh][1] = v.y;
            }
        }
    }
    // lane (g, t) has token 8 t + g
    const int mine = t < 2 ? place.page[0] : place.page[1];
    k.before = 0.0f;
    if (kept && mine >= 0) k.before = base.weights[mine * base.page_entries + ((tok0 + 8 * t + g) & in_page)];
}

template <int D, int NT, bool kMasked>
__device__ __forceinline__ void tile_sums(const Tile<D>& k, const FewRows<D, NT>& R, float scale, int tok0, int window, int sinks, float (&sum)[4]) {
    constexpr int NG = D / 64;
    const int g = (threadIdx.x & 31) >> 2;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float x[NT][4];
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            float acc[NT][4];
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const uint32_t a = k.w[i][0][2 * j + v], c = k.w[i][1][2 * j + v], as = a >> 8, cs = c >> 8;
                const uint32_t a0 = codes<0>(a, as), a1 = codes<0>(c, cs), a2 = codes<1>(a, as), a3 = codes<1>(c, cs);
                const uint32_t b0 = codes<2>(a, as), b1 = codes<2>(c, cs), b2 = codes<3>(a, as), b3 = codes<3>(c, cs);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (v == 0) mma_from(acc[n], a0, a1, a2, a3, R.q[n][j][v].x, R.q[n][j][v].y, 0.0f, 0.0f, 0.0f, 0.0f);
                    else mma_16816(acc[n], a0, a1, a2, a3, R.q[n][j][v].x, R.q[n][j][v].y);
                    mma_16816(acc[n], b0, b1, b2, b3, R.q[n][j][v].z, R.q[n][j][v].w);
                }
            }
            const float d0 = half_bits_to_float(j & 1 ? k.d[i][0][j / 2] >> 16 : k.d[i][0][j / 2] & 0xFFFFu);
            const float d1 = half_bits_to_float(j & 1 ? k.d[i][1][j / 2] >> 16 : k.d[i][1][j / 2] & 0xFFFFu);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[n][e] = j ? fmaf(e < 2 ? d0 : d1, acc[n][e], x[n][e]) : (e < 2 ? d0 : d1) * acc[n][e];
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float p = ex2(fmaf(x[n][e], scale, R.less[n][e & 1]));
                if constexpr (kMasked) {
                    const int tok = tok0 + i * kKvTokens + (e >> 1) * 8 + g;
                    p = tok <= R.pos[n][e & 1] && (tok > R.pos[n][e & 1] - window || tok < sinks) ? p : 0.0f;
                }
                sum[2 * i + (e >> 1)] = fmaf(p, R.share[n][e & 1], sum[2 * i + (e >> 1)]);
            }
    }
}

// The same with rows in shared memory, which are read once for both records.
template <int D, int NT, bool kMasked>
__device__ __forceinline__ void tile_sums(const Tile<D>& k, const Rows<D>* rows, float scale, int tok0, int window, int sinks, float (&sum)[4]) {
    constexpr int NG = D / 64;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float x[2][NT][4];
#pragma unroll
    for (int j = 0; j < NG; ++j) {
        float acc[2][NT][4];
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            uint4 b[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) b[n] = rows[n].q[j][v][lane];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t a = k.w[i][0][2 * j + v], c = k.w[i][1][2 * j + v], as = a >> 8, cs = c >> 8;
                const uint32_t a0 = codes<0>(a, as), a1 = codes<0>(c, cs), a2 = codes<1>(a, as), a3 = codes<1>(c, cs);
                const uint32_t b0 = codes<2>(a, as), b1 = codes<2>(c, cs), b2 = codes<3>(a, as), b3 = codes<3>(c, cs);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (v == 0) mma_from(acc[i][n], a0, a1, a2, a3, b[n].x, b[n].y, 0.0f, 0.0f, 0.0f, 0.0f);
                    else mma_16816(acc[i][n], a0, a1, a2, a3, b[n].x, b[n].y);
                    mma_16816(acc[i][n], b0, b1, b2, b3, b[n].z, b[n].w);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float d0 = half_bits_to_float(j & 1 ? k.d[i][0][j / 2] >> 16 : k.d[i][0][j / 2] & 0xFFFFu);
            const float d1 = half_bits_to_float(j & 1 ? k.d[i][1][j / 2] >> 16 : k.d[i][1][j / 2] & 0xFFFFu);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[i][n][e] = j ? fmaf(e < 2 ? d0 : d1, acc[i][n][e], x[i][n][e]) : (e < 2 ? d0 : d1) * acc[i][n][e];
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const float2 less = *reinterpret_cast<const float2*>(rows[n].less + 2 * t), share = *reinterpret_cast<const float2*>(rows[n].share + 2 * t);
        int2 pos{};
        if constexpr (kMasked) pos = *reinterpret_cast<const int2*>(rows[n].pos + 2 * t);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float p = ex2(fmaf(x[i][n][e], scale, e & 1 ? less.y : less.x));
                if constexpr (kMasked) {
                    const int tok = tok0 + i * kKvTokens + (e >> 1) * 8 + g, at = e & 1 ? pos.y : pos.x;
                    p = tok <= at && (tok > at - window || tok < sinks) ? p : 0.0f;
                }
                sum[2 * i + (e >> 1)] = fmaf(p, e & 1 ? share.y : share.x, sum[2 * i + (e >> 1)]);
            }
    }
}

// Threads of a block and blocks to an SM: registers for a tile, the next one and the rows.
// (16 rows of 128 in registers spilled: 61 us for 64 ragged requests and 4 heads, 50 from
// shared memory; of 64, 33 and 39)
template <int D, int NT>
constexpr bool kFewShared = NT > (D == 64 ? 2 : 1);
template <int D, int NT>
constexpr int kFewThreads = D == 256 || kFewShared<D, NT> ? 384 : 256;
template <int D, int NT>
constexpr int kFewBlocks = D == 256 || kFewShared<D, NT> ? 1 : D == 64 && NT == 1 ? 3 : 2;

template <int D, int NT>
__global__ void __launch_bounds__(kFewThreads<D, NT>, kFewBlocks<D, NT>) weigh_few_kernel(const __grid_constant__ Params P, int groups) {
    constexpr int kThreads = kFewThreads<D, NT>, kWarps = kThreads / 32;
    constexpr bool kShared = kFewShared<D, NT>;
    extern __shared__ __align__(16) uint8_t few_smem[];        // kShared: Rows<D> [kWarps][groups], groups a multiple of NT
    __shared__ uint64_t scan[kThreads + 1];
    __shared__ uint64_t warp_sums[kWarps];
    const WeighArgs& a = P.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int heads = P.cache.heads, window = a.window ? a.window : INT32_MAX, shift = P.cache.page_shift, in_page = P.cache.page_size - 1;
    const uint32_t pages = static_cast<uint32_t>(P.cache.pages);
    const bool one_page = P.cache.page_size >= kTile;
    const int each = scan_units<kTile, kThreads>(P, scan, warp_sums);
    const uint64_t total = scan[kThreads], warps = static_cast<uint64_t>(gridDim.x) * kWarps, w = static_cast<uint64_t>(blockIdx.x) * kWarps + warp;
    uint64_t u = total / warps * w + min(w, total % warps);
    const uint64_t u1 = u + total / warps + (w < total % warps);
    if (u >= u1) return;
    Request r;
    int b, h, first;
    locate<kTile, kThreads>(P, scan, each, u, r, b, h, first);
    while (u < u1) {
        const int last = static_cast<int>(min(static_cast<uint64_t>(units_of<kTile>(r) - first), u1 - u)) + first;
        const int32_t* row = a.table + static_cast<int64_t>(b) * a.table_stride;
        const HeadBase base{P.cache.data + h * P.cache.head_bytes(), a.weights + static_cast<int64_t>(h) * P.cache.page_size,
                            a.out + static_cast<int64_t>(h) * P.cache.page_size, heads * P.cache.head_bytes(), static_cast<int64_t>(heads) << shift};
        // entries of the table for a tile's two records (of one page where it holds both); behind the last token its own again
        auto look = [&](int tile, int (&page)[2]) {
            page[0] = row[min(tile * kTile, r.len - 1) >> shift];
            page[1] = one_page ? page[0] : row[min(tile * kTile + kKvTokens, r.len - 1) >> shift];
        };
        auto place_of = [&](int tile, const int (&page)[2]) {
            Place p;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                p.page[i] = static_cast<uint32_t>(page[i]) < pages && tile * kTile + i * kKvTokens < r.len ? page[i] : -1;
            return p;
        };
        const int pos_hi = r.pos0 + r.n - 1;
        auto seen = [&](int tile) { return tile * kTile <= pos_hi && (!a.window || tile * kTile < a.sinks || tile * kTile + kTile - 1 > r.pos0 - window); };
        auto kept = [&](int tile) { return a.weights && tile * kTile + 8 * t + g < r.pos0; };
        int page[2];
        look(first, page);
        Place here = place_of(first, page);
        look(min(first + 1, last - 1), page);
        Tile<D> even, odd;
        load_tile<D>(base, here, first * kTile, in_page, kept(first), even);
        FewRows<D, kShared ? 1 : NT> R;
        Rows<D>* const ready = reinterpret_cast<Rows<D>*>(few_smem) + warp * groups;
        if constexpr (kShared) {
            __syncwarp();                      // the rows before have been read
            for (int n = 0; n < groups; ++n) make_ready<D>(P, r, h, 8 * n, ready[n]);
            __syncwarp();
        } else {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int mine = min(8 * n + g, r.rows - 1), qi = mine / P.group, head = h * P.group + mine - qi * P.group;
                load_fragments<D>(a.q + (r.q0 + qi) * a.q_stride + head * D, R.q[n]);
                const bool real = 8 * n + g < r.rows;
                const LogSum l = log_sum_of(real ? a.lse[static_cast<int64_t>(r.q0 + qi) * a.heads + head] : -INFINITY, P.scale_rest);
                if (l.less == -INFINITY) drop_fragments(R.q[n]);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int from = (2 * t + c) << 2;             // the columns' rows are those of lanes (2t + c, .)
                    R.less[n][c] = __shfl_sync(0xFFFFFFFFu, l.less, from);
                    R.share[n][c] = __shfl_sync(0xFFFFFFFFu, l.factor, from);
                    R.pos[n][c] = r.pos0 + __shfl_sync(0xFFFFFFFFu, qi, from);
                }
            }
        }
        auto step = [&](int tile, const Tile<D>& cur, Tile<D>& next) {
            const int tok0 = tile * kTile;
            const Place behind = place_of(tile + 1, page);
            if (tile + 1 < last) load_tile<D>(base, behind, tok0 + kTile, in_page, kept(tile + 1), next);
            look(min(tile + 2, last - 1), page);
            float sum[4] = {};
            if (seen(tile)) {
                const bool plain = (here.page[0] | here.page[1]) >= 0 && tok0 + kTile - 1 <= r.pos0 && (tok0 > pos_hi - window || tok0 + kTile <= a.sinks);
                if constexpr (kShared) {
                    for (int n = 0; n < groups; n += NT)
                        if (plain) tile_sums<D, NT, false>(cur, ready + n, P.scale_log2, tok0, window, a.sinks, sum);
                        else tile_sums<D, NT, true>(cur, ready + n, P.scale_log2, tok0, window, a.sinks, sum);
                } else if (plain) tile_sums<D, NT, false>(cur, R, P.scale_log2, tok0, window, a.sinks, sum);
                else tile_sums<D, NT, true>(cur, R, P.scale_log2, tok0, window, a.sinks, sum);
            }
            // over the four lanes of a token; lane (g, t) keeps that of token 8 t + g
            const bool upper = t & 2, second = t & 1;
            const float s0 = (upper ? sum[2] : sum[0]) + __shfl_xor_sync(0xFFFFFFFFu, upper ? sum[0] : sum[2], 2);
            const float s1 = (upper ? sum[3] : sum[1]) + __shfl_xor_sync(0xFFFFFFFFu, upper ? sum[1] : sum[3], 2);
            const float all = (second ? s1 : s0) + __shfl_xor_sync(0xFFFFFFFFu, second ? s0 : s1, 1);
            const int mine = upper ? here.page[1] : here.page[0];
            if (mine >= 0 && tok0 + 8 * t + g < r.len) base.out[mine * base.page_entries + ((tok0 + 8 * t + g) & in_page)] = fmaf(a.decay, cur.before, all);
            here = behind;
        };
        for (int tile = first; tile < last; tile += 2) {
            step(tile, even, odd);
            if (tile + 1 < last) step(tile + 1, odd, even);
        }
        u += static_cast<uint64_t>(last - first);
        first = 0;
        if (u >= u1) break;
        if (++h == heads) {                    // the next request with tiles: there is one
            h = 0;
            do r.read(P, ++b); while (units_of<kTile>(r) == 0);
        }
    }
}

template <int D, int NT>
cudaError_t launch_few(const Params& P, int groups, int num_sms, cudaStream_t s) {
    groups = (groups + NT - 1) / NT * NT;
    size_t smem = 0;
    if constexpr (kFewShared<D, NT>) {
        smem = sizeof(Rows<D>) * groups * (kFewThreads<D, NT> / 32);
        static std::atomic<uint64_t> smem_set{0};
        if (cudaError_t e = set_smem_limit_once(weigh_few_kernel<D, NT>, static_cast<int>(sizeof(Rows<D>) * (weigh_few_rows(D) / 8) * (kFewThreads<D, NT> / 32)), smem_set); e != cudaSuccess) return e;
    }
    weigh_few_kernel<D, NT><<<num_sms * kFewBlocks<D, NT>, kFewThreads<D, NT>, smem, s>>>(P, groups);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch(const Params& P, int num_sms, cudaStream_t s) {
    const int64_t rows = static_cast<int64_t>(P.a.max_queries) * P.group;
    if (rows > weigh_few_rows(D)) {
        weigh_kernel<D><<<num_sms * 2, kThreads, 0, s>>>(P);
        return cudaGetLastError();
    }
    const int groups = static_cast<int>((rows + 7) / 8);
    if (groups == 1) return launch_few<D, 1>(P, groups, num_sms, s);
    if (D == 256 || groups == 2) return launch_few<D, 2>(P, groups, num_sms, s);
    if constexpr (D < 256) {
        // three or four at a time, whichever computes fewer that are none
        if ((groups + 3) / 4 * 4 <= (groups + 2) / 3 * 3) return launch_few<D, 4>(P, groups, num_sms, s);
        return launch_few<D, 3>(P, groups, num_sms, s);
    }
}

}  // namespace

cudaError_t launch_weigh(const WeighArgs& a, const KvGeometry& g, int num_sms, uint64_t timeout_ns, int stall, uint32_t* status, cudaStream_t s) {
    int shift = 0;
    while ((1 << shift) < g.page_size) ++shift;
    const double exact = static_cast<double>(a.scale) * 1.4426950408889634;
    const float scale_log2 = static_cast<float>(exact), rest = exact != 0.0 ? static_cast<float>((exact - scale_log2) / exact) : 0.0f;
    const Params P{a, KvCache{g.data, g.pages, g.page_size, shift, g.heads, g.D}, a.heads / g.heads, scale_log2, rest, timeout_ns, stall, status};
    if (weigh_tc_takes(a, g)) return launch_weigh_tc(P, num_sms, s);
    if (g.D == 64) return launch<64>(P, num_sms, s);
    return g.D == 128 ? launch<128>(P, num_sms, s) : launch<256>(P, num_sms, s);
}

}  // namespace pn
