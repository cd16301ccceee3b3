// pn_evict.cu -- requests past a limit keep a budget of tokens.
//
// For each key/value head by itself: the first `sinks` tokens, the last `recent`,
// and of those between them the ones with the largest weights, the lower position
// first where weights are equal.  They go in their order into pages from the
// ring's head; the request's old pages go behind its tail.  Nothing that any block
// reads is written (new pages were free, the table is written to another one), so a
// call can be repeated and no block waits for another.
//
// Two launches.  select: a block to a request and head (a cluster of up to 8 with a
// share of the positions each, where there are few heads in all) finds the kept
// positions.  It holds the upper 15 bits of the weights, as whole numbers in their
// order, in shared memory (64 steps to a power of two); a histogram over their range
// gives the step with the last kept weight, and the few weights of that step are ranked
// among themselves.  Then every warp counts in its share what is kept, and writes the
// positions behind those of the warps before.  Where the step holds more than a thread
// to a weight (all weights equal, say) or a request has more tokens than fit, histograms
// of 2048 bins fix 11 bits of the last kept weight at a time, over weights read again
// each time.  move: a warp to a record of 16 new tokens gathers their codes, scales and
// weights.
//
// 64 ragged requests to 16384 tokens, 8 heads of 128, cut back to 512: select 37 us (its 17
// MB of weights are 2.5: bound by five passes with barriers between; whole keys read
// again for each pass took about 70), move 31 us for 34 MB in and as much out (a chain of
// position, page and record to each load; and V's words of a token lie 8 bytes in every
// 64, so the sectors read are some three times what is wanted).
#include <cooperative_groups.h>
#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "pn_device.cuh"
#include "pn_internal.h"
#include "pn_kv.cuh"

namespace cg = cooperative_groups;

namespace pn {
namespace {

constexpr int kSelectThreads = 512;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 2048;
constexpr int kMostKeys = 96 * 1024;           // of a block, whose upper bits are kept in shared memory
constexpr int kLowBits = 17;                   // the others
constexpr int kMostParts = 8;                  // blocks to a request and head
constexpr int kMoveThreads = 256;
constexpr int kMoveRecords = kMoveThreads / 32;        // of a block

struct Params {
    EvictArgs a;
    KvCache cache;
    int each;                  // pages of a request that was cut back
    int keys;                  // places for keys in shared memory (even)
};

__device__ __forceinline__ int64_t wrap(int64_t i, int64_t n) {
    const int64_t r = i % n;
    return r < 0 ? r + n : r;
}

__device__ __forceinline__ int length_of(const Params& P, int b) {
    return static_cast<int>(min(static_cast<int64_t>(max(P.a.lens[b], 0)), static_cast<int64_t>(P.a.max_pages) << P.cache.page_shift));
}
__device__ __forceinline__ int held_of(const Params& P, int b) { return min(max(P.a.held[b], 0), P.a.max_pages); }

// Requests that the free pages are enough for.
__device__ __forceinline__ int64_t most_served(const Params& P) {
    const int64_t avail = min(max(P.a.ring[1] - P.a.ring[0], static_cast<int64_t>(0)), P.a.pages);
    return avail / P.each;
}

// The sum of v over the block's threads, in all of them; `part` a number per warp, free again behind it.
template <int kWarps, typename T>
__device__ __forceinline__ T block_sum(T v, T* part) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += part[w];
    __syncthreads();
    return v;
}

// What does not belong to one request: the ring and how many were refused.
__device__ void totals(const Params& P, int64_t* part) {
    const EvictArgs& a = P.a;
    const int64_t room = most_served(P);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t over = 0, given = 0;               // requests past the limit so far, pages that come back
    for (int b0 = 0; b0 < a.batch; b0 += kSelectThreads) {
        const int b = b0 + static_cast<int>(threadIdx.x);
        const bool past = b < a.batch && length_of(P, b) > a.limit;
        const uint32_t in = __ballot_sync(0xFFFFFFFFu, past);
        if (lane == 0) part[warp] = __popc(in);
        __syncthreads();
        int64_t turn = over + __popc(in & ((1u << lane) - 1u));
        for (int w = 0; w < kSelectWarps; ++w) {
            turn += w < warp ? part[w] : 0;
            over += part[w];
        }
        __syncthreads();
        given += past && turn < room ? held_of(P, b) : 0;
    }
    given = block_sum<kSelectWarps>(given, part);
    if (threadIdx.x != 0) return;
    const int64_t served = min(over, room);
    a.ring_out[0] = a.ring[0] + served * P.each;
    a.ring_out[1] = a.ring[1] + given;
    a.refused[0] = static_cast<int>(over - served);
}

// The order of weights as that of whole numbers; NaN lowest.
__device__ __forceinline__ uint32_t key_of(float w) {
    const uint32_t u = __float_as_uint(w + 0.0f);      // -0 is 0
    return w == w ? (u & 0x80000000u ? ~u : u | 0x80000000u) : 0u;
}

// What the blocks of a request and head tell each other.
struct Shared {
    alignas(16) uint32_t bins[kBins];      // a histogram, then the candidates' keys and positions
    uint32_t low, high;        // the range of the block's keys
    uint32_t candidates;
    uint32_t above, equal;     // kept in the block's share (equal: of those equal to the last kept key)
};

// The blocks of a request and head, one or a cluster.
struct Team {
    cg::cluster_group cluster;
    int parts, rank;
    __device__ __forceinline__ void sync() const {
        if (parts > 1) cluster.sync();
        else __syncthreads();
    }
    __device__ __forceinline__ const Shared& of(Shared* mine, int r) const { return parts > 1 ? *cluster.map_shared_rank(mine, r) : *mine; }
};

// The range of the team's keys, from low and high of each thread.
__device__ __forceinline__ void team_range(const Team& team, Shared* s, uint32_t& low, uint32_t& high, uint32_t* part0, uint32_t* part1) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    low = __reduce_min_sync(0xFFFFFFFFu, low);
    high = __reduce_max_sync(0xFFFFFFFFu, high);
    if (lane == 0) {
        part0[warp] = low;
        part1[warp] = high;
    }
    __syncthreads();
    low = __reduce_min_sync(0xFFFFFFFFu, part0[lane % kSelectWarps]);
    high = __reduce_max_sync(0xFFFFFFFFu, part1[lane % kSelectWarps]);
    if (threadIdx.x == 0) {
        s->low = low;
        s->high = high;
    }
    team.sync();
    if (team.parts > 1) {
        low = __reduce_min_sync(0xFFFFFFFFu, team.of(s, lane % team.parts).low);
        high = __reduce_max_sync(0xFFFFFFFFu, team.of(s, lane % team.parts).high);
    }
}

// The bin, from the largest down, with the `left`-th count of the team's histogram,
// whose blocks' bins are complete; left becomes its place in the bin and in_bin what the
// bin holds.  Every thread gets the answer, and the bins may be written again.
__device__ __forceinline__ uint32_t bin_of(const Team& team, Shared* s, uint32_t& left, uint32_t& in_bin, uint32_t* part, uint32_t* found) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kEach = kBins / kSelectThreads;      // of a thread
    const int top = kBins - 1 - static_cast<int>(threadIdx.x) * kEach;
    team.sync();
    static_assert(kEach == 4, "a thread's bins are read as one uint4");
    uint32_t n[kEach] = {}, mine = 0;
#pragma unroll
    for (int r = 0; r < kMostParts; ++r)               // (all loads on their way together)
        if (r < team.parts) {
            const uint4 x = *reinterpret_cast<const uint4*>(&team.of(s, r).bins[top - 3]);
            n[0] += x.w;
            n[1] += x.z;
            n[2] += x.y;
            n[3] += x.x;
        }
#pragma unroll
    for (int i = 0; i < kEach; ++i) mine += n[i];
    uint32_t in = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, in, d);
        if (lane >= d) in += o;
    }
    if (lane == 31) part[warp] = in;
    __syncthreads();
    uint32_t above = in - mine + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? part[lane] : 0u);
    if (above < left && left <= above + mine) {        // one thread's
        int i = 0;
        while (left > above + n[i]) above += n[i++];
        found[0] = static_cast<uint32_t>(top - i);
        found[1] = left - above;
        found[2] = n[i];
    }
    team.sync();
    left = found[1];
    in_bin = found[2];
    return found[0];
}

__global__ void __launch_bounds__(kSelectThreads) select_kernel(const __grid_constant__ Params P) {
    extern __shared__ uint16_t upper[];        // [P.keys], kMark: kept among those of the last kept weight's step
    __shared__ Shared s;
    __shared__ uint2 gathered[kBins / 2];      // the candidates of all blocks
    __shared__ int64_t part[kSelectWarps];
    __shared__ uint32_t warp_above[kSelectWarps], warp_equal[kSelectWarps];
    __shared__ uint32_t found[3];
    constexpr uint16_t kMark = 0xFFFF;
    const EvictArgs& a = P.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, heads = P.cache.heads;
    Team team{cg::this_cluster(), 0, 0};
    team.parts = static_cast<int>(team.cluster.num_blocks());
    team.rank = static_cast<int>(team.cluster.block_rank());
    const int64_t index = blockIdx.x / team.parts;     // of the request and head
    if (index == static_cast<int64_t>(a.batch) * heads) {
        if (team.rank == 0) totals(P, part);
        return;
    }
    const int b = static_cast<int>(index / heads), h = static_cast<int>(index % heads);
    const int len = length_of(P, b);
    int32_t* kept = a.kept + index * a.budget;
    const int32_t* row = a.table + static_cast<int64_t>(b) * a.table_stride;
    bool served = len > a.limit;
    int64_t turn = 0, behind = 0;              // requests past the limit before this one, and the pages that they give back
    if (served) {
        for (int o = threadIdx.x; o < b; o += kSelectThreads)
            if (length_of(P, o) > a.limit) {
                ++turn;
                behind += held_of(P, o);
            }
        if (b > 0) {
            turn = block_sum<kSelectWarps>(turn, part);
            behind = block_sum<kSelectWarps>(behind, part);
        }
        served = turn < most_served(P);
    }
    if (h == 0 && team.rank == 0) {
        const int held = held_of(P, b);
        int32_t* out = a.table_out + static_cast<int64_t>(b) * a.out_stride;
        for (int i = threadIdx.x; i < a.max_pages; i += kSelectThreads)
            out[i] = !served ? row[i] : i < P.each ? a.free_pages[wrap(a.ring[0] + turn * P.each + i, a.pages)] : -1;
        if (served)
            for (int i = threadIdx.x; i < held; i += kSelectThreads) a.free_pages[wrap(a.ring[1] + behind + i, a.pages)] = row[i];
        if (threadIdx.x == 0) {
            a.lens_out[b] = served ? a.budget : a.lens[b];
            a.held_out[b] = served ? P.each : a.held[b];
        }
    }
    const int everyone = team.rank * kSelectThreads + threadIdx.x, all_threads = team.parts * kSelectThreads;
    if (!served) {
        for (int i = everyone; i < a.budget; i += all_threads) kept[i] = -1;
        return;
    }
    for (int i = everyone; i < a.sinks; i += all_threads) kept[i] = i;
    for (int i = everyone; i < a.recent; i += all_threads) kept[a.budget - a.recent + i] = len - a.recent + i;
    const int all = len - a.sinks - a.recent, need = a.budget - a.sinks - a.recent;        // all > need
    if (need == 0) return;
    // the block's share of the positions between
    const int begin = static_cast<int>(static_cast<int64_t>(all) * team.rank / team.parts), count = static_cast<int>(static_cast<int64_t>(all) * (team.rank + 1) / team.parts) - begin;
    const int first_tok = a.sinks + begin;
    auto weight_key = [&](int i) -> uint32_t {         // of position first_tok + i
        const int tok = first_tok + i, page = row[tok >> P.cache.page_shift];
        const bool there = page >= 0 && page < P.cache.pages;
        // (loaded in any case: under a branch every load waits for the one before)
        const float w = __ldcg(a.weights + ((static_cast<int64_t>(there ? page : 0) * heads + h) << P.cache.page_shift) + (tok & (P.cache.page_size - 1)));
        return there ? key_of(w) : 0u;
    };
    const uint32_t lower = (1u << lane) - 1u;
    // a contiguous share of them to each warp
    const int share = (count + kSelectWarps * 32 - 1) / (kSelectWarps * 32) * 32;
    const int i0 = min(warp * share, count), i1 = min(i0 + share, count);
    // places of what the warps, then the blocks, before this one keep
    auto before_of = [&](const uint32_t* warps, uint32_t Shared::*block) {
        uint32_t n = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? warps[lane] : 0u);
        if (team.parts > 1) n += __reduce_add_sync(0xFFFFFFFFu, lane < team.rank ? team.of(&s, min(lane, team.parts - 1)).*block : 0u);
        return n;
    };
    constexpr int kAtOnce = 8;                 // loads of a thread on their way together
    // (the last share is no smaller than the others: all blocks take the same way)
    if ((all + team.parts - 1) / team.parts <= P.keys) {
        // the upper bits of all keys, and their range
        uint32_t low = 0xFFFFFFFFu, high = 0u;
        for (int first = threadIdx.x; first < count; first += kAtOnce * kSelectThreads) {
            uint32_t k[kAtOnce];
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) k[j] = weight_key(min(first + j * kSelectThreads, count - 1)) >> kLowBits;
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const int i = first + j * kSelectThreads;
                if (i < count) upper[i] = static_cast<uint16_t>(k[j]);
                low = min(low, k[j]);
                high = max(high, k[j]);
            }
        }
        for (int i = threadIdx.x; i < kBins; i += kSelectThreads) s.bins[i] = 0;
        if (threadIdx.x == 0) s.candidates = 0;
        team_range(team, &s, low, high, warp_above, warp_equal);
        // (of more than 2048 steps several share a bin)
        const int shift = max(21 - __clz(high - low), 0);
#pragma unroll 4
        for (int i = threadIdx.x; i < count; i += kSelectThreads) atomicAdd(&s.bins[(upper[i] - low) >> shift], 1u);
        uint32_t left = static_cast<uint32_t>(need), in_bin;
        const uint32_t bin = bin_of(team, &s, left, in_bin, warp_above, found);
        if (in_bin <= kBins / 2) {
            // keys and positions of the bin's, in the histogram's place; those kept get the mark
            uint2* list = reinterpret_cast<uint2*>(s.bins);
            const uint32_t from = low + (bin << shift), range = (1u << shift) - 1u;
#pragma unroll 4
            for (int i = threadIdx.x; i < count; i += kSelectThreads)
                if (upper[i] - from <= range) list[atomicAdd(&s.candidates, 1u)] = make_uint2(weight_key(i), static_cast<uint32_t>(begin + i));
            team.sync();
            const uint2* everyones = list;
            if (team.parts > 1) {              // in_bin of them
                const int r = warp % team.parts, step = kSelectWarps / team.parts * 32;        // a block to each of some warps
                const uint32_t n = lane < team.parts ? team.of(&s, lane).candidates : 0u;
                const uint32_t before = __reduce_add_sync(0xFFFFFFFFu, lane < r ? n : 0u), there = __shfl_sync(0xFFFFFFFFu, n, r);
                const uint2* theirs = reinterpret_cast<const uint2*>(team.of(&s, r).bins);
#pragma unroll 2
                for (uint32_t o = warp / team.parts * 32 + lane; o < there; o += step) gathered[before + o] = theirs[o];
                __syncthreads();
                everyones = gathered;
            }
            for (uint32_t c = threadIdx.x; c < s.candidates; c += kSelectThreads) {
                const uint2 mine = list[c];
                uint32_t place = 0;
#pragma unroll 4
                for (uint32_t o = 0; o < in_bin; ++o) {
                    const uint2 x = everyones[o];
                    place += x.x > mine.x || (x.x == mine.x && x.y < mine.y);
                }
                if (place < left) upper[mine.y - begin] = kMark;
            }
            __syncthreads();
            const uint32_t above_bin = from + range;
            uint32_t mine = 0;
#pragma unroll 4
            for (int i = i0 + lane; i < i1; i += 32) mine += upper[i] > above_bin;
            mine = __reduce_add_sync(0xFFFFFFFFu, mine);
            if (lane == 0) warp_above[warp] = mine;
            __syncthreads();
            if (team.parts > 1) {
                if (threadIdx.x < 32) {
                    const uint32_t n = __reduce_add_sync(0xFFFFFFFFu, lane < kSelectWarps ? warp_above[lane] : 0u);
                    if (lane == 0) s.above = n;
                }
                team.sync();
            }
            int to = a.sinks + static_cast<int>(before_of(warp_above, &Shared::above));
#pragma unroll 4
            for (int i = i0; i < i1; i += 32) {
                const uint32_t in = __ballot_sync(0xFFFFFFFFu, i + lane < i1 && upper[min(i + lane, i1 - 1)] > above_bin);
                if ((in >> lane) & 1u) kept[to + __popc(in & lower)] = first_tok + i + lane;
                to += __popc(in);
            }
            if (team.parts > 1) team.sync();   // no block leaves while another may read from it
            return;
        }
    }
    // bit by bit over whole keys
    uint32_t low = 0xFFFFFFFFu, high = 0u;
#pragma unroll 8
    for (int i = threadIdx.x; i < count; i += kSelectThreads) {
        const uint32_t k = weight_key(i);
        low = min(low, k);
        high = max(high, k);
    }
    __syncthreads();
    team_range(team, &s, low, high, warp_above, warp_equal);
    // the smallest kept key, from `least` on below 2^bits more, and how many of those equal to it are kept
    uint32_t least = low, left = static_cast<uint32_t>(need), in_bin;
    for (int bits = 32 - __clz(high - low);;) {
        const int shift = max(bits - 11, 0);
        const uint32_t range = bits == 32 ? 0xFFFFFFFFu : (1u << bits) - 1u;
        for (int i = threadIdx.x; i < kBins; i += kSelectThreads) s.bins[i] = 0;
        __syncthreads();
#pragma unroll 4
        for (int i = threadIdx.x; i < count; i += kSelectThreads) {
            const uint32_t k = weight_key(i) - least;  // (smaller keys: past the range)
            if (k <= range) atomicAdd(&s.bins[k >> shift], 1u);
        }
        least += bin_of(team, &s, left, in_bin, warp_above, found) << shift;
        if (shift == 0) break;
        bits = shift;
    }
    uint32_t above = 0, equal = 0;
#pragma unroll 4
    for (int i = i0 + lane; i < i1; i += 32) {
        const uint32_t k = weight_key(i);
        above += k > least;
        equal += k == least;
    }
    above = __reduce_add_sync(0xFFFFFFFFu, above);
    equal = __reduce_add_sync(0xFFFFFFFFu, equal);
    __syncthreads();
    if (lane == 0) {
        warp_above[warp] = above;
        warp_equal[warp] = equal;
    }
    __syncthreads();
    if (team.parts > 1) {
        if (threadIdx.x < 32) {
            const uint32_t n = __reduce_add_sync(0xFFFFFFFFu, lane < kSelectWarps ? warp_above[lane] : 0u);
            const uint32_t m = __reduce_add_sync(0xFFFFFFFFu, lane < kSelectWarps ? warp_equal[lane] : 0u);
            if (lane == 0) {
                s.above = n;
                s.equal = m;
            }
        }
        team.sync();
    }
    above = before_of(warp_above, &Shared::above);
    equal = before_of(warp_equal, &Shared::equal);
#pragma unroll 4
    for (int i = i0; i < i1; i += 32) {
        const uint32_t k = weight_key(min(i + lane, i1 - 1));
        const uint32_t up = __ballot_sync(0xFFFFFFFFu, i + lane < i1 && k > least), same = __ballot_sync(0xFFFFFFFFu, i + lane < i1 && k == least);
        const uint32_t before = equal + __popc(same & lower);
        const uint32_t place = above + __popc(up & lower) + min(before, left);
        // (place < need in any case, but for weights that another call changes meanwhile)
        if ((((up >> lane) & 1u) || (((same >> lane) & 1u) && before < left)) && place < static_cast<uint32_t>(need))
            kept[a.sinks + place] = first_tok + i + lane;
        above += __popc(up);
        equal += __popc(same);
    }
    if (team.parts > 1) team.sync();           // no block leaves while another may read from it
}

// Bytes of kv_record_bytes(D) / 16 that a token has in a record lie in pieces: of K
// codes a run for each half and plane, of V codes one for each word, two scales.
template <int D>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const __grid_constant__ Params P) {
    constexpr int NG = D / 64, GP = kv_plane_groups(D), PL = kv_planes(D);
    using KBits = typename std::conditional<GP == 2, uint4, uint2>::type;      // a lane's bytes of a token's K codes
    using VBits = typename std::conditional<GP == 2, uint2, uint32_t>::type;   // a word of V codes for each group of a plane
    using DBits = typename std::conditional<NG == 4, uint2, typename std::conditional<NG == 2, uint32_t, uint16_t>::type>::type;
    const EvictArgs& a = P.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, heads = P.cache.heads;
    const int b = static_cast<int>(blockIdx.x) / heads, h = static_cast<int>(blockIdx.x) % heads;
    const int32_t* kept = a.kept + static_cast<int64_t>(blockIdx.x) * a.budget;
    griddep_wait();                            // for select's writes
    if (kept[0] < 0) return;                   // left as it was
    const int32_t* from_row = a.table + static_cast<int64_t>(b) * a.table_stride;
    const int32_t* to_row = a.table_out + static_cast<int64_t>(b) * a.out_stride;
    const int records = (a.budget + kKvTokens - 1) / kKvTokens;
    const int rec0 = static_cast<int>(blockIdx.y) * kMoveRecords, rec1 = min(rec0 + kMoveRecords, records);
    for (int rec = rec0 + warp; rec < rec1; rec += kMoveThreads / 32) {
        const int to_tok = rec * kKvTokens, to_page = to_row[to_tok >> P.cache.page_shift];
        if (to_page < 0 || to_page >= P.cache.pages) continue;
        const int64_t to_slot = (static_cast<int64_t>(to_page) << P.cache.page_shift) + (to_tok & (P.cache.page_size - 1));
        uint8_t* to = P.cache.record(to_slot, h);
        const int have = min(a.budget - to_tok, kKvTokens);    // tokens of the record
        // lane i (and i + 16): where the record's token i comes from
        const uint8_t* from = nullptr;
        int place = 0;
        float weight = 0.0f;
        if ((lane & 15) < have) {
            const int tok = kept[to_tok + (lane & 15)], at = tok >> P.cache.page_shift;
            const int page = at >= 0 && at < a.max_pages ? from_row[at] : -1;
            if (page >= 0 && page < P.cache.pages) {
                const int in_page = tok & (P.cache.page_size - 1);
                from = P.cache.record((static_cast<int64_t>(page) << P.cache.page_shift) + in_page, h);
                place = in_page & 15;
                weight = a.weights[((static_cast<int64_t>(page) * heads + h) << P.cache.page_shift) + in_page];
            }
        }
        auto source = [&](int token, int& r) {
            r = __shfl_sync(0xFFFFFFFFu, place, token);
            return reinterpret_cast<const uint8_t*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(from), token));
        };
        // (reads of a plane whose D differs are compiled away; a token of no page becomes zeros)
        KBits kb[2][PL];
        VBits vb[2][PL][2];
        DBits db{};
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            int r;
            const uint8_t* s = source(hh * 8 + (lane >> 2), r);
#pragma unroll
            for (int pl = 0; pl < PL; ++pl) {
                kb[hh][pl] = KBits{};
                if (s) kb[hh][pl] = *reinterpret_cast<const KBits*>(s + (((r >> 3) * PL + pl) * 32 + (r & 7) * 4 + (lane & 3)) * sizeof(KBits));
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {      // words lane / 4 of tokens 2 (lane % 4), + 1
                s = source(hh * 8 + 2 * (lane & 3) + i, r);
#pragma unroll
                for (int pl = 0; pl < PL; ++pl) {
                    vb[hh][pl][i] = VBits{};
                    if (s) vb[hh][pl][i] = *reinterpret_cast<const VBits*>(s + kv_v_codes(D) + (((r >> 3) * PL + pl) * 64 + (lane >> 2) * 8 + (r & 7)) * sizeof(VBits));
                }
            }
        }
        if (from) db = *reinterpret_cast<const DBits*>(from + (lane < 16 ? kv_k_scales(D) : kv_v_scales(D)) + place * sizeof(DBits));
#pragma unroll
        for (int hh = 0; hh < 2; ++hh)
#pragma unroll
            for (int pl = 0; pl < PL; ++pl) {
                if (hh * 8 + (lane >> 2) < have) *reinterpret_cast<KBits*>(to + ((hh * PL + pl) * 32 + lane) * sizeof(KBits)) = kb[hh][pl];
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (hh * 8 + 2 * (lane & 3) + i < have)
                        *reinterpret_cast<VBits*>(to + kv_v_codes(D) + ((hh * PL + pl) * 64 + 2 * lane + i) * sizeof(VBits)) = vb[hh][pl][i];
            }
        if ((lane & 15) < have) {
            *reinterpret_cast<DBits*>(to + (lane < 16 ? kv_k_scales(D) : kv_v_scales(D)) + (lane & 15) * sizeof(DBits)) = db;
            if (lane < 16)
                a.weights[((static_cast<int64_t>(to_page) * heads + h) << P.cache.page_shift) + (to_tok & (P.cache.page_size - 1)) + lane] = weight;
        }
    }
}

template <int D>
cudaError_t move(const Params& P, cudaStream_t s) {
    const int records = (P.a.budget + kKvTokens - 1) / kKvTokens;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(P.a.batch) * P.cache.heads, (records + kMoveRecords - 1) / kMoveRecords);
    cfg.blockDim = dim3(kMoveThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;       // its blocks start while select's end
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, move_kernel<D>, P);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, const KvGeometry& g, int num_sms, cudaStream_t s) {
    int shift = 0;
    while ((1 << shift) < g.page_size) ++shift;
    const int64_t room = static_cast<int64_t>(a.max_pages) * g.page_size;
    // blocks to a request and head: until the GPU is full, none with less than 4096
    // positions (one against several: a request of 33000 tokens and 8 heads 31 us against
    // 22, three of 96205 97 and 54, one of 300000 and one head 718 and 38; of 9000, 18.8 and 18.6,
    // of 4500, 14.8 and 16.3 in two)
    const int64_t teams = static_cast<int64_t>(a.batch) * g.heads;
    int parts = 1;
    while (parts < kMostParts && teams * parts * 2 <= num_sms * 2 && room / (parts * 2) >= 4096) parts *= 2;
    const int64_t each = (room + parts - 1) / parts, keys = each < kMostKeys ? each + each % 2 : kMostKeys;
    const Params P{a, KvCache{g.data, g.pages, g.page_size, shift, g.heads, g.D}, (a.budget + g.page_size - 1) / g.page_size, static_cast<int>(keys)};
    static std::atomic<uint64_t> smem_set{0};
    if (cudaError_t e = set_smem_limit_once(select_kernel, kMostKeys * 2, smem_set); e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>((teams + 1) * parts));
    cfg.blockDim = dim3(kSelectThreads);
    cfg.dynamicSmemBytes = P.keys * 2;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = parts;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaError_t e = cudaLaunchKernelEx(&cfg, select_kernel, P); e != cudaSuccess) return e;
    if (g.D == 64) return move<64>(P, s);
    return g.D == 128 ? move<128>(P, s) : move<256>(P, s);
}

}  // namespace pn
