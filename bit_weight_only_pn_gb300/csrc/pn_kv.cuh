// pn_kv.cuh -- layout of the 4-bit key/value cache (include/pn.h, "4-bit cache").
//
// A page holds page_size tokens (a power of two, 16 at least) of every
// key/value head; for each head it is page_size / 16 records of 16 tokens:
//
//   K codes (8 D bytes) | K scales (D / 2) | V codes (8 D) | V scales (D / 2)
//
// so a page's tokens of one head are contiguous and one bulk copy moves any
// run of records.  Values are pn4t's (groups of 64 with one signed fp16 scale
// d, value d * (n - 8), eight 4-bit codes to a word, even codes in the low
// half).  The words lie in the order in which the attention kernel's MMA
// fragments take them, so a warp reads 16 (D = 64: 8) consecutive bytes per
// lane, without bank conflicts and without any shuffling afterwards:
//
//   K [h][plane][token g][word pair t][group in plane][2]   lane 4 g + t holds
//     words 2t, 2t+1 of token 8 h + g: MMA row g (h = 0) or g + 8 (h = 1);
//   V [h][plane][word g][token pair t][2][group in plane]   lane 4 g + t holds
//     word g of tokens 8 h + 2t, + 1: MMA columns 2t, 2t+1 (+ 8 for h = 1).
//
// A plane is two groups (one for D = 64).
#pragma once

#include <cstdint>

namespace pn {

constexpr int kKvTokens = 16;                  // tokens per record

__host__ __device__ constexpr int kv_record_bytes(int D) { return 17 * D; }
__host__ __device__ constexpr int kv_k_scales(int D) { return 8 * D; }
__host__ __device__ constexpr int kv_v_codes(int D) { return 8 * D + D / 2; }
__host__ __device__ constexpr int kv_v_scales(int D) { return 16 * D + D / 2; }
__host__ __device__ constexpr int kv_planes(int D) { return D >= 128 ? D / 128 : 1; }
__host__ __device__ constexpr int kv_plane_groups(int D) { return D >= 128 ? 2 : 1; }

// Byte offset, in its record, of K / V code word i (values 8 i .. 8 i + 7 of
// the group) of group j of token r (0 .. 15).
template <int D>
__host__ __device__ constexpr int kv_k_word(int r, int j, int i) {
    constexpr int gp = kv_plane_groups(D), pl = kv_planes(D);
    return ((((r >> 3) * pl + j / gp) * 32 + (r & 7) * 4 + (i >> 1)) * gp + j % gp) * 8 + (i & 1) * 4;
}
template <int D>
__host__ __device__ constexpr int kv_v_word(int r, int j, int i) {
    constexpr int gp = kv_plane_groups(D), pl = kv_planes(D);
    return kv_v_codes(D) +
           (((((r >> 3) * pl + j / gp) * 32 + i * 4 + ((r & 7) >> 1)) * 2 + (r & 1)) * gp + j % gp) * 4;
}

// Where a slot (page * page_size + place in the page) of a head lies.
struct KvCache {
    uint8_t* data;
    int64_t pages;
    int page_size;             // power of two
    int page_shift;            // log2(page_size)
    int heads;
    int D;
    __host__ __device__ int64_t head_bytes() const { return static_cast<int64_t>(page_size >> 4) * kv_record_bytes(D); }
    __host__ __device__ int64_t slots() const { return pages << page_shift; }
    // the record that holds `slot` of head h
    __device__ __forceinline__ uint8_t* record(int64_t slot, int h) const {
        const int64_t page = slot >> page_shift;
        const int at = static_cast<int>(slot) & (page_size - 1);
        return data + (page * heads + h) * head_bytes() + static_cast<int64_t>(at >> 4) * kv_record_bytes(D);
    }
};

}  // namespace pn
