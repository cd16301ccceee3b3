// pn_attn.cuh -- what the attention kernels share.
#pragma once

#include <cstdint>

#include <cuda_fp16.h>

#include "pn_device.cuh"
#include "pn_internal.h"
#include "pn_kv.cuh"

namespace pn {

constexpr uint32_t kAttnInvalid = 1;         // PN_EINVAL
constexpr uint32_t kAttnTimeout = 5;         // PN_ETIMEOUT
constexpr uint64_t kAttnDrainNs = 200ull * 1000 * 1000;

struct AttnParams {
    AttnArgs a;
    KvCache cache;
    int group;                 // query heads per key/value head
    float scale_log2;          // scale * log2 e
    uint32_t* status;
    uint32_t* counters;        // one per thread block
    float* block_slots;        // two per thread block
    float* warp_slots;         // one per consumer warp
    uint64_t timeout_ns;
    int stall;                 // testing aid: see pn_set_test_stall
    int depth;                 // stages per warp (kernel for few rows), and by how much
    int early;                 // shared memory behind them moves forward for it
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Sums of units that stop at 2^32 - 1, which no call reaches whose starts are in
// order (the host sees to that).  One that does has no units: nothing is written.
constexpr uint32_t kTooManyUnits = 0xFFFFFFFFu;
__device__ __forceinline__ uint32_t add_units(uint32_t a, uint32_t b) { return a + b < a ? kTooManyUnits : a + b; }
__device__ __forceinline__ uint32_t all_units(const AttnParams& P, uint32_t all) {
    if (all != kTooManyUnits) return all;
    atomicCAS(P.status, 0u, kAttnInvalid);
    return 0u;
}

// Nanoseconds in SM cycles, at the fastest clock: limits are at least as long as asked.
__device__ __forceinline__ int64_t cycles_of(uint64_t ns) { return static_cast<int64_t>(ns) * 21 / 10; }

// Polls: a thread parked in mbarrier.try_wait notices a completed phase late,
// and so does one that reads the global timer in between (about a thousand
// cycles); the limit goes by the SM's clock.
// nap: nanoseconds between polls, for a wait that is in no hurry.
static __device__ bool wait_phase(uint32_t bar, uint32_t parity, uint64_t limit_ns, volatile uint32_t* abort, uint32_t nap = 0) {
    if (mbar_try_wait(bar, parity)) return true;
    const int64_t end = clock64() + cycles_of(limit_ns);
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i) {
            if (nap) __nanosleep(nap);
            if (mbar_try_wait(bar, parity)) return true;
        }
        if ((abort && *abort) || clock64() > end) return false;
    }
}

// The first cached token in the window (at least 1) of a query at `pos`, which is
// negative for a query before the cache; pos - window may pass 32 bits.
__device__ __forceinline__ int window_first(int pos, int window) { return pos >= window ? pos - window + 1 : 0; }

__device__ __forceinline__ float log_sum(float ref, float sum) {
    return sum == 0.0f ? -INFINITY : 0.6931471805599453f * (ref + log2f(sum));
}

// Bytes of the counters at the head of an attention workspace, behind the
// status word's 256: one per thread block, two blocks to an SM at most.
constexpr size_t attn_counter_bytes(int num_sms) { return (static_cast<size_t>(num_sms) * 2 * 4 + 255) / 256 * 256; }

// The kernel for many query rows to a key/value head (pn_attn_tc.cu).
bool attn_tc_takes(const AttnArgs& a, const KvGeometry& g);
double attn_tc_units(const AttnArgs& a, const KvGeometry& g);            // at most
size_t attn_tc_workspace_bytes(int num_sms);
cudaError_t launch_attention_tc(AttnParams P, uint8_t* ws, int num_sms, cudaStream_t s);

}  // namespace pn
