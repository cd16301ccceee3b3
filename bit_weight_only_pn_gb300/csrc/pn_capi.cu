// pn_capi.cu -- the C ABI declared in include/pn.h: argument checks, kernel choice, launches.
#include <atomic>
#include <cstdint>
#include <cstring>
#include <mutex>

#include <cuda_runtime.h>

#include "../../include/pn.h"
#include "pn_internal.h"

namespace {

constexpr int kMaxDevices = 64;
std::atomic<int> g_sm_count[kMaxDevices];
std::atomic<int> g_cc_major[kMaxDevices];
std::atomic<uint64_t> g_timeout_ns{1000000000ull};
std::atomic<int> g_test_stall{0};
thread_local cudaError_t g_last_cuda_error = cudaSuccess;   // behind this thread's last PN_ECUDA

int per_block(int type) { return type == PN_TYPE_PN3T ? 80 : (type == PN_TYPE_PN4T ? 64 : 0); }

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
    return pa < pb + nb && pb < pa + na;
}

struct Range {
    const void* p;
    size_t n;                  // bytes
};
// Whether an output shares memory with an input or with another output.  (Blocks read the inputs while others write.)
template <size_t O, size_t I>
bool shared(const Range (&out)[O], const Range (&in)[I]) {
    auto meet = [](const Range& a, const Range& b) { return a.p && b.p && a.n && b.n && overlaps(a.p, a.n, b.p, b.n); };
    for (size_t o = 0; o < O; ++o) {
        for (const Range& i : in)
            if (meet(out[o], i)) return true;
        for (size_t j = 0; j < o; ++j)
            if (meet(out[o], out[j])) return true;
    }
    return false;
}

// Elements between rows of `cols`: byte offsets of up to 2^31 rows stay below 2^63.
bool stride_ok(int64_t stride, int64_t cols) { return stride >= cols && stride <= (int64_t{1} << 29); }

// Pages of the 4-bit cache hold a power of two of tokens, whole records of 16.
bool page_size_ok(int page_size) { return page_size >= 16 && page_size <= 1024 && (page_size & (page_size - 1)) == 0; }

// A cache's shape, of at most 2^63 - 1 bytes.
bool kv_shape_ok(int64_t pages, int page_size, int kv_heads, int head_dim) {
    return pages >= 1 && pages <= INT32_MAX && page_size_ok(page_size) && kv_heads >= 1 && kv_heads <= 65536 &&
           (head_dim == 64 || head_dim == 128 || head_dim == 256) &&
           pages * kv_heads * (page_size / 16) <= INT64_MAX / (17 * head_dim);
}

}  // namespace

namespace pn {
pn_status cuda_error(cudaError_t e) {
    g_last_cuda_error = e;
    cudaGetLastError();             // clear it (a sticky error stays regardless)
    return PN_ECUDA;
}

WorkspaceLayout workspace_layout(int num_sms) {
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    WorkspaceLayout L;
    L.status = 0;
    L.tagged = 256;
    L.partials = up(L.tagged + stream_tagged_bytes(num_sms));
    L.counters = up(L.partials + tc_partial_bytes(num_sms));
    L.total = up(L.counters + static_cast<size_t>(tc_max_ctas(num_sms) + 1) * sizeof(uint32_t));
    return L;
}
}  // namespace pn

namespace {

// SM count and compute-capability major of the current device (cached).
pn_status device_info(int* sms, int* major) {
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return pn::cuda_error(e);
    if (dev < 0 || dev >= kMaxDevices) return PN_EUNSUPPORTED;
    int s = g_sm_count[dev].load(std::memory_order_relaxed);
    int m = g_cc_major[dev].load(std::memory_order_relaxed);
    if (s <= 0) {
        cudaError_t e = cudaDeviceGetAttribute(&s, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&m, cudaDevAttrComputeCapabilityMajor, dev);
        if (e != cudaSuccess) return pn::cuda_error(e);
        g_cc_major[dev].store(m, std::memory_order_relaxed);
        g_sm_count[dev].store(s, std::memory_order_relaxed);
    }
    *sms = s;
    *major = m;
    return PN_OK;
}

// Shared checks of one GEMV operand set; fills `t`.
pn_status check_tensor(int type, const void* W, int64_t N, int64_t K, const uint16_t* x, int M,
                       float* y, pn::GemvTensor* t) {
    const int bpb = per_block(type);
    if (bpb == 0 || K <= 0 || K % bpb != 0 || N < 0) return PN_EINVAL;
    if (M < 1 || M > PN_MAX_M) return PN_EINVAL;
    const int64_t nb = K / bpb;
    if (N > INT32_MAX / 2 || nb > INT32_MAX / 8 || K > INT32_MAX / PN_MAX_M) return PN_EINVAL;
    if (N > 0 && (!W || !x || !y)) return PN_EINVAL;
    if (!aligned(W, 2) || !aligned(x, 2) || !aligned(y, 4)) return PN_EALIGN;
    const size_t wbytes = static_cast<size_t>(N) * nb * PN_BLOCK_BYTES;
    const size_t xbytes = static_cast<size_t>(M) * K * 2, ybytes = static_cast<size_t>(M) * N * 4;
    if (N > 0 && (overlaps(y, ybytes, W, wbytes) || overlaps(y, ybytes, x, xbytes))) return PN_EINVAL;
    t->W = static_cast<const uint8_t*>(W);
    t->x = x;
    t->y = y;
    t->type = type;
    t->N = static_cast<int>(N);
    t->nb = static_cast<int>(nb);
    return PN_OK;
}

bool tc_eligible(const pn::GemvTensor& t) {
    return t.nb % 8 == 0 && aligned(t.W, 16) && aligned(t.x, 16);
}

// Sorts the tensors of a call into the tensor-core and CUDA-core kernels.
pn_status route(const pn::GemvTensor* ts, int count, int algo, int major, pn::GemvTensor* tc, int* ntc,
                pn::GemvTensor* simt, int* nsimt) {
    if (algo != PN_ALGO_AUTO && algo != PN_ALGO_TENSOR_CORE && algo != PN_ALGO_CUDA_CORE &&
        algo != PN_ALGO_CUDA_CORE_STAGED)
        return PN_EINVAL;
    *ntc = *nsimt = 0;
    for (int e = 0; e < count; ++e) {
        if (ts[e].N == 0) continue;
        const bool ok_tc = tc_eligible(ts[e]) && major >= 10;
        if ((algo == PN_ALGO_TENSOR_CORE || algo == PN_ALGO_CUDA_CORE_STAGED) && !ok_tc)
            return major >= 10 ? PN_EALIGN : PN_EUNSUPPORTED;
        if (algo == PN_ALGO_CUDA_CORE_STAGED && ts[e].nb / 8 > pn::ffma_max_chunks()) return PN_EUNSUPPORTED;
        if (algo != PN_ALGO_CUDA_CORE && ok_tc) tc[(*ntc)++] = ts[e];
        else simt[(*nsimt)++] = ts[e];
    }
    return PN_OK;
}

pn_status run_layer(const pn::GemvTensor* ts, int count, int M, void* ws, size_t ws_bytes, int algo,
                    cudaStream_t s) {
    int sms = 0, major = 0;
    pn_status st = device_info(&sms, &major);
    if (st != PN_OK) return st;
    pn::GemvTensor tc[pn::kMaxLayer];
    pn::GemvTensor simt[pn::kMaxLayer];
    int ntc = 0, nsimt = 0;
    if ((st = route(ts, count, algo, major, tc, &ntc, simt, &nsimt)) != PN_OK) return st;
    if (algo == PN_ALGO_CUDA_CORE_STAGED) {
        if (M > 8) return PN_EUNSUPPORTED;
        if (ntc == 0) return PN_OK;
        if (!ws || !aligned(ws, 256)) return PN_EINVAL;
        if (pn::workspace_layout(sms).total > ws_bytes) return PN_EINVAL;
        uint32_t* status = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(ws));
        const cudaError_t e = pn::launch_gemv_ffma(tc, ntc, M, status, sms, g_timeout_ns.load(), s);
        return e == cudaSuccess ? PN_OK : pn::cuda_error(e);
    }
    if (ntc > 0) {
        if (!ws || !aligned(ws, 256)) return PN_EINVAL;
        const pn::WorkspaceLayout L = pn::workspace_layout(sms);
        if (L.total > ws_bytes) return PN_EINVAL;
        uint8_t* base = static_cast<uint8_t*>(ws);
        uint32_t* status = reinterpret_cast<uint32_t*>(base + L.status);
        // one or two tokens: one block per SM streams a range of units (rows of
        // at most stream_max_chunks() chunks); more tokens or longer rows:
        // thread blocks share each staged activation chunk among eight tiles
        bool stream = M <= 2;
        for (int i = 0; i < ntc; ++i) stream = stream && tc[i].nb / 8 <= pn::stream_max_chunks();
        // two tokens over several tensors: the one-token kernel only where it
        // keeps their activations resident (measured on GB300: 16.3 against
        // 20.5 us on two pn3t tensors whose activations fit; 37.9 against
        // 38.0 and 48.9 against 41.8 us on sets that do not fit, the
        // 27B-class layer the latter)
        if (stream && M == 2 && ntc > 1 && !pn::stream_resident_fits(tc, ntc, M, sms)) stream = false;
        cudaError_t e = stream
            ? pn::launch_gemv_stream(tc, ntc, M, status, reinterpret_cast<uint64_t*>(base + L.tagged), sms,
                                     g_timeout_ns.load(), g_test_stall.load(), s)
            : pn::launch_gemv_tc(tc, ntc, M, status, reinterpret_cast<float*>(base + L.partials),
                                 reinterpret_cast<uint32_t*>(base + L.counters), sms, g_timeout_ns.load(),
                                 g_test_stall.load(), s);
        if (e != cudaSuccess) return pn::cuda_error(e);
    }
    for (int i = 0; i < nsimt; ++i)
        if (cudaError_t e = pn::launch_gemv_simt(simt[i], M, s); e != cudaSuccess) return pn::cuda_error(e);
    return PN_OK;
}

// No output of a layer call may overlap another entry's operands or output.
pn_status check_layer_overlaps(const pn_gemv_desc* descs, int count, int M) {
    for (int a = 0; a < count; ++a) {
        if (descs[a].N == 0) continue;
        const size_t ya = static_cast<size_t>(M) * descs[a].N * 4;
        for (int b = 0; b < count; ++b) {
            if (b == a || descs[b].N == 0) continue;
            const int bpb = per_block(descs[b].type);
            const size_t wb = static_cast<size_t>(descs[b].N) * (descs[b].K / bpb) * PN_BLOCK_BYTES;
            const size_t xb = static_cast<size_t>(M) * descs[b].K * 2;
            const size_t yb = static_cast<size_t>(M) * descs[b].N * 4;
            if (overlaps(descs[a].y, ya, descs[b].W, wb) || overlaps(descs[a].y, ya, descs[b].x, xb) ||
                overlaps(descs[a].y, ya, descs[b].y, yb))
                return PN_EINVAL;
        }
    }
    return PN_OK;
}

// Checks shared by pn_gemm_f16 and pn_prefill (w16 is the fp16 operand: the
// caller's matrix or the scratch chunk).
pn_status check_gemm(int64_t N, int64_t K, const void* x, int64_t M, const float* y, int64_t ldy,
                     void* workspace, size_t workspace_bytes, int* sms, int* major) {
    if (N < 0 || K <= 0 || K % 8 != 0 || K > INT32_MAX || M < 1 || M > INT32_MAX || ldy < N) return PN_EINVAL;
    if (N > 65535LL * 128) return PN_EINVAL;
    if (N == 0) return PN_OK;
    if (!x || !y || !workspace) return PN_EINVAL;
    if (!aligned(x, 16) || !aligned(y, 4)) return PN_EALIGN;
    if (!aligned(workspace, 256)) return PN_EINVAL;
    pn_status st = device_info(sms, major);
    if (st != PN_OK) return st;
    if (*major < 10) return PN_EUNSUPPORTED;
    if (pn::workspace_layout(*sms).total > workspace_bytes) return PN_EINVAL;
    const size_t ybytes = (static_cast<size_t>(M - 1) * ldy + N) * 4;
    if (overlaps(y, ybytes, x, static_cast<size_t>(M) * K * 2)) return PN_EINVAL;
    return PN_OK;
}

}  // namespace

extern "C" {

int pn_abi_version(void) { return 1; }

const char* pn_status_string(pn_status s) {
    switch (s) {
        case PN_OK: return "ok";
        case PN_EINVAL: return "invalid argument";
        case PN_EALIGN: return "misaligned pointer";
        case PN_EUNSUPPORTED: return "unsupported on this device or build";
        case PN_ECUDA: return "CUDA error";
        case PN_ETIMEOUT: return "device-side wait timed out";
    }
    return "unknown status";
}

int pn_weights_per_block(int type) { return per_block(type); }

size_t pn_row_bytes(int type, int64_t K) {
    const int bpb = per_block(type);
    if (bpb == 0 || K <= 0 || K % bpb != 0) return 0;
    return static_cast<size_t>(K / bpb) * PN_BLOCK_BYTES;
}

pn_status pn_pack(int type, const float* w, int64_t N, int64_t K, void* W, pn_stream stream) {
    const int bpb = per_block(type);
    if (bpb == 0 || K <= 0 || K % bpb != 0 || N < 0) return PN_EINVAL;
    if (N == 0) return PN_OK;
    if (!w || !W) return PN_EINVAL;
    if (!aligned(w, 4) || !aligned(W, 2)) return PN_EALIGN;
    if (overlaps(w, static_cast<size_t>(N) * K * 4, W, static_cast<size_t>(N) * (K / bpb) * PN_BLOCK_BYTES))
        return PN_EINVAL;
    const cudaError_t e = pn::launch_pack(type, w, N, K / bpb, W, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PN_OK : pn::cuda_error(e);
}

pn_status pn_unpack(int type, const void* W, int64_t N, int64_t K, float* w, pn_stream stream) {
    const int bpb = per_block(type);
    if (bpb == 0 || K <= 0 || K % bpb != 0 || N < 0) return PN_EINVAL;
    if (N == 0) return PN_OK;
    if (!w || !W) return PN_EINVAL;
    if (!aligned(w, 4) || !aligned(W, 2)) return PN_EALIGN;
    if (overlaps(w, static_cast<size_t>(N) * K * 4, W, static_cast<size_t>(N) * (K / bpb) * PN_BLOCK_BYTES))
        return PN_EINVAL;
    const cudaError_t e = pn::launch_unpack(type, W, N, K / bpb, w, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PN_OK : pn::cuda_error(e);
}

size_t pn_workspace_bytes(int64_t total_rows) {
    int sms = 0, major = 0;
    if (total_rows < 0 || device_info(&sms, &major) != PN_OK) return 0;
    return pn::workspace_layout(sms).total;
}

pn_status pn_workspace_init(void* workspace, size_t workspace_bytes, pn_stream stream) {
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < 256) return PN_EINVAL;
    const cudaError_t e = cudaMemsetAsync(workspace, 0, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PN_OK : pn::cuda_error(e);
}

pn_status pn_workspace_status(void* workspace, size_t workspace_bytes, pn_stream stream) {
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < 256) return PN_EINVAL;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint32_t word = 0;
    cudaError_t e = cudaStreamSynchronize(s);
    if (e == cudaSuccess) e = cudaMemcpy(&word, workspace, sizeof(word), cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return pn::cuda_error(e);
    if (word == 0) return PN_OK;
    if (cudaError_t e2 = cudaMemset(workspace, 0, workspace_bytes); e2 != cudaSuccess) return pn::cuda_error(e2);
    return word == PN_ETIMEOUT || word == PN_EINVAL ? static_cast<pn_status>(word) : PN_ECUDA;
}

}  // extern "C"

namespace pn {
pn_status gemv_check(int type, const void* W, int64_t N, int64_t K, const uint16_t* x, int M, float* y,
                     int algo, bool* uses_workspace) {
    *uses_workspace = false;
    pn::GemvTensor t{};
    pn_status st = check_tensor(type, W, N, K, x, M, y, &t);
    if (st != PN_OK || N == 0) return st;
    int sms = 0, major = 0;
    if ((st = device_info(&sms, &major)) != PN_OK) return st;
    pn::GemvTensor tc[1], simt[1];
    int ntc = 0, nsimt = 0;
    if ((st = route(&t, 1, algo, major, tc, &ntc, simt, &nsimt)) != PN_OK) return st;
    *uses_workspace = ntc > 0;
    return PN_OK;
}
}  // namespace pn

extern "C" {

pn_status pn_gemv_ex(int type, const void* W, int64_t N, int64_t K, const uint16_t* x, int M,
                     float* y, void* workspace, size_t workspace_bytes, int algo, pn_stream stream) {
    pn::GemvTensor t{};
    pn_status st = check_tensor(type, W, N, K, x, M, y, &t);
    if (st != PN_OK) return st;
    if (N == 0) return PN_OK;
    return run_layer(&t, 1, M, workspace, workspace_bytes, algo, reinterpret_cast<cudaStream_t>(stream));
}

pn_status pn_gemv(int type, const void* W, int64_t N, int64_t K, const uint16_t* x, int M,
                  float* y, void* workspace, size_t workspace_bytes, pn_stream stream) {
    return pn_gemv_ex(type, W, N, K, x, M, y, workspace, workspace_bytes, PN_ALGO_AUTO, stream);
}

pn_status pn_gemv_layer_ex(const pn_gemv_desc* descs, int count, int M, void* workspace,
                           size_t workspace_bytes, int algo, pn_stream stream) {
    if (!descs || count < 1 || count > PN_MAX_LAYER) return PN_EINVAL;
    pn::GemvTensor ts[pn::kMaxLayer];
    for (int e = 0; e < count; ++e) {
        const pn_gemv_desc& d = descs[e];
        pn_status st = check_tensor(d.type, d.W, d.N, d.K, d.x, M, d.y, &ts[e]);
        if (st != PN_OK) return st;
    }
    if (pn_status st = check_layer_overlaps(descs, count, M); st != PN_OK) return st;
    return run_layer(ts, count, M, workspace, workspace_bytes, algo, reinterpret_cast<cudaStream_t>(stream));
}

pn_status pn_gemv_layer(const pn_gemv_desc* descs, int count, int M, void* workspace,
                        size_t workspace_bytes, pn_stream stream) {
    return pn_gemv_layer_ex(descs, count, M, workspace, workspace_bytes, PN_ALGO_AUTO, stream);
}

pn_status pn_gemv_layer_host(const pn_gemv_desc* descs, int count, int M, const uint16_t* x_host, float* y_host,
                             void* workspace, size_t workspace_bytes, pn_stream stream) {
    if (!descs || count < 1 || count > PN_MAX_LAYER || !x_host || !y_host) return PN_EINVAL;
    pn::GemvTensor ts[pn::kMaxLayer];
    for (int e = 0; e < count; ++e) {
        const pn_gemv_desc& d = descs[e];
        pn_status st = check_tensor(d.type, d.W, d.N, d.K, d.x, M, d.y, &ts[e]);
        if (st != PN_OK) return st;
    }
    if (pn_status st = check_layer_overlaps(descs, count, M); st != PN_OK) return st;
    int sms = 0, major = 0;
    if (pn_status st = device_info(&sms, &major); st != PN_OK) return st;
    if (!workspace || !aligned(workspace, 256) || pn::workspace_layout(sms).total > workspace_bytes)
        return PN_EINVAL;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // one copy per run of entries whose device buffers follow each other (the
    // host buffers always do)
    auto copy_runs = [&](bool in) -> cudaError_t {
        size_t host_off = 0, run_host = 0, run_bytes = 0;
        uint8_t* run_dev = nullptr;
        auto flush = [&]() -> cudaError_t {
            if (!run_bytes) return cudaSuccess;
            return in ? cudaMemcpyAsync(run_dev, reinterpret_cast<const uint8_t*>(x_host) + run_host, run_bytes,
                                        cudaMemcpyHostToDevice, s)
                      : cudaMemcpyAsync(reinterpret_cast<uint8_t*>(y_host) + run_host, run_dev, run_bytes,
                                        cudaMemcpyDeviceToHost, s);
        };
        for (int e = 0; e < count; ++e) {
            const pn_gemv_desc& d = descs[e];
            const size_t bytes = in ? static_cast<size_t>(M) * d.K * 2 : static_cast<size_t>(M) * d.N * 4;
            uint8_t* dev = in ? reinterpret_cast<uint8_t*>(const_cast<uint16_t*>(d.x)) : reinterpret_cast<uint8_t*>(d.y);
            if (d.N > 0 && bytes > 0) {
                if (run_bytes && dev == run_dev + run_bytes && host_off == run_host + run_bytes) {
                    run_bytes += bytes;
                } else {
                    if (cudaError_t e2 = flush(); e2 != cudaSuccess) return e2;
                    run_dev = dev;
                    run_host = host_off;
                    run_bytes = bytes;
                }
            }
            host_off += bytes;
        }
        return flush();
    };
    if (cudaError_t e = copy_runs(true); e != cudaSuccess) return pn::cuda_error(e);
    if (pn_status st = run_layer(ts, count, M, workspace, workspace_bytes, PN_ALGO_AUTO, s); st != PN_OK) return st;
    if (cudaError_t e = copy_runs(false); e != cudaSuccess) return pn::cuda_error(e);
    if (cudaError_t e = cudaStreamSynchronize(s); e != cudaSuccess) return pn::cuda_error(e);
    return PN_OK;
}

}  // extern "C"

namespace {

// GEMVs of `count` checked tensors on their activations rotated by blocks of
// `block` (pn_hadamard's arithmetic), in one launch of the one-/two-token
// kernel, which keeps the rotated activations in shared memory.
pn_status run_rotated(const pn::GemvTensor* ts, int count, int M, int block, void* ws, size_t ws_bytes,
                      cudaStream_t s) {
    if (block < 32 || block > 1024 || (block & (block - 1))) return PN_EINVAL;
    for (int e = 0; e < count; ++e)
        if ((static_cast<int64_t>(ts[e].nb) * per_block(ts[e].type)) % block) return PN_EINVAL;
    int sms = 0, major = 0;
    pn_status st = device_info(&sms, &major);
    if (st != PN_OK) return st;
    pn::GemvTensor live[pn::kMaxLayer];
    int n = 0;
    for (int e = 0; e < count; ++e) {
        if (ts[e].N == 0) continue;
        if (major < 10) return PN_EUNSUPPORTED;
        if (!tc_eligible(ts[e])) return PN_EALIGN;
        if (ts[e].nb / 8 > pn::stream_max_chunks()) return PN_EUNSUPPORTED;
        live[n++] = ts[e];
    }
    if (M > 2) return PN_EUNSUPPORTED;
    if (n == 0) return PN_OK;
    if (!pn::stream_rotation_fits(live, n, M, sms, block)) return PN_EUNSUPPORTED;
    if (!ws || !aligned(ws, 256)) return PN_EINVAL;
    const pn::WorkspaceLayout L = pn::workspace_layout(sms);
    if (L.total > ws_bytes) return PN_EINVAL;
    uint8_t* base = static_cast<uint8_t*>(ws);
    const cudaError_t e = pn::launch_gemv_stream(live, n, M, reinterpret_cast<uint32_t*>(base + L.status),
                                                 reinterpret_cast<uint64_t*>(base + L.tagged), sms,
                                                 g_timeout_ns.load(), g_test_stall.load(), s, block);
    return e == cudaSuccess ? PN_OK : pn::cuda_error(e);
}

}  // namespace

extern "C" {

pn_status pn_gemv_hadamard(int type, const void* W, int64_t N, int64_t K, const uint16_t* x, int M, int block,
                           float* y, void* workspace, size_t workspace_bytes, pn_stream stream) {
    pn::GemvTensor t{};
    pn_status st = check_tensor(type, W, N, K, x, M, y, &t);
    if (st != PN_OK) return st;
    return run_rotated(&t, 1, M, block, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

pn_status pn_gemv_layer_hadamard(const pn_gemv_desc* descs, int count, int M, int block, void* workspace,
                                 size_t workspace_bytes, pn_stream stream) {
    if (!descs || count < 1 || count > PN_MAX_LAYER) return PN_EINVAL;
    pn::GemvTensor ts[pn::kMaxLayer];
    for (int e = 0; e < count; ++e) {
        const pn_gemv_desc& d = descs[e];
        pn_status st = check_tensor(d.type, d.W, d.N, d.K, d.x, M, d.y, &ts[e]);
        if (st != PN_OK) return st;
    }
    if (pn_status st = check_layer_overlaps(descs, count, M); st != PN_OK) return st;
    return run_rotated(ts, count, M, block, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

pn_status pn_hadamard(const uint16_t* x, int M, int64_t K, int block, uint16_t* out, pn_stream stream) {
    if (M < 1 || M > 65535 || K <= 0 || block < 2 || block > 4096 || (block & (block - 1)) || K % block)
        return PN_EINVAL;
    if (!x || !out) return PN_EINVAL;
    if (!aligned(x, 2) || !aligned(out, 2)) return PN_EALIGN;
    const size_t bytes = static_cast<size_t>(M) * static_cast<size_t>(K) * 2;
    if (x != out && overlaps(x, bytes, out, bytes)) return PN_EINVAL;
    if (K / block > INT32_MAX) return PN_EINVAL;
    const cudaError_t e = pn::launch_hadamard(x, M, K, block, out, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PN_OK : pn::cuda_error(e);
}

pn_status pn_unpack_f16(int type, const void* W, int64_t N, int64_t K, uint16_t* w16, pn_stream stream) {
    const int bpb = per_block(type);
    if (bpb == 0 || K <= 0 || K % bpb != 0 || N < 0) return PN_EINVAL;
    if (N == 0) return PN_OK;
    if (!W || !w16) return PN_EINVAL;
    if (!aligned(W, 2) || !aligned(w16, 4)) return PN_EALIGN;
    if (overlaps(w16, static_cast<size_t>(N) * K * 2, W, static_cast<size_t>(N) * (K / bpb) * PN_BLOCK_BYTES))
        return PN_EINVAL;
    const cudaError_t e = pn::launch_unpack_f16(type, W, N, K / bpb, w16, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PN_OK : pn::cuda_error(e);
}

pn_status pn_gemm_f16(const uint16_t* w16, int64_t N, int64_t K, const uint16_t* x, int64_t M, float* y,
                      int64_t ldy, void* workspace, size_t workspace_bytes, pn_stream stream) {
    int sms = 0, major = 0;
    pn_status st = check_gemm(N, K, x, M, y, ldy, workspace, workspace_bytes, &sms, &major);
    if (st != PN_OK || N == 0) return st;
    if (!w16) return PN_EINVAL;
    if (!aligned(w16, 16)) return PN_EALIGN;
    const size_t ybytes = (static_cast<size_t>(M - 1) * ldy + N) * 4;
    if (overlaps(y, ybytes, w16, static_cast<size_t>(N) * K * 2)) return PN_EINVAL;
    uint32_t* status = static_cast<uint32_t*>(workspace);
    const cudaError_t e = pn::launch_gemm_f16(w16, N, K, x, M, y, ldy, status, sms, g_timeout_ns.load(),
                                              g_test_stall.load(), reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PN_OK : pn::cuda_error(e);
}

pn_status pn_prefill(int type, const void* W, int64_t N, int64_t K, const uint16_t* x, int64_t M, float* y,
                     void* scratch, size_t scratch_bytes, void* workspace, size_t workspace_bytes,
                     pn_stream stream) {
    const int bpb = per_block(type);
    if (bpb == 0 || K <= 0 || K % bpb != 0) return PN_EINVAL;
    int sms = 0, major = 0;
    pn_status st = check_gemm(N, K, x, M, y, N, workspace, workspace_bytes, &sms, &major);
    if (st != PN_OK || N == 0) return st;
    if (!W || !scratch) return PN_EINVAL;
    if (!aligned(W, 2) || !aligned(scratch, 16)) return PN_EALIGN;
    const int tile = pn::gemm_f16_tile_rows();
    int64_t chunk = static_cast<int64_t>(scratch_bytes / (static_cast<size_t>(K) * 2)) / tile * tile;
    if (chunk < tile) return PN_EINVAL;
    if (chunk > N) chunk = N;
    const size_t wbytes = static_cast<size_t>(N) * (K / bpb) * PN_BLOCK_BYTES;
    const size_t ybytes = static_cast<size_t>(M) * N * 4;
    const size_t sbytes = static_cast<size_t>(chunk) * K * 2;
    if (overlaps(y, ybytes, W, wbytes) || overlaps(scratch, sbytes, W, wbytes) ||
        overlaps(scratch, sbytes, x, static_cast<size_t>(M) * K * 2) || overlaps(scratch, sbytes, y, ybytes))
        return PN_EINVAL;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint16_t* w16 = static_cast<uint16_t*>(scratch);
    uint32_t* status = static_cast<uint32_t*>(workspace);
    const int64_t nb = K / bpb;
    const size_t row_bytes = static_cast<size_t>(nb) * PN_BLOCK_BYTES;
    for (int64_t r0 = 0; r0 < N; r0 += chunk) {
        const int64_t rows = N - r0 < chunk ? N - r0 : chunk;
        cudaError_t e = pn::launch_unpack_f16(type, static_cast<const uint8_t*>(W) + r0 * row_bytes, rows, nb, w16, s);
        if (e == cudaSuccess)
            e = pn::launch_gemm_f16(w16, rows, K, x, M, y + r0, N, status, sms, g_timeout_ns.load(),
                                    g_test_stall.load(), s);
        if (e != cudaSuccess) return pn::cuda_error(e);
    }
    return PN_OK;
}

pn_status pn_read_ranges(const void* const* ptrs, const size_t* bytes, int count, uint32_t* sink,
                         pn_stream stream) {
    if (!ptrs || !bytes || !sink || count < 1 || count > PN_MAX_LAYER) return PN_EINVAL;
    for (int e = 0; e < count; ++e) {
        if (!ptrs[e] && bytes[e] >= 16) return PN_EINVAL;
        if (!aligned(ptrs[e], 16)) return PN_EALIGN;
    }
    if (!aligned(sink, 4)) return PN_EALIGN;
    int sms = 0, major = 0;
    pn_status st = device_info(&sms, &major);
    if (st != PN_OK) return st;
    const cudaError_t e = pn::launch_read_ranges(ptrs, bytes, count, sink, sms, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PN_OK : pn::cuda_error(e);
}

// ------------------------------------------------- 4-bit cache, serving step --

size_t pn_kv_cache_bytes(int64_t pages, int page_size, int kv_heads, int head_dim) {
    if (!kv_shape_ok(pages, page_size, kv_heads, head_dim)) return 0;
    return static_cast<size_t>(pages) * kv_heads * (page_size / 16) * 17 * head_dim;
}

pn_status pn_kv_plan(const int32_t* lens, const int32_t* add, const int32_t* held, int batch, int32_t* table,
                     int64_t table_stride, int max_pages, int32_t* free_pages, int64_t pages, const int64_t* ring,
                     int page_size, int64_t capacity, int64_t* slots, int32_t* positions, int32_t* requests,
                     int32_t* starts, int32_t* lens_out, int32_t* held_out, int64_t* ring_out, int32_t* refused,
                     pn_stream stream) {
    if (batch < 1 || batch > pn::kKvMaxBatch || max_pages < 1 || table_stride < max_pages || pages < 1 ||
        pages > INT32_MAX || !page_size_ok(page_size) || capacity < 0 || capacity > INT32_MAX - 16 ||
        static_cast<int64_t>(max_pages) * page_size > INT32_MAX)
        return PN_EINVAL;
    if (!lens || !add || !held || !table || !free_pages || !ring || !starts || !lens_out || !held_out || !ring_out ||
        !refused || (capacity > 0 && (!slots || !positions || !requests)))
        return PN_EINVAL;
    for (const void* p : {static_cast<const void*>(lens), static_cast<const void*>(add), static_cast<const void*>(held),
                          static_cast<const void*>(table), static_cast<const void*>(free_pages),
                          static_cast<const void*>(positions), static_cast<const void*>(requests),
                          static_cast<const void*>(starts), static_cast<const void*>(lens_out),
                          static_cast<const void*>(held_out), static_cast<const void*>(refused)})
        if (!aligned(p, 4)) return PN_EALIGN;
    if (!aligned(ring, 8) || !aligned(ring_out, 8) || !aligned(slots, 8)) return PN_EALIGN;
    const size_t nb = static_cast<size_t>(batch) * 4, nc = static_cast<size_t>(capacity);
    const Range in[] = {{lens, nb}, {add, nb}, {held, nb}, {ring, 16}},
        out[] = {{table, (static_cast<size_t>(batch - 1) * table_stride + max_pages) * 4},
                 {free_pages, static_cast<size_t>(pages) * 4}, {slots, nc * 8}, {positions, nc * 4},
                 {requests, nc * 4}, {starts, nb + 4}, {lens_out, nb}, {held_out, nb}, {ring_out, 16}, {refused, 4}};
    if (shared(out, in)) return PN_EINVAL;
    int sms = 0, major = 0;
    if (pn_status st = device_info(&sms, &major); st != PN_OK) return st;
    const pn::KvPlanArgs a{lens, add, held, batch, table, table_stride, max_pages, free_pages, pages, ring, page_size,
                           capacity, slots, positions, requests, starts, lens_out, held_out, ring_out, refused};
    const cudaError_t e = pn::launch_kv_plan(a, sms, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PN_OK : pn::cuda_error(e);
}

pn_status pn_kv_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                       int64_t v_stride, int dtype, int64_t tokens, int heads, const float* q_weight,
                       const float* k_weight, float eps, const float* cos, const float* sin, int64_t table_rows,
                       int rotary, int interleaved, const int32_t* positions, const int64_t* slots, void* cache,
                       int64_t pages, int page_size, int kv_heads, int head_dim, uint16_t* q_out, pn_stream stream) {
    if (!kv_shape_ok(pages, page_size, kv_heads, head_dim)) return PN_EINVAL;
    if (dtype != PN_DTYPE_F32 && dtype != PN_DTYPE_F16) return PN_EINVAL;
    if (tokens < 0 || tokens > INT32_MAX || heads < 0 || heads > 65536) return PN_EINVAL;
    if (rotary < 0 || rotary > head_dim || rotary % 2 || table_rows < 0 || !(eps >= 0.0f)) return PN_EINVAL;
    if (tokens == 0) return PN_OK;
    if (!k || !v || !slots || !cache || (heads > 0 && (!q || !q_out))) return PN_EINVAL;
    if (rotary > 0 && (!cos || !sin || !positions)) return PN_EINVAL;
    const int64_t kv_cols = static_cast<int64_t>(kv_heads) * head_dim, q_cols = static_cast<int64_t>(heads) * head_dim;
    if (k_stride < kv_cols || v_stride < kv_cols || (heads > 0 && q_stride < q_cols)) return PN_EINVAL;
    const uintptr_t size = dtype == PN_DTYPE_F32 ? 4 : 2;
    if (!aligned(q, size) || !aligned(k, size) || !aligned(v, size) || !aligned(q_weight, 4) || !aligned(k_weight, 4) ||
        !aligned(cos, 4) || !aligned(sin, 4) || !aligned(positions, 4) || !aligned(slots, 8) || !aligned(cache, 16) ||
        !aligned(q_out, 16))
        return PN_EALIGN;
    const size_t cache_bytes = pn_kv_cache_bytes(pages, page_size, kv_heads, head_dim);
    const size_t nt = static_cast<size_t>(tokens), turn = rotary > 0 ? static_cast<size_t>(table_rows) * (rotary / 2) * 4 : 0,
                 row = static_cast<size_t>(head_dim) * 4;
    const Range in[] = {{q, heads > 0 ? ((tokens - 1) * q_stride + q_cols) * size : 0}, {k, ((tokens - 1) * k_stride + kv_cols) * size},
                        {v, ((tokens - 1) * v_stride + kv_cols) * size}, {q_weight, row}, {k_weight, row}, {cos, turn}, {sin, turn},
                        {positions, rotary > 0 ? nt * 4 : 0}, {slots, nt * 8}},
                out[] = {{cache, cache_bytes}, {q_out, nt * q_cols * 2}};
    if (shared(out, in)) return PN_EINVAL;
    int sms = 0, major = 0;
    if (pn_status st = device_info(&sms, &major); st != PN_OK) return st;
    const pn::KvAppendArgs a{q, k, v, q_stride, k_stride, v_stride, dtype == PN_DTYPE_F16, tokens, heads, q_weight,
                             k_weight, eps, cos, sin, rotary / 2, table_rows, interleaved != 0, positions, slots,
                             reinterpret_cast<__half*>(q_out)};
    const pn::KvGeometry g{static_cast<uint8_t*>(cache), pages, page_size, kv_heads, head_dim};
    const cudaError_t e = pn::launch_kv_append(a, g, sms, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PN_OK : pn::cuda_error(e);
}

pn_status pn_kv_read(const void* cache, int64_t pages, int page_size, int kv_heads, int head_dim,
                     const int64_t* slots, int64_t tokens, float* k, float* v, pn_stream stream) {
    if (!kv_shape_ok(pages, page_size, kv_heads, head_dim) || tokens < 0 || tokens > INT32_MAX) return PN_EINVAL;
    if (tokens == 0) return PN_OK;
    if (!cache || !slots || !k || !v) return PN_EINVAL;
    if (!aligned(cache, 16) || !aligned(slots, 8) || !aligned(k, 16) || !aligned(v, 16)) return PN_EALIGN;
    const size_t n = static_cast<size_t>(tokens) * kv_heads * head_dim * 4;
    const size_t bytes = pn_kv_cache_bytes(pages, page_size, kv_heads, head_dim);
    const Range in[] = {{cache, bytes}, {slots, static_cast<size_t>(tokens) * 8}}, out[] = {{k, n}, {v, n}};
    if (shared(out, in)) return PN_EINVAL;
    int sms = 0, major = 0;
    if (pn_status st = device_info(&sms, &major); st != PN_OK) return st;
    const pn::KvGeometry g{static_cast<uint8_t*>(const_cast<void*>(cache)), pages, page_size, kv_heads, head_dim};
    const cudaError_t e = pn::launch_kv_read(g, slots, tokens, k, v, sms, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PN_OK : pn::cuda_error(e);
}

size_t pn_attention_workspace_bytes(void) {
    int sms = 0, major = 0;
    return device_info(&sms, &major) == PN_OK ? pn::attn_workspace_bytes(sms) : 0;
}

pn_status pn_attention(const uint16_t* q, int64_t q_stride, int64_t tokens, int heads, const void* cache,
                       int64_t pages, int page_size, int kv_heads, int head_dim, const int32_t* table,
                       int64_t table_stride, int max_pages, const int32_t* lens, const int32_t* starts, int batch,
                       int max_queries, float scale, int window, int sinks, uint16_t* out, float* lse,
                       void* workspace, size_t workspace_bytes, pn_stream stream) {
    if (!kv_shape_ok(pages, page_size, kv_heads, head_dim)) return PN_EINVAL;
    if (tokens < 0 || tokens > INT32_MAX || heads < 1 || heads > 65536 || heads % kv_heads) return PN_EINVAL;
    if (batch < 1 || batch > pn::kKvMaxBatch || max_queries < 1 || max_pages < 1 || table_stride < max_pages ||
        window < 0 || sinks < 0 || !(scale - scale == 0.0f))
        return PN_EINVAL;
    if (static_cast<int64_t>(max_pages) * page_size > INT32_MAX - 128 ||
        static_cast<int64_t>(max_queries) * (heads / kv_heads) > INT32_MAX - 128)
        return PN_EINVAL;
    const int64_t cols = static_cast<int64_t>(heads) * head_dim;
    if (q_stride < cols) return PN_EINVAL;
    if (tokens == 0) return PN_OK;
    if (!q || !cache || !table || !lens || !starts || !out || !workspace) return PN_EINVAL;
    if (!aligned(q, 16) || q_stride % 8 || !aligned(cache, 16) || !aligned(table, 4) || !aligned(lens, 4) ||
        !aligned(starts, 4) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(workspace, 256))
        return PN_EALIGN;
    const size_t nt = static_cast<size_t>(tokens), nb = static_cast<size_t>(batch) * 4;
    const Range ins[] = {{q, ((nt - 1) * q_stride + cols) * 2}, {cache, pn_kv_cache_bytes(pages, page_size, kv_heads, head_dim)},
                         {table, (static_cast<size_t>(batch - 1) * table_stride + max_pages) * 4}, {lens, nb}, {starts, nb + 4}},
                outs[] = {{out, nt * cols * 2}, {lse, nt * heads * 4}, {workspace, workspace_bytes}};
    if (shared(outs, ins)) return PN_EINVAL;
    // no request has more cached tokens than its row of the table has room for: a window of as many hides nothing, and
    // no more first tokens are there (with both below 2^31 - 128 no index of a tile passes 32 bits)
    const int room = max_pages * page_size;
    const pn::AttnArgs a{reinterpret_cast<const __half*>(q), q_stride, tokens, heads, table, table_stride, max_pages,
                         lens, starts, batch, max_queries, scale, window < room ? window : 0, sinks < room ? sinks : room,
                         reinterpret_cast<__half*>(out), lse};
    const pn::KvGeometry g{static_cast<uint8_t*>(const_cast<void*>(cache)), pages, page_size, kv_heads, head_dim};
    if (!pn::attn_fits(a, g)) return PN_EUNSUPPORTED;
    int sms = 0, major = 0;
    if (pn_status st = device_info(&sms, &major); st != PN_OK) return st;
    if (major < 10) return PN_EUNSUPPORTED;
    if (pn::attn_workspace_bytes(sms) > workspace_bytes) return PN_EINVAL;
    const cudaError_t e = pn::launch_attention(a, g, workspace, sms, g_timeout_ns.load(), g_test_stall.load(),
                                               reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PN_OK : pn::cuda_error(e);
}

pn_status pn_verify(const int32_t* tokens, const float* target, int64_t target_stride, const float* draft,
                    int64_t draft_stride, const float* uniforms, const int32_t* counts, int batch, int drafts,
                    int vocab, int32_t* accepted, int32_t* out, pn_stream stream) {
    if (batch < 0 || batch > (1 << 24) || drafts < 0 || drafts > PN_MAX_DRAFTS || vocab < 1 || vocab > PN_MAX_VOCAB)
        return PN_EINVAL;
    if (target_stride < vocab || (draft && draft_stride < vocab)) return PN_EINVAL;
    if (batch == 0) return PN_OK;
    if ((drafts > 0 && !tokens) || !target || !uniforms || !accepted || !out) return PN_EINVAL;
    if (!aligned(tokens, 4) || !aligned(target, 4) || !aligned(draft, 4) || !aligned(uniforms, 4) ||
        !aligned(counts, 4) || !aligned(accepted, 4) || !aligned(out, 4))
        return PN_EALIGN;
    const size_t nb = static_cast<size_t>(batch) * 4, nt = nb * drafts, row = static_cast<size_t>(vocab) * 4;
    const Range ins[] = {{tokens, nt}, {target, (static_cast<size_t>(batch) * (drafts + 1) - 1) * target_stride * 4 + row},
                         {draft, drafts > 0 ? (static_cast<size_t>(batch) * drafts - 1) * draft_stride * 4 + row : 0},
                         {uniforms, nt + nb}, {counts, nb}},
                outs[] = {{accepted, nb}, {out, nt + nb}};
    if (shared(outs, ins)) return PN_EINVAL;
    int sms = 0, major = 0;
    if (pn_status st = device_info(&sms, &major); st != PN_OK) return st;
    if (major < 9) return PN_EUNSUPPORTED;
    const pn::VerifyArgs a{tokens, target, target_stride, draft, draft_stride, uniforms, counts, batch, drafts, vocab,
                           accepted, out};
    const cudaError_t e = pn::launch_verify(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PN_OK : pn::cuda_error(e);
}

pn_status pn_logprobs(const void* logits, int64_t stride, int dtype, int64_t rows, int vocab, float scale,
                      const int32_t* tokens, int count, float* logprobs, float* entropy, int top,
                      int32_t* top_tokens, float* top_logprobs, pn_stream stream) {
    if (dtype != PN_DTYPE_F32 && dtype != PN_DTYPE_F16) return PN_EINVAL;
    if (rows < 0 || rows > INT32_MAX || vocab < 1 || vocab > PN_MAX_VOCAB || count < 0 || count > PN_MAX_VOCAB || top < 0 ||
        top > PN_MAX_TOP || !(scale >= 0x1p-64f && scale <= 0x1p64f) || !stride_ok(stride, vocab))
        return PN_EINVAL;
    if (rows == 0) return PN_OK;
    if (!logits || (count > 0 && (!tokens || !logprobs)) || (top > 0 && (!top_tokens || !top_logprobs))) return PN_EINVAL;
    const size_t size = dtype == PN_DTYPE_F32 ? 4 : 2, nr = static_cast<size_t>(rows) * 4;
    if (!aligned(logits, size) || !aligned(tokens, 4) || !aligned(logprobs, 4) || !aligned(entropy, 4) || !aligned(top_tokens, 4) ||
        !aligned(top_logprobs, 4))
        return PN_EALIGN;
    const Range ins[] = {{logits, ((rows - 1) * stride + vocab) * size}, {tokens, nr * count}},
                outs[] = {{logprobs, nr * count}, {entropy, nr}, {top_tokens, nr * top}, {top_logprobs, nr * top}};
    if (shared(outs, ins)) return PN_EINVAL;
    int sms = 0, major = 0;
    if (pn_status st = device_info(&sms, &major); st != PN_OK) return st;
    if (major < 9) return PN_EUNSUPPORTED;
    const pn::LogprobsArgs a{logits, stride, dtype == PN_DTYPE_F16, rows, vocab, scale, tokens, count, logprobs, entropy, top,
                             top_tokens, top_logprobs};
    const cudaError_t e = pn::launch_logprobs(a, sms, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PN_OK : pn::cuda_error(e);
}

pn_status pn_norm(const void* y, int64_t y_stride, int y_dtype, const void* residual, int64_t residual_stride,
                  int residual_dtype, const float* gate, int64_t gate_stride, float scale, int64_t tokens, int hidden,
                  int post, const float* post_weight, const float* post_bias, int pre, const float* pre_weight,
                  const float* pre_bias, float eps, void* residual_out, int64_t out_stride, uint16_t* x,
                  pn_stream stream) {
    for (int d : {y_dtype, residual_dtype})
        if (d != PN_DTYPE_F32 && d != PN_DTYPE_F16) return PN_EINVAL;
    for (int k : {post, pre})
        if (k != PN_NORM_NONE && k != PN_NORM_RMS && k != PN_NORM_LAYER) return PN_EINVAL;
    if (tokens < 0 || tokens > INT32_MAX || hidden < 1 || hidden > PN_MAX_HIDDEN || !(eps >= 0.0f) || !(scale - scale == 0.0f)) return PN_EINVAL;
    if ((post == PN_NORM_NONE && (post_weight || post_bias)) || (pre == PN_NORM_NONE && (pre_weight || pre_bias))) return PN_EINVAL;
    if ((y && !stride_ok(y_stride, hidden)) || (residual && !stride_ok(residual_stride, hidden)) ||
        (gate && gate_stride != 0 && !stride_ok(gate_stride, hidden)) || (residual_out && !stride_ok(out_stride, hidden)))
        return PN_EINVAL;
    if (tokens == 0) return PN_OK;
    if ((!y && !residual) || (!residual_out && !x)) return PN_EINVAL;
    // what nothing would be done with
    if ((!y && (gate || post != PN_NORM_NONE)) || (!x && pre != PN_NORM_NONE)) return PN_EINVAL;
    const size_t ys = y_dtype == PN_DTYPE_F32 ? 4 : 2, rs = residual_dtype == PN_DTYPE_F32 ? 4 : 2;
    if (!aligned(y, ys) || !aligned(residual, rs) || !aligned(residual_out, rs) || !aligned(gate, 4) || !aligned(post_weight, 4) ||
        !aligned(post_bias, 4) || !aligned(pre_weight, 4) || !aligned(pre_bias, 4) || !aligned(x, 2))
        return PN_EALIGN;
    const bool in_place = residual_out && residual_out == residual && out_stride == residual_stride;
    const size_t row = static_cast<size_t>(hidden) * 4;
    auto rows_of = [&](int64_t stride, size_t size) { return ((tokens - 1) * stride + hidden) * size; };
    const Range ins[] = {{y, rows_of(y_stride, ys)}, {in_place ? nullptr : residual, rows_of(residual_stride, rs)},
                         {gate, rows_of(gate_stride, 4)}, {post_weight, row}, {post_bias, row}, {pre_weight, row}, {pre_bias, row}},
                outs[] = {{residual_out, rows_of(out_stride, rs)}, {x, static_cast<size_t>(tokens) * hidden * 2}};
    if (shared(outs, ins)) return PN_EINVAL;
    int sms = 0, major = 0;
    if (pn_status st = device_info(&sms, &major); st != PN_OK) return st;
    const pn::NormArgs a{y, y_stride, y_dtype == PN_DTYPE_F16, residual, residual_stride, residual_dtype == PN_DTYPE_F16, gate, gate_stride,
                         scale, tokens, hidden, post, post_weight, post_bias, pre, pre_weight, pre_bias, eps, residual_out, out_stride,
                         reinterpret_cast<__half*>(x)};
    const cudaError_t e = pn::launch_norm(a, sms, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PN_OK : pn::cuda_error(e);
}

pn_status pn_kv_weigh(const uint16_t* q, int64_t q_stride, int64_t tokens, int heads, const void* cache,
                      int64_t pages, int page_size, int kv_heads, int head_dim, const int32_t* table,
                      int64_t table_stride, int max_pages, const int32_t* lens, const int32_t* starts, int batch,
                      int max_queries, const float* lse, float scale, int window, int sinks, const float* weights,
                      float decay, float* out, pn_stream stream) {
    return pn_kv_weigh_ex(q, q_stride, tokens, heads, cache, pages, page_size, kv_heads, head_dim, table, table_stride, max_pages, lens, starts, batch,
                          max_queries, lse, scale, window, sinks, weights, decay, out, nullptr, 0, stream);
}

pn_status pn_kv_weigh_ex(const uint16_t* q, int64_t q_stride, int64_t tokens, int heads, const void* cache,
                         int64_t pages, int page_size, int kv_heads, int head_dim, const int32_t* table,
                         int64_t table_stride, int max_pages, const int32_t* lens, const int32_t* starts, int batch,
                         int max_queries, const float* lse, float scale, int window, int sinks, const float* weights,
                         float decay, float* out, void* workspace, size_t workspace_bytes, pn_stream stream) {
    if (!kv_shape_ok(pages, page_size, kv_heads, head_dim)) return PN_EINVAL;
    if (tokens < 0 || tokens > INT32_MAX || heads < 1 || heads > 65536 || heads % kv_heads) return PN_EINVAL;
    if (batch < 1 || batch > pn::kKvMaxBatch || max_queries < 1 || max_pages < 1 || table_stride < max_pages || window < 0 || sinks < 0 ||
        !(scale - scale == 0.0f) || !(decay >= 0.0f && decay <= 1.0f))
        return PN_EINVAL;
    if (static_cast<int64_t>(max_pages) * page_size > INT32_MAX - 1024 ||
        static_cast<int64_t>(max_queries) * (heads / kv_heads) > INT32_MAX - 128)
        return PN_EINVAL;
    const int64_t cols = static_cast<int64_t>(heads) * head_dim;
    if (!stride_ok(q_stride, cols)) return PN_EINVAL;
    if (tokens == 0) return PN_OK;
    if (!q || !cache || !table || !lens || !starts || !lse || !out) return PN_EINVAL;
    if (!aligned(q, 16) || q_stride % 8 || !aligned(cache, 16) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(starts, 4) ||
        !aligned(lse, 4) || !aligned(weights, 4) || !aligned(out, 4) || !aligned(workspace, 256))
        return PN_EALIGN;
    if (workspace && workspace_bytes < 256) return PN_EINVAL;
    const size_t nt = static_cast<size_t>(tokens), nb = static_cast<size_t>(batch) * 4, nw = static_cast<size_t>(pages) * kv_heads * page_size * 4;
    const Range ins[] = {{q, ((nt - 1) * q_stride + cols) * 2}, {cache, pn_kv_cache_bytes(pages, page_size, kv_heads, head_dim)},
                         {table, (static_cast<size_t>(batch - 1) * table_stride + max_pages) * 4}, {lens, nb}, {starts, nb + 4},
                         {lse, nt * heads * 4}, {weights == out ? nullptr : weights, nw}},
                outs[] = {{out, nw}, {workspace, workspace_bytes}};
    if (shared(outs, ins)) return PN_EINVAL;
    int sms = 0, major = 0;
    if (pn_status st = device_info(&sms, &major); st != PN_OK) return st;
    if (major < 10) return PN_EUNSUPPORTED;
    const int room = max_pages * page_size;            // as in pn_attention
    const pn::WeighArgs a{reinterpret_cast<const __half*>(q), q_stride, tokens, heads, table, table_stride, max_pages, lens, starts, batch,
                          max_queries, lse, scale, window < room ? window : 0, sinks < room ? sinks : room, decay > 0.0f ? weights : nullptr, decay, out};
    const pn::KvGeometry g{static_cast<uint8_t*>(const_cast<void*>(cache)), pages, page_size, kv_heads, head_dim};
    const cudaError_t e = pn::launch_weigh(a, g, sms, g_timeout_ns.load(), g_test_stall.load(), static_cast<uint32_t*>(workspace), reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PN_OK : pn::cuda_error(e);
}

pn_status pn_kv_evict(void* cache, int64_t pages, int page_size, int kv_heads, int head_dim, float* weights,
                      const int32_t* table, int64_t table_stride, int max_pages, const int32_t* lens,
                      const int32_t* held, int batch, int limit, int budget, int sinks, int recent,
                      int32_t* free_pages, int64_t ring_pages, const int64_t* ring, int32_t* table_out,
                      int64_t out_stride, int32_t* lens_out, int32_t* held_out, int64_t* ring_out, int32_t* kept,
                      int32_t* refused, pn_stream stream) {
    if (!kv_shape_ok(pages, page_size, kv_heads, head_dim)) return PN_EINVAL;
    if (batch < 1 || batch > pn::kKvMaxBatch || max_pages < 1 || table_stride < max_pages || out_stride < max_pages || ring_pages < 1 ||
        ring_pages > INT32_MAX || budget < 1 || budget > limit || budget > PN_MAX_BUDGET || sinks < 0 || recent < 0 ||
        static_cast<int64_t>(sinks) + recent > budget)
        return PN_EINVAL;
    if (static_cast<int64_t>(max_pages) * page_size > INT32_MAX - 1024) return PN_EINVAL;
    // (blocks are numbered in 31 bits)
    if (static_cast<int64_t>(batch) * kv_heads >= INT32_MAX) return PN_EUNSUPPORTED;
    if (!cache || !weights || !table || !lens || !held || !free_pages || !ring || !table_out || !lens_out || !held_out || !ring_out || !kept || !refused)
        return PN_EINVAL;
    for (const void* p : {static_cast<const void*>(weights), static_cast<const void*>(table), static_cast<const void*>(lens), static_cast<const void*>(held),
                          static_cast<const void*>(free_pages), static_cast<const void*>(table_out), static_cast<const void*>(lens_out),
                          static_cast<const void*>(held_out), static_cast<const void*>(kept), static_cast<const void*>(refused)})
        if (!aligned(p, 4)) return PN_EALIGN;
    if (!aligned(cache, 16) || !aligned(ring, 8) || !aligned(ring_out, 8)) return PN_EALIGN;
    const size_t nb = static_cast<size_t>(batch) * 4;
    auto rows_of = [&](int64_t stride) { return (static_cast<size_t>(batch - 1) * stride + max_pages) * 4; };
    const Range in[] = {{table, rows_of(table_stride)}, {lens, nb}, {held, nb}, {ring, 16}},
        out[] = {{cache, pn_kv_cache_bytes(pages, page_size, kv_heads, head_dim)}, {weights, static_cast<size_t>(pages) * kv_heads * page_size * 4},
                 {free_pages, static_cast<size_t>(ring_pages) * 4}, {table_out, rows_of(out_stride)}, {lens_out, nb}, {held_out, nb}, {ring_out, 16},
                 {kept, nb * kv_heads * budget}, {refused, 4}};
    if (shared(out, in)) return PN_EINVAL;
    int sms = 0, major = 0;
    if (pn_status st = device_info(&sms, &major); st != PN_OK) return st;
    if (major < 9) return PN_EUNSUPPORTED;
    const pn::EvictArgs a{weights, table, table_stride, max_pages, lens, held, batch, limit, budget, sinks, recent, free_pages, ring_pages, ring,
                          table_out, out_stride, lens_out, held_out, ring_out, kept, refused};
    const pn::KvGeometry g{static_cast<uint8_t*>(cache), pages, page_size, kv_heads, head_dim};
    const cudaError_t e = pn::launch_evict(a, g, sms, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PN_OK : pn::cuda_error(e);
}

const char* pn_last_cuda_error(void) { return cudaGetErrorName(g_last_cuda_error); }

void pn_set_wait_timeout_ns(uint64_t ns) { g_timeout_ns.store(ns); }

void pn_set_test_stall(int on) { g_test_stall.store(on ? 1 : 0); }

pn_status pn_tc_split(const int* types, const int64_t* N, const int64_t* K, int count, int M, int num_sms,
                      uint32_t* starts, int* grid) {
    if (!types || !N || !K || !starts || !grid) return PN_EINVAL;
    if (count < 1 || count > PN_MAX_LAYER || M < 3 || M > PN_MAX_M || num_sms < 1) return PN_EINVAL;
    pn::GemvTensor ts[pn::kMaxLayer] = {};
    for (int e = 0; e < count; ++e) {
        const int bpb = per_block(types[e]);
        if (bpb == 0 || K[e] <= 0 || K[e] % (8 * bpb) != 0 || N[e] < 1) return PN_EINVAL;
        const int64_t nb = K[e] / bpb;
        if (N[e] > INT32_MAX / 2 || nb > INT32_MAX / 8) return PN_EINVAL;
        ts[e].type = types[e];
        ts[e].N = static_cast<int>(N[e]);
        ts[e].nb = static_cast<int>(nb);
    }
    return pn::tc_split(ts, count, M, num_sms, grid, starts) ? PN_OK : PN_EINVAL;
}

}  // extern "C"
