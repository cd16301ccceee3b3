/*
 * pn.h -- C ABI of the PN weight-only decode GEMV library for GB300 (sm_103a).
 *
 * The PN formats come from the tensorless documentation, page "Why a P100-native
 * weight format":
 *   - "Every block is 34 bytes": a block is a 2-byte fp16 scale d and eight
 *     32-bit code words; pn3t holds 80 weights (ten 3-bit codes per word,
 *     3.40 bits/weight), pn4t holds 64 weights (eight 4-bit codes per word,
 *     4.25 bits/weight).  A row holds a whole number of blocks.
 *   - "Codes never straddle the two halves of a word": even codes fill bits
 *     0..15, odd codes bits 16..31, at the same offsets.
 *   - "Exact decode in fp32": weight = d * (n - z), exact in fp32.
 *   - "Zero is a code, and the scale has a sign": mid-tread codes, z = 4 for
 *     pn3t (steps -4..+3); the signed scale puts the extra step on the side of
 *     the block's largest weight.
 *
 * Where the page leaves the layout open this library reads it as follows (the
 * same readings as the CPU oracle used by the tests):
 *   - block bytes 0..1 = d (IEEE binary16, little-endian), bytes 2..33 = code
 *     words w0..w7 (little-endian);
 *   - weight k of a block is code c = k % cpw of word k / cpw (cpw = 10 pn3t,
 *     8 pn4t); code c sits in half (c & 1) at bit offset bits * (c >> 1);
 *     pn3t bits 15 and 31 are written as 0 and ignored on decode;
 *   - z = 4 (pn3t) and z = 8 (pn4t, steps -8..+7);
 *   - the packer rounds to nearest with d = fp16(a / -z), a = the block's
 *     largest-magnitude weight (first on ties); codes n = clamp(rint(v / d),
 *     -z, z-1) + z (fp32 divides, ties to even); a block whose scale is 0 or
 *     underflows fp16 is the zero block (d = +0, all codes z); a scale above
 *     the fp16 range saturates to +-65504.
 *
 * Layouts.  W: N rows of pn_row_bytes(type, K) bytes, row-major, no padding.
 * Dense weights w: fp32 [N][K] row-major.  Activations x: IEEE binary16 bit
 * patterns [M][K] row-major.  Outputs y: fp32 [M][N] row-major.
 *
 * Conventions.  Every pointer except descriptor arrays is device memory owned
 * by the caller; the library allocates nothing.  Every call is asynchronous on
 * the given CUDA stream (NULL = the legacy default stream) and returns after
 * the launch.  Arguments are checked on the host before anything is launched;
 * a failed check returns an error status and launches nothing.  A CUDA launch
 * error is returned as PN_ECUDA.  No call aborts, throws or prints.
 *
 * Thread safety: calls may be made from several host threads; calls that share
 * a workspace must be ordered on one stream.
 */
#ifndef PN_H
#define PN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st;                      /* == cudaStream_t / CUstream */
typedef struct CUstream_st* pn_stream;

/* Weight types; the values are the GGUF type ids the page gives for PN
 * ("Why the format is specific to this engine": 124 and 125). */
typedef enum { PN_TYPE_PN3T = 124, PN_TYPE_PN4T = 125 } pn_type;

typedef enum {
    PN_OK = 0,
    PN_EINVAL = 1,        /* bad type, size, count, null pointer, small workspace */
    PN_EALIGN = 2,        /* a pointer is not aligned as documented */
    PN_EUNSUPPORTED = 3,  /* valid request this build cannot serve (e.g. not sm_10x) */
    PN_ECUDA = 4,         /* a CUDA runtime call or launch failed */
    PN_ETIMEOUT = 5       /* a device-side wait gave up (reported by pn_workspace_status) */
} pn_status;

/* GEMV algorithm selection for pn_gemv_ex / pn_gemv_layer_ex. */
typedef enum {
    PN_ALGO_AUTO = 0,         /* tensor-core kernel where eligible, else CUDA cores */
    PN_ALGO_TENSOR_CORE = 1,  /* TMA-staged rows, decode into mma.sync fragments   */
    PN_ALGO_CUDA_CORE = 2,    /* one lane per code word, fp32 FMAs                 */
    PN_ALGO_CUDA_CORE_STAGED = 3  /* TMA-staged rows as for the tensor cores; each
                                     decoded fp16 (n - z) times fp16 x added in fp32
                                     on the FMA pipe (fma.rn.f32.f16) for every
                                     token; 1 <= M <= 8, rows of at most 64 chunks
                                     of 8 blocks, tensor-core alignment rules
                                     (PN_EUNSUPPORTED / PN_EALIGN otherwise) */
} pn_algo;

#define PN_BLOCK_BYTES 34
#define PN_MAX_M 16           /* largest activation count M per GEMV */
#define PN_MAX_LAYER 8        /* most tensors per pn_gemv_layer call */

/* Version of this ABI (incremented on any incompatible change). */
int pn_abi_version(void);

/* Human-readable name of a status code (static string). */
const char* pn_status_string(pn_status s);

/* Name of the CUDA runtime error (as cudaGetErrorName gives it) behind the
 * latest PN_ECUDA that a failing CUDA call caused on the calling host thread;
 * "cudaSuccess" if there was none.  Static string. */
const char* pn_last_cuda_error(void);

/* Weights per block (80 / 64) or 0 for an unknown type. */
int pn_weights_per_block(int type);

/* Bytes per PN row: (K / weights_per_block) * 34, or 0 if the type is unknown
 * or K is not a positive multiple of the block size ("A row must hold a whole
 * number of blocks"). */
size_t pn_row_bytes(int type, int64_t K);

/*
 * pn_pack: quantise fp32 weights w [N][K] into PN rows W [N][row_bytes] with
 * the signed-scale round-to-nearest rule above.  w must be 4-byte aligned, W
 * 2-byte aligned; inputs must be finite (the result for non-finite inputs is
 * unspecified).  Deterministic and byte-identical to the CPU oracle.
 */
pn_status pn_pack(int type, const float* w, int64_t N, int64_t K, void* W, pn_stream stream);

/*
 * pn_unpack: decode PN rows W [N][row_bytes] into fp32 w [N][K]; each weight is
 * the single IEEE fp32 product d * (n - z), exact ("Exact decode in fp32"),
 * including the sign of zero.  W 2-byte aligned, w 4-byte aligned.
 */
pn_status pn_unpack(int type, const void* W, int64_t N, int64_t K, float* w, pn_stream stream);

/*
 * Workspace for the GEMV calls.  The tensor-core kernels split the rows and K
 * blocks of all tensors of a call evenly over their thread blocks; a tile of
 * rows whose K range is split between two thread blocks is finished by one of
 * them, which adds the other block's part in a fixed order, so results are
 * deterministic.  That needs device scratch: a status word and, per
 * thread-block boundary, hand-off slots and a counter.  The size depends only
 * on the device's SM count (about 2.3 KiB per SM), so calls of any shape can
 * share one workspace.
 *
 * pn_workspace_bytes(total_rows): bytes needed by one call whose tensors have
 * total_rows rows in all (sum of N), on the current device.
 * pn_workspace_init: zero a workspace (required once before first use; every
 * call that completes leaves it zeroed again).
 * pn_workspace_status: synchronise `stream`, read and clear the device status
 * word of the workspace; returns PN_OK or the device-side error (PN_ETIMEOUT,
 * of pn_attention also PN_EINVAL), and re-zeroes the whole workspace after an
 * error.
 * Workspace pointers must be 256-byte aligned.
 */
size_t pn_workspace_bytes(int64_t total_rows);
pn_status pn_workspace_init(void* workspace, size_t workspace_bytes, pn_stream stream);
pn_status pn_workspace_status(void* workspace, size_t workspace_bytes, pn_stream stream);

/*
 * pn_gemv: y[m][r] = sum_k w[r][k] * x[m][k] for m < M (1 <= M <= 16), r < N,
 * where w is W decoded as in pn_unpack.  This is the decode GEMV of token
 * generation (M = 1) and its skinny verification batch (M <= 16, one token
 * plus up to 15 drafts); the weights cross memory once whatever M is.  Products are exact in fp32 and sums are kept in fp32; every output
 * is within 1e-5 * sum_k |w[r][k] x[m][k]| + 1e-6 of the exact value.
 * Alignment: W and x 16-byte aligned for the tensor-core kernel (otherwise
 * PN_ALGO_AUTO uses the CUDA-core kernel, which needs W and x 2-byte and y
 * 4-byte aligned).  y must not overlap W or x.
 */
pn_status pn_gemv(int type, const void* W, int64_t N, int64_t K, const uint16_t* x, int M,
                  float* y, void* workspace, size_t workspace_bytes, pn_stream stream);

pn_status pn_gemv_ex(int type, const void* W, int64_t N, int64_t K, const uint16_t* x, int M,
                     float* y, void* workspace, size_t workspace_bytes, int algo,
                     pn_stream stream);

/*
 * pn_gemv_layer: the GEMVs of several independent tensors (one decoder layer's
 * projections) in one launch, all with the same M.  The thread blocks share
 * out the rows and K blocks of every tensor in proportion to their bytes.
 * Descriptors are read on the host during the call.  No entry's y may overlap
 * any entry's W, x or y.  At most PN_MAX_LAYER entries.
 */
typedef struct {
    int type;               /* PN_TYPE_PN3T or PN_TYPE_PN4T            */
    const void* W;          /* device, [N][pn_row_bytes(type, K)]      */
    int64_t N;              /* rows                                    */
    int64_t K;              /* input width                             */
    const uint16_t* x;      /* device, fp16 [M][K]                     */
    float* y;               /* device, fp32 [M][N]                     */
} pn_gemv_desc;

pn_status pn_gemv_layer(const pn_gemv_desc* descs, int count, int M, void* workspace,
                        size_t workspace_bytes, pn_stream stream);

pn_status pn_gemv_layer_ex(const pn_gemv_desc* descs, int count, int M, void* workspace,
                           size_t workspace_bytes, int algo, pn_stream stream);

/*
 * pn_gemv_layer_host: pn_gemv_layer with the activations taken from and the
 * outputs returned to host memory, end to end in one call.  x_host holds every
 * entry's x fp16 [M][K] one after the other in entry order, y_host every
 * entry's y fp32 [M][N] the same way.  The call copies x_host into the
 * entries' device x buffers, runs the GEMVs (PN_ALGO_AUTO) on `stream`, copies
 * the entries' device y into y_host and waits for the stream: it returns when
 * y_host is written.  Entries whose device buffers follow each other are
 * copied in one transfer.  Page-locked (pinned) host memory keeps the copies
 * at full speed.  Every check (the descriptors as for pn_gemv_layer, null host
 * pointers, the workspace, which is required) runs before anything is
 * enqueued.
 */
pn_status pn_gemv_layer_host(const pn_gemv_desc* descs, int count, int M, const uint16_t* x_host, float* y_host,
                             void* workspace, size_t workspace_bytes, pn_stream stream);

/*
 * pn_gemv_noalloc: pn_gemv for callers that cannot allocate device memory --
 * code running where cudaMalloc is not allowed (a host callback, a stream
 * owned by another runtime), a plugin whose host framework owns every
 * allocation, or a serving loop that must not touch the allocator once the
 * model is loaded.  (The pages have no counterpart: this entry point only
 * changes where the scratch memory comes from.)  Same arguments, layouts,
 * results and alignment rules as pn_gemv; no workspace argument.
 *
 * Scratch: a fixed 512 KiB array in the library's device image, which every
 * GPU that loads the library holds until the process exits.  A device whose
 * workspace (pn_workspace_bytes) would not fit (more than 226 SMs) gets
 * PN_EINVAL and nothing is launched.  The first call on each device looks up
 * the array's device address (cudaGetSymbolAddress, which may load the
 * library's device module); make that first call before capturing a stream
 * into a CUDA graph.  The address is kept for the life of the process: after
 * cudaDeviceReset on a device, do not call pn_gemv_noalloc on that device
 * again (the array may have moved).  Arguments are checked first, exactly as
 * pn_gemv checks them; a refused call enqueues nothing.  Every call shares the
 * array and it keeps the last call's contents: each call that launches a
 * tensor-core kernel first clears, on `stream`, the parts that must start at
 * zero.  Calls whose executions overlap on the GPU (other streams, other host
 * threads) race on the array and give wrong results; order them on one
 * stream.  A device-side wait that gives up (see pn_set_wait_timeout_ns)
 * leaves the outputs undefined and, unlike pn_gemv, cannot be read back.
 * Allocates nothing: no cudaMalloc, cudaFree or allocating library call.
 */
pn_status pn_gemv_noalloc(int type, const void* W, int64_t N, int64_t K, const uint16_t* x, int M,
                          float* y, pn_stream stream);

/*
 * pn_hadamard: the runtime Hadamard rotation of the activations that reach the
 * PN weights (tensorless docs, "Why a P100-native weight format", section "How
 * Qwen3.8-27B-PN3 uses it"; the page gives no size or normalisation, read
 * here as follows).  Every run of `block` consecutive activations of each of
 * the M rows of x (fp16 [M][K]) is multiplied by the orthonormal Sylvester
 * Hadamard matrix H_block / sqrt(block) (H_1 = [1], H_2n = [[H, H], [H, -H]]),
 * written to out (fp16 [M][K]; out may equal x, otherwise the two must not
 * overlap).  block is a power of two, 2 <= block <= 4096, dividing K;
 * 1 <= M <= 65535.  Arithmetic, fixed so results are reproducible bit for
 * bit: fp16 -> fp32; butterfly stages h = 1, 2, ..., block/2 in that order,
 * each replacing (v[i], v[i+h]) for (i & h) == 0 by (v[i] + v[i+h],
 * v[i] - v[i+h]) in fp32; one fp32 multiply by 2^(-m/2) (block = 2^m, m even)
 * or 2^(-(m+1)/2) * fp32(sqrt 2) (m odd); fp16 round-to-nearest-even.  x and
 * out 2-byte aligned.  Asynchronous on `stream`; a following pn_gemv on the
 * same stream reads the rotated activations.
 */
pn_status pn_hadamard(const uint16_t* x, int M, int64_t K, int block, uint16_t* out, pn_stream stream);

/*
 * pn_gemv_hadamard / pn_gemv_layer_hadamard: pn_gemv / pn_gemv_layer on the
 * activations rotated as pn_hadamard rotates them (runs of `block`, same
 * arithmetic, so the multiplied fp16 values are exactly pn_hadamard's
 * output), in one launch: the rotation is fused into the GEMV (tensorless
 * docs, "How Qwen3.8-27B-PN3 uses it": the engine applies the rotation at
 * run time).  x is read, not modified.  Limits of the fused path: 1 <= M <= 2;
 * block a power of two from 32 to 1024 dividing every K (else PN_EINVAL);
 * the tensor-core alignment rules and rows of at most 64 chunks of 8 blocks
 * (else PN_EALIGN / PN_EUNSUPPORTED); the rotated activations of the tensors
 * one SM works on must fit its shared memory (about 70 K activations per
 * token pair; else PN_EUNSUPPORTED).  Outside these limits, call pn_hadamard
 * and then pn_gemv.  Same workspace, result and tolerance as pn_gemv.
 */
pn_status pn_gemv_hadamard(int type, const void* W, int64_t N, int64_t K, const uint16_t* x, int M, int block,
                           float* y, void* workspace, size_t workspace_bytes, pn_stream stream);
pn_status pn_gemv_layer_hadamard(const pn_gemv_desc* descs, int count, int M, int block, void* workspace,
                                 size_t workspace_bytes, pn_stream stream);

/*
 * pn_gptq: GPTQ-style quantisation of fp32 weights w [N][K] into PN rows
 * W [N][pn_row_bytes(type, K)] (tensorless docs, "How Qwen3.8-27B-PN3 uses
 * it": the weights were quantised "GPTQ-style").  The published GPTQ
 * (Frantar et al., ICLR 2023, Algorithm 1) with the PN blocks as its groups:
 * H = 2 X^T X + lambda I over calibration inputs X fp32 [n][K] (lambda = damp
 * times the mean of diag(2 X^T X), damp > 0, typically 0.01); U the upper
 * Cholesky factor of H^-1; columns in order, each row's block scale taken by
 * the signed-scale rule from the block's current weights when the block
 * starts, each column rounded with that scale and its error / U[k][k] fed to
 * the later columns through U's row k.  fp64 throughout (fp32 for the scale
 * and the rounding), each sum in index order, so the bytes equal the CPU
 * oracle's.  Synchronous (returns when W is written).  scratch: device,
 * 256-byte aligned, pn_gptq_scratch_bytes(N, K) bytes (4 K^2 + N K doubles).
 * w and X 4-byte aligned, W any alignment.  K at most 65536.  PN_EINVAL for
 * bad sizes, a small scratch, or a Hessian that is not positive definite;
 * N = 0 does nothing.
 * Not part of the GEMV's path: an offline tool, quadratic in K.
 */
size_t pn_gptq_scratch_bytes(int64_t N, int64_t K);
pn_status pn_gptq(int type, const float* w, int64_t N, int64_t K, const float* X, int64_t n, double damp,
                  void* W, void* scratch, size_t scratch_bytes, pn_stream stream);

/*
 * Prefill (large M).  The pages' engine dequantizes the weights for prefill
 * and runs a chunked GEMM, rebuilding weights transiently from the packed
 * codes without keeping them (tensorless docs, "What the fork adds";
 * v100-skinny README, "How QPN works").  Reading taken here: each rebuilt
 * weight is the exact decode d * (n - z) rounded once to fp16 (nearest, ties
 * to even; beyond the fp16 range +-inf), and the GEMM multiplies fp16 by fp16
 * exactly and accumulates in fp32 (on the tcgen05 tensor cores).
 *
 * pn_unpack_f16: PN rows W [N][row_bytes] -> fp16 w16 [N][K] as above.  W
 * 2-byte and w16 4-byte aligned; they must not overlap.
 *
 * pn_gemm_f16: y[m * ldy + r] = sum_k w16[r][k] * x[m][k] for r < N, m < M
 * (w16 fp16 [N][K], x fp16 [M][K], y fp32 rows of ldy >= N floats).  w16 and
 * x 16-byte aligned, K a positive multiple of 8, y 4-byte aligned and not
 * overlapping w16 or x; 1 <= M < 2^31, N <= 8,388,480.  The workspace is the
 * GEMV's (pn_workspace_bytes); only its status word is used, which records
 * PN_ETIMEOUT if a device-side wait gives up (read with pn_workspace_status).
 * Each output sums its K products in fp32 in K order, 16 at a time; it is
 * within (K/16 + 16) * 2^-24 * sum_k |w16 x| + 1e-6 of the exact sum.
 *
 * pn_prefill: the whole path, y[m][r] = sum_k w16[r][k] x[m][k] for the PN
 * tensor W [N][row_bytes]: the rows are rebuilt chunk by chunk into `scratch`
 * (fp16, caller-owned, 16-byte aligned; a chunk is the largest multiple of
 * 128 rows that fits, at least 128 rows = 256 K bytes) and multiplied by x;
 * y is fp32 [M][N].  Same alignment rules as pn_gemm_f16; all launches are
 * asynchronous on `stream`, in order, so scratch is reused safely.
 */
pn_status pn_unpack_f16(int type, const void* W, int64_t N, int64_t K, uint16_t* w16, pn_stream stream);
pn_status pn_gemm_f16(const uint16_t* w16, int64_t N, int64_t K, const uint16_t* x, int64_t M, float* y,
                      int64_t ldy, void* workspace, size_t workspace_bytes, pn_stream stream);
pn_status pn_prefill(int type, const void* W, int64_t N, int64_t K, const uint16_t* x, int64_t M, float* y,
                     void* scratch, size_t scratch_bytes, void* workspace, size_t workspace_bytes,
                     pn_stream stream);

/*
 * ------------------------------------------------------------ 4-bit cache --
 *
 * A serving step between two GEMVs: pages and slots for its tokens
 * (pn_kv_plan), norms and rotation of queries and keys with the write into a
 * paged cache held in 4 bits (pn_kv_append), the step's queries against that
 * cache (pn_attention), and the drafted tokens against the target's
 * probabilities (pn_verify).  (The pages' engine keeps its cache in 4 bits and
 * splits the cached tokens of a decode step over the GPU: tensorless docs,
 * "What the fork adds".  They give no layout; the one here is this library's.)
 *
 * The cache: `pages` pages of page_size tokens (a power of two, 16 .. 1024)
 * of kv_heads heads of head_dim values (64, 128 or 256), in all
 * pn_kv_cache_bytes(...) bytes (0 for a shape outside these, with more than
 * 2^31 - 1 pages or 65536 heads, or past 2^63 - 1 bytes), 16-byte aligned:
 *
 *   uint8 [pages][kv_heads][page_size / 16][17 * head_dim]
 *
 * A record holds 16 consecutive tokens of one head: K codes (8 D bytes), K
 * scales (D / 2), V codes (8 D), V scales (D / 2).  Values are pn4t's: groups
 * of 64 with a signed fp16 scale d and codes n, value d * (n - 8), chosen by
 * pn_pack's rule; eight codes to a 32-bit word as in a PN block.  With token r
 * = 8 h + g of the record (h = 0, 1), group j = 2 plane + s (D = 64: plane =
 * s = 0), word i of the group, the words lie in the order
 *   K  [h][plane][g][i / 2][s][i % 2]
 *   V  [h][plane][i][g / 2][g % 2][s]
 * (s absent for D = 64), and the scales [token][group].  Bytes that no token
 * was written to may hold anything.  A slot is page * page_size + place in the
 * page (64 bits).
 */
size_t pn_kv_cache_bytes(int64_t pages, int page_size, int kv_heads, int head_dim);

/*
 * pn_kv_plan: one step's bookkeeping on the device.  For request b < batch
 * (at most 16384; capacity at most 2^31 - 17): lens[b] tokens are cached, held[b] pages are its own (the
 * first held[b] entries of row b of table: int32 [batch][table_stride], of
 * which max_pages are used), and add[b] >= 0 tokens join it; add[b] < 0: the
 * request is finished.  Free pages are a ring free_pages[pages] with
 * ring = {head, tail}: entries head .. tail - 1, modulo pages, are free.
 *   starts[b] (b <= batch): tokens of the step before request b (2^31 - 16
 *   where there are more).
 *   Taking: request b needs max(ceil((lens + add) / page_size) - held, 0)
 *   pages, taken from the ring's head in request order.  A request whose pages
 *   pass max_pages, whose tokens end behind `capacity`, or whose need together
 *   with those of the requests before it passes the free pages is refused: it
 *   takes nothing, its length stays, its tokens get no slots.
 *   Giving: a finished request's held pages go behind the ring's tail in
 *   request order, its length and held become 0.  (A shorter lens with the same held, after
 *   drafts were turned down, keeps the pages for the tokens to come.)
 *   Token t < starts[batch] of request b: requests[t] = b, positions[t] =
 *   lens[b] + t - starts[b], slots[t] = its place in the cache; -1 in the
 *   latter two where b was refused, in all three for starts[batch] <= t <
 *   capacity.
 *   lens_out, held_out [batch], ring_out {head, tail}, refused[1] (how many):
 *   the state after the step.
 * Inputs stay as they are but for the new entries of table and free_pages, so
 * a call repeated on them gives the same; no output may overlap an input or
 * another output.  The ring's invariant (tail - head + all held pages at most
 * `pages`) is the caller's; no access leaves the arrays without it.
 */
pn_status pn_kv_plan(const int32_t* lens, const int32_t* add, const int32_t* held, int batch, int32_t* table,
                     int64_t table_stride, int max_pages, int32_t* free_pages, int64_t pages, const int64_t* ring,
                     int page_size, int64_t capacity, int64_t* slots, int32_t* positions, int32_t* requests,
                     int32_t* starts, int32_t* lens_out, int32_t* held_out, int64_t* ring_out, int32_t* refused,
                     pn_stream stream);

/*
 * pn_kv_append: for each of `tokens` tokens with `heads` query heads and
 * kv_heads key and value heads (q, k, v of `dtype`, rows of q_stride / k_stride
 * / v_stride elements, heads contiguous in a row):
 *   norm (where q_weight / k_weight, fp32 [head_dim], is given): y = x * (1 /
 *   sqrt(mean(x^2) + eps)) * weight per head;
 *   rotation (rotary > 0, even): with row positions[t] of cos and sin (fp32
 *   [table_rows][rotary / 2]; a position outside the table leaves the row as
 *   it is), the first `rotary` values as pairs (a, b) = (y[i], y[i + rotary/2])
 *   or, interleaved, (y[2i], y[2i+1]) become (a c - b s, b c + a s);
 *   q_out[t][heads][head_dim]: the queries rounded to fp16;
 *   keys, and values as they are, by pn_pack's rule into slot slots[t]; a
 *   token whose slot is negative or outside the cache writes no cache.
 * The arithmetic is fp32 with every operation rounded by itself, in a fixed
 * order, so the cache's bytes are reproducible bit for bit: squares are added
 * pairwise, the upper half of the row to the lower until one is left, times
 * 1 / head_dim; fp32 quotients and square roots are IEEE.  Inputs must be
 * finite (else that head's codes are unspecified).  q_out and cache 16-byte
 * aligned, other arrays to their element.  No two tokens of a call may share
 * a slot.  heads = 0: keys and values alone.  q_out and cache share no memory
 * with each other or an input (PN_EINVAL).
 */
typedef enum { PN_DTYPE_F32 = 0, PN_DTYPE_F16 = 1 } pn_dtype;
pn_status pn_kv_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                       int64_t v_stride, int dtype, int64_t tokens, int heads, const float* q_weight,
                       const float* k_weight, float eps, const float* cos, const float* sin, int64_t table_rows,
                       int rotary, int interleaved, const int32_t* positions, const int64_t* slots, void* cache,
                       int64_t pages, int page_size, int kv_heads, int head_dim, uint16_t* q_out, pn_stream stream);

/* pn_kv_read: the cached keys and values of `tokens` slots as fp32
 * [tokens][kv_heads][head_dim], exact; zeros for a slot outside the cache.
 * k and v 16-byte aligned, sharing no memory with each other or an input. */
pn_status pn_kv_read(const void* cache, int64_t pages, int page_size, int kv_heads, int head_dim,
                     const int64_t* slots, int64_t tokens, float* k, float* v, pn_stream stream);

/*
 * pn_attention: for request b < batch (at most 16384) the query tokens
 * starts[b] .. starts[b + 1] - 1 of q (fp16, rows of q_stride elements, heads
 * contiguous; at most max_queries of them), the last of which sits at cached
 * token lens[b] - 1; `heads` is a multiple of kv_heads, and query head h reads
 * key/value head h / (heads / kv_heads).  A query at position p sees the
 * cached tokens t <= p with, where window > 0, t > p - window or t < sinks (any
 * number from 0 on; a length past max_pages * page_size counts as that).
 *   x_t = scale * q . k_t;  lse = ln sum_t exp(x_t);
 *   out = sum_t exp(x_t - lse) v_t
 * A query that sees nothing gets out = 0 and lse = -inf.  Hidden tokens have
 * no influence whatever their bytes hold, and neither have pages that the
 * table gives outside the cache: their tokens are hidden.  Rows of out that
 * belong to no request are not written.
 * out fp16 [tokens][heads][head_dim], lse fp32 [tokens][heads] or NULL.
 * Scores, sums and outputs are held in fp32; exp(x_t) times the scale of v_t
 * is rounded to fp16 before it is multiplied by v_t's codes, so an output is
 * within 2^-11 (sum_t p_t |v_t|) + 2^-11 |out| of the exact value, and a
 * little more for the fp32 sums and, where V's scales differ by powers of ten,
 * for products far below the largest (2^-32 max |v| to a token where many rows
 * share a head, 2^-35 where few do).  Deterministic: a call repeated on a GPU of
 * the same kind gives the same bits.  Which kernel runs goes by batch,
 * max_queries, the heads and head_dim alone; the last bits also go by where the
 * work is cut and joined again, that is by every request's length and queries,
 * the window, the first tokens and the number of SMs.  So a request's last bits
 * can differ with the requests beside it.
 * The work is numbered in 32 bits.  With group = heads / kv_heads and rows taken
 * 16 at a time (8 where max_queries * group <= 8 or head_dim is 256), PN_EUNSUPPORTED
 * if batch * kv_heads * ceil(max_queries * group / 16) reaches 2^31, or if kv_heads *
 * min(that many row groups, tokens * group / 16 + batch) * (max_pages * page_size /
 * 32 + 1) reaches 2^32 (where the kernel for many rows runs: by whole query tokens
 * that fit 128 rows, 64 cached tokens at a time, 32 for head_dim 256).  The second
 * limit takes starts to be in order; where they are not and the work passes it,
 * nothing is written and the status word says PN_EINVAL.
 * workspace: pn_attention_workspace_bytes() bytes, 256-byte aligned, zeroed
 * once (pn_workspace_init); every completed call leaves its counters zeroed.
 * pn_workspace_status reads its status word.  Calls that share a workspace
 * must be ordered on one stream.  q, cache and out 16-byte aligned, q_stride a
 * multiple of 8; out, lse and workspace share no memory with each other or an
 * input.
 */
size_t pn_attention_workspace_bytes(void);
pn_status pn_attention(const uint16_t* q, int64_t q_stride, int64_t tokens, int heads, const void* cache,
                       int64_t pages, int page_size, int kv_heads, int head_dim, const int32_t* table,
                       int64_t table_stride, int max_pages, const int32_t* lens, const int32_t* starts, int batch,
                       int max_queries, float scale, int window, int sinks, uint16_t* out, float* lse,
                       void* workspace, size_t workspace_bytes, pn_stream stream);

/*
 * pn_verify: speculative verification.  For request b < batch with counts[b]
 * (NULL: drafts) of at most `drafts` (0 .. PN_MAX_DRAFTS) drafted tokens
 * tokens[b][i], target probabilities target[b][i] (fp32 rows of vocab values,
 * row b * (drafts + 1) + i at target_stride elements), the draft model's
 * draft[b][i] (row b * drafts + i; NULL: each draft was certain, q = 1 at its
 * token) and random numbers uniforms[b][drafts + 1] in [0, 1):
 *   draft i is accepted while uniforms[b][i] * q_i(token) < p_i(token)
 *   (fp32; a token outside the vocabulary is turned down);
 *   accepted[b] is the number n of them;
 *   out[b][0 .. n - 1] the accepted tokens, out[b][n] one more, -1 behind it.
 * The last token is the lowest index whose cumulated weight passes
 * floor(uniforms[b][drafts] * total), the weights being those of row n: p
 * after the last draft, max(p - q, 0) where draft n was turned down (p itself
 * should that leave nothing), each limited to [0, 1] (NaN: 0) and rounded to a
 * whole multiple of 2^-42, so that the token does not depend on the order of
 * the sums.  -1 if the whole row weighs nothing.  accepted and out share no
 * memory with each other or an input (counts among them).
 */
#define PN_MAX_DRAFTS 31
#define PN_MAX_VOCAB (1 << 20)
pn_status pn_verify(const int32_t* tokens, const float* target, int64_t target_stride, const float* draft,
                    int64_t draft_stride, const float* uniforms, const int32_t* counts, int batch, int drafts,
                    int vocab, int32_t* accepted, int32_t* out, pn_stream stream);

/*
 * pn_read_ranges (diagnostic): the plain read-bandwidth ceiling a GEMV is
 * measured against.  Reads the first floor(bytes[i] / 16) * 16 bytes of each
 * of `count` (1 .. PN_MAX_LAYER) device ranges ptrs[i] once, with 16-byte
 * loads, and XORs the 32-bit words read into sink[i] (device, `count` words;
 * zero them first if the value matters).  ptrs and bytes are host arrays
 * read during the call; every ptrs[i] 16-byte aligned, sink 4-byte aligned.
 */
pn_status pn_read_ranges(const void* const* ptrs, const size_t* bytes, int count, uint32_t* sink,
                         pn_stream stream);

/*
 * Testing aid: the time limit, in nanoseconds, of every device-side wait in
 * the tensor-core GEMV kernels and the prefill GEMM (default 1e9).  A wait that runs out stops its thread
 * block, which records PN_ETIMEOUT in the workspace status word and returns
 * after its outstanding copies land.  Process-wide; not for concurrent use.
 */
void pn_set_wait_timeout_ns(uint64_t ns);

/*
 * Testing aid for the failure path: while on (non-zero), every thread block of
 * the tensor-core GEMV kernels and of the prefill GEMM announces the bytes of
 * its first step but never copies them, so its consumers' wait can only end
 * by timing out; the call then reports PN_ETIMEOUT through
 * pn_workspace_status and its outputs are undefined.  Off by default.
 * Process-wide; not for concurrent use.
 */
void pn_set_test_stall(int on);

/*
 * Testing aid (host only; needs no device): the work split the tensor-core
 * GEMV kernel for 3 <= M <= 16 would use for a pn_gemv_layer call on
 * tensors of these types and shapes on a GPU with num_sms SMs.  types, N
 * and K are host arrays of `count` (1 .. PN_MAX_LAYER) entries; every N >= 1
 * and every K a positive multiple of 8 blocks (640 for pn3t, 512 for pn4t),
 * else PN_EINVAL.  Units are numbered over the tensors in order, each
 * tensor's 16-row tiles in turn and each tile's 8-block chunks within it.
 * On PN_OK, *grid is the number of thread blocks and block c takes units
 * [starts[c], starts[c + 1]) (starts: host array of at least num_sms + 1
 * entries; starts[0] = 0, starts[*grid] = all units).  Every range holds at
 * least one whole tile's units, so a tile has at most two owners; the split
 * depends only on the arguments.
 */
pn_status pn_tc_split(const int* types, const int64_t* N, const int64_t* K, int count, int M, int num_sms,
                      uint32_t* starts, int* grid);

#ifdef __cplusplus
}
#endif

#endif /* PN_H */
