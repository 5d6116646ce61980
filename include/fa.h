/*
 * fa.h -- C ABI of libfa: fused FlashAttention forward (plain, causal,
 * grouped-query, split-KV), its backward, and split-KV decode (per-head and
 * grouped-query) for one NVIDIA GB300 GPU (sm_103a); rotary positions, with
 * norms of the heads in the same pass or without, a paged key/value cache, its
 * bookkeeping, the decode that reads it, with or without a prefix that all
 * sequences share, and the attention of chunks of new tokens over it.
 *
 * Sources (web pages, cited by title and section):
 *   [T1] "FlashAttention 简化版：Tiling + Online Softmax" (forceinjection.github.io)
 *   [T2] "Flash Attention 代码填空 (Level 2-3)" (boots-coder.github.io, LLM-101-CN)
 *   [T3] "CS349E 第 11 讲 01_online_softmax.py" (semidirectx.com)
 *   [T4] "从零手写 FlashAttention（PyTorch实现 + 原理推导）" (mokono.cn)
 *
 * Conventions shared by every entry point
 *   - Tensors are contiguous row-major [B, H, N, d] (d fastest).  Decode q and
 *     o are [B, H, d] (one query per head).  LSE is fp32 [B, H, Nq].
 *   - Every tensor pointer is a DEVICE pointer owned by the caller (except the
 *     tensors of fa_fwd_host, which are host pointers); device base addresses
 *     must be 16-byte aligned.  The library never frees caller memory and
 *     keeps no pointer after a call returns.
 *   - Calls are asynchronous: they validate, enqueue kernels on `stream`
 *     (NULL = the legacy default stream) and return.  A return of FA_OK means
 *     the work was enqueued; timeouts detected on the device are reported
 *     later by fa_check_device_error().
 *   - Arguments are validated before anything is launched; on any error
 *     nothing is enqueued.  No call prints or exits.
 *   - Calls are reentrant and may be made from several host threads.
 */
#ifndef FA_H_
#define FA_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t, declared here so this header needs no CUDA header. */
struct CUstream_st;
typedef struct CUstream_st* fa_stream_t;

typedef enum { FA_FP32 = 0, FA_BF16 = 1 } fa_dtype;

typedef enum {
    FA_OK = 0,
    FA_ERR_INVALID_ARG = 1, /* NULL or misaligned pointer, non-positive size, overflow, bad scale */
    FA_ERR_UNSUPPORTED = 2, /* valid but unsupported: head dim not 64/128, dtype, device not sm_103 */
    FA_ERR_CUDA = 3,        /* a CUDA runtime/driver call failed (launch, allocation, tensor map) */
    FA_ERR_TIMEOUT = 4      /* a device-side wait ran past its limit (from fa_check_device_error) */
} fa_status;

/*
 * fa_fwd -- exact attention O = softmax(Q K^T * scale) V, computed tile by
 * tile with the online-softmax recurrence so the Nq x Nk score matrix never
 * reaches device memory ([T1] §2.3, §3.1; [T3] attn_row_1pass).  For each
 * query row the running maximum m, running sum l and unnormalised O are
 * updated per key tile with correction alpha = exp(m_old - m_new); O is
 * divided by l once at the end ([T3] demo 3, deferred normalisation).
 *
 *   q   [B, H, Nq, d]  in dtype       k, v [B, H, Nk, d] in dtype
 *   o   [B, H, Nq, d]  out, dtype     lse  [B, H, Nq] fp32 out, or NULL
 *   lse = m + ln(l) in natural log, in units of scaled scores ([T3] demo 2).
 *   dtype FA_BF16: bf16 operands, fp32 accumulation, P rounded to bf16 for P V.
 *   dtype FA_FP32: fp32 operands multiplied as TF32, P kept at TF32.  A prep
 *     pass first writes tf32-rounded (nearest) copies of Q and K and a
 *     key-major tf32 copy of V (tf32 tensor-core operands must be K-major).
 *   When the query tiles cannot fill the GPU (small B*H*Nq) the keys are also
 *   split across CTAs and merged (see fa_fwd_ex).  Any workspace these need
 *   (fa_fwd_workspace_bytes) is taken stream-ordered (cudaMallocAsync /
 *   cudaFreeAsync on `stream`).
 *   d must be 64 or 128; Nq, Nk >= 1 (ragged tails are masked); B, H >= 1;
 *   scale must be finite (1/sqrt(d) is the usual value; 1 reproduces [T4]-style
 *   unscaled scores).  Returns FA_OK or an fa_status code.
 */
int fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
           int B, int H, int Nq, int Nk, int d, float scale, int dtype,
           fa_stream_t stream);

/*
 * fa_fwd_ex -- fa_fwd with every option exposed.  fa_fwd(...) is
 * fa_fwd_ex(..., Hkv = H, causal = 0, kv_splits = 0, workspace = NULL, 0, stream).
 *   Hkv        key/value heads per batch (grouped-query attention): k and v are
 *              [B, Hkv, Nk, d]; query head h reads key/value head h / (H / Hkv).
 *              H must be a multiple of Hkv (Hkv = H: plain multi-head).
 *   causal     1 = causal mask aligned to the bottom-right corner: query row i
 *              sees keys 0 .. i + (Nk - Nq), so the last query sees every key
 *              and Nq == Nk gives the usual lower triangle ([T1] §7 names the
 *              extension).  Requires Nq <= Nk (FA_ERR_INVALID_ARG otherwise).
 *              Key tiles above the diagonal are skipped, not just masked.
 *   kv_splits  0 = automatic; 1 = one pass over all keys per query tile;
 *              n > 1 = the keys are cut into n ranges handled by separate CTAs,
 *              each writing an fp32 partial state (m, l, unnormalised O) that a
 *              merge kernel combines ([T3] demo 2, split-KV / flash-decoding
 *              applied to every query row).  Automatic splitting is used only
 *              when the query tiles alone cannot fill the GPU.  n may not exceed
 *              the number of key tiles (FA_ERR_INVALID_ARG).
 *              Automatic mode also shortens a short last wave (bf16, d = 64, no
 *              mask): when the CTAs of 256 query rows do not fill whole waves of
 *              two per SM and the rest is at most one per SM, the rows of that
 *              rest go to CTAs of 128 rows whose two halves of the keys run side
 *              by side and merge inside the CTA ([T3] demo 2).  No workspace; the
 *              result depends only on the shape and the GPU's SM count.
 *              kv_splits = 1 keeps every CTA on the whole key range.
 *   workspace  device buffer of at least fa_fwd_workspace_bytes(...) bytes,
 *              16-byte aligned, or NULL to allocate it stream-ordered.  Needed
 *              by the fp32 path (rounded / transposed operand copies) and by
 *              split runs; a bf16 call with one split needs none.
 */
int fa_fwd_ex(const void* q, const void* k, const void* v, void* o, float* lse,
              int B, int H, int Hkv, int Nq, int Nk, int d, float scale, int dtype,
              int causal, int kv_splits, void* workspace, size_t workspace_bytes,
              fa_stream_t stream);

/* Bytes of workspace fa_fwd_ex needs for these arguments (kv_splits = 0 asks the
 * current device's SM count); 0 when none is needed or the arguments are invalid. */
size_t fa_fwd_workspace_bytes(int B, int H, int Hkv, int Nq, int Nk, int d, int dtype,
                              int causal, int kv_splits);

/*
 * fa_fwd_host -- fa_fwd_ex (kv_splits = 0) on HOST-resident tensors: the library
 * copies q, k, v to the device, computes, and copies o and lse back, in chunks
 * of whole key/value heads (about one wave of CTAs each) so that the
 * copies of one chunk overlap the compute of the previous one (copy-in and
 * copy-out on two internal streams, compute on `stream`, ordered by events).  The
 * exact attention computed is fa_fwd_ex's.
 *   q, k, v, o, lse   HOST pointers, same shapes and dtypes as fa_fwd_ex; lse may
 *                     be NULL.  Page-locked (pinned) memory is needed for the
 *                     copies to overlap; pageable memory works but serialises.
 *   workspace         device buffer of at least fa_fwd_host_workspace_bytes(...)
 *                     bytes (16-byte aligned) that receives the device copies, or
 *                     NULL to allocate it stream-ordered on `stream`.
 * Asynchronous: o and lse hold the result once `stream` has completed the work
 * enqueued up to this call (the call makes `stream` wait for the last copy out).
 * Calls on one device are serialised on the host while they enqueue.  Returns
 * FA_OK or an fa_status code.
 */
int fa_fwd_host(const void* q, const void* k, const void* v, void* o, float* lse,
                int B, int H, int Hkv, int Nq, int Nk, int d, float scale, int dtype,
                int causal, void* workspace, size_t workspace_bytes, fa_stream_t stream);

/* Bytes of device workspace fa_fwd_host needs (0 for invalid arguments). */
size_t fa_fwd_host_workspace_bytes(int B, int H, int Hkv, int Nq, int Nk, int d, int dtype,
                                   int causal);

/*
 * fa_bwd -- gradients of exact attention (bf16 or fp32 tensors).
 * Given the forward's inputs, its output O and natural-log LSE, and dO (the
 * gradient of a loss with respect to O), writes
 *   dV = P^T dO, dQ = scale dS K, dK = scale dS^T Q, with P = exp(scale Q K^T - LSE)
 *   recomputed block by block from the saved LSE ("Flash Attention 代码填空
 *   (Level 2-3)", Exercise 5: the forward keeps O and the row statistics, the
 *   backward rebuilds P_ij and accumulates dV_j += P_ij^T dO_i), dP = dO V^T and
 *   dS = P * (dP - D), D_i = sum_c dO_ic O_ic (chain rule through the softmax).
 *   q, o, dout, dq  [B, H, Nq, d] in dtype   k, v, dk, dv [B, Hkv, Nk, d] in dtype
 *   lse             [B, H, Nq] fp32 in: as written by fa_fwd / fa_fwd_ex
 *   Hkv, causal     as in fa_fwd_ex; with Hkv < H, dk and dv sum over the query
 *                   heads that share a key/value head.
 *   dtype           FA_BF16: bf16 operands on the tensor cores, fp32 accumulation,
 *                   P and dS rounded to bf16 for their products.
 *                   FA_FP32: every product and sum in fp32 on the CUDA cores (the
 *                   tensor cores would round the operands to tf32).  d 64 or 128.
 *   workspace       device buffer of at least fa_bwd_workspace_bytes(B, H, Nq, d)
 *                   bytes (16-byte aligned) for D and the rescaled LSE, or NULL
 *                   to allocate it stream-ordered on `stream`.
 * No atomics: every gradient element is written once, by one CTA, so repeated
 * calls give bit-identical results.  Inputs are read only; outputs are fully
 * overwritten.  Returns FA_OK or an fa_status code; argument errors are
 * reported before anything is launched.
 */
int fa_bwd(const void* q, const void* k, const void* v, const void* o, const void* dout,
           const float* lse, void* dq, void* dk, void* dv, int B, int H, int Hkv,
           int Nq, int Nk, int d, float scale, int dtype, int causal,
           void* workspace, size_t workspace_bytes, fa_stream_t stream);

/* Bytes of workspace fa_bwd needs (0 for invalid arguments). */
size_t fa_bwd_workspace_bytes(int B, int H, int Nq, int d);

/*
 * fa_decode_splitkv -- attention of one bf16 query per head over Nk keys,
 * split into `splits` chunks of ceil(Nk/splits) keys processed in parallel
 * (flash-decoding); each chunk yields a partial state (m, l, o) with o
 * unnormalised, and a second kernel merges the states ([T3] demo 2: the merge
 * is associative and commutative) and writes O = o / l as bf16.
 *
 *   q [B, H, d] bf16, k/v [B, H, Nk, d] bf16, o [B, H, d] bf16 out.
 *   scale is fixed at 1/sqrt(d).  1 <= splits <= Nk; d in {64, 128}.
 *   The fp32 workspace for the partial states is taken stream-ordered
 *   (cudaMallocAsync / cudaFreeAsync on `stream`).
 */
int fa_decode_splitkv(const void* q, const void* k, const void* v, void* o,
                      int B, int H, int Nk, int d, int splits,
                      fa_stream_t stream);

/*
 * fa_decode_splitkv_ex -- fa_decode_splitkv with every option exposed.
 *   scale        finite score scale.
 *   workspace    device buffer of at least fa_decode_workspace_bytes(B, H, d,
 *                splits) bytes, 16-byte aligned; NULL = allocate stream-ordered.
 *   merge_order  device int32 [splits], a permutation of 0..splits-1 giving the
 *                order in which chunk states are accumulated by the merge; NULL
 *                = index order.  The result is the same up to rounding for
 *                every order ([T3] demo 2).  Entries are validated on the
 *                device; a non-permutation makes the merge write NaN outputs.
 *   lse          fp32 [B, H] out (natural log, scaled-score units), or NULL.
 */
int fa_decode_splitkv_ex(const void* q, const void* k, const void* v, void* o,
                         int B, int H, int Nk, int d, int splits, float scale,
                         void* workspace, size_t workspace_bytes,
                         const int* merge_order, float* lse, fa_stream_t stream);

/* Bytes of fp32 partial-state workspace fa_decode_splitkv_ex (and _gqa) needs; 0 on bad arguments. */
size_t fa_decode_workspace_bytes(int B, int H, int d, int splits);

/*
 * fa_decode_splitkv_gqa -- split-KV decode where Hkv key/value heads serve H
 * query heads ("FlashAttention 简化版：Tiling + Online Softmax" §7 names
 * MQA/GQA): query head h reads key/value head h / (H / Hkv).  Each chunk of
 * each key/value head is read from device memory once for all the query heads
 * of its group; the chunk states and their merge are those of
 * fa_decode_splitkv_ex ([T3] demo 2), one state per (query head, chunk).
 *   q [B, H, d] bf16, k/v [B, Hkv, Nk, d] bf16, o [B, H, d] bf16 out.
 *   H / Hkv must be 1, 2, 4 or a multiple of 8 (FA_ERR_UNSUPPORTED otherwise);
 *   H % Hkv != 0 is FA_ERR_INVALID_ARG.  Other arguments as in
 *   fa_decode_splitkv_ex; the workspace size is fa_decode_workspace_bytes(B, H,
 *   d, splits).
 */
int fa_decode_splitkv_gqa(const void* q, const void* k, const void* v, void* o,
                          int B, int H, int Hkv, int Nk, int d, int splits, float scale,
                          void* workspace, size_t workspace_bytes,
                          const int* merge_order, float* lse, fa_stream_t stream);

/* Size of the fixed device scratch array behind fa_decode_splitkv_noalloc. */
#define FA_DECODE_NOALLOC_SCRATCH_BYTES ((size_t)8 << 20)

/*
 * fa_decode_splitkv_noalloc -- fa_decode_splitkv for callers that cannot
 * allocate device memory during a call (for example serving processes that
 * reserve nearly all device memory up front and forbid later allocations, or
 * whose memory manager must own every allocation; cudaMalloc may also block
 * on the device).  The pages have no counterpart: this is a deployment
 * variant of the same split and merge kernels.
 *
 *   Arguments, layouts and results are those of fa_decode_splitkv (bf16,
 *   scale 1/sqrt(d)).  The partial states live in a fixed array of
 *   FA_DECODE_NOALLOC_SCRATCH_BYTES inside the library's device image, which
 *   every GPU that loads the library holds until the process exits.  The call
 *   allocates and frees nothing.
 *   - FA_ERR_UNSUPPORTED if fa_decode_workspace_bytes(B, H, d, splits) exceeds
 *     FA_DECODE_NOALLOC_SCRATCH_BYTES, or if the current device is not an
 *     sm_103 GPU (nothing is launched in either case).
 *   - All calls share the array: calls whose kernels may overlap on the GPU
 *     (unordered streams) race and must be ordered by the caller.  The array
 *     keeps the previous call's contents; nothing needs clearing, since every
 *     partial state is written before it is read.
 *   - The first call on each device looks up the array's address
 *     (cudaGetSymbolAddress, with that device current); make it before any
 *     stream capture.
 */
int fa_decode_splitkv_noalloc(const void* q, const void* k, const void* v, void* o,
                              int B, int H, int Nk, int d, int splits,
                              fa_stream_t stream);

/*
 * fa_rope -- rotary positions on q and k (or, with inverse = 1, the backward
 * pass: the same rotation by the negative angle on the gradients of fa_rope's
 * outputs, as fa_bwd writes them for its q and k).
 *
 * The first `rot` elements of a head form rot/2 pairs: elements (i, i + rot/2),
 * or (2i, 2i + 1) with interleaved = 1.  Pair i turns by the angle
 * phi = positions[axis(i)][b][n] * freqs[i]:
 *   (x1, x2) -> (x1 cos phi - x2 sin phi, x1 sin phi + x2 cos phi)
 * and the elements from `rot` on are copied.  One axis gives text positions;
 * three (time, height, width) those of images and video.  Angles are formed in
 * 64-bit integers, not in fp32: position times frequency is exact modulo a turn,
 * and off by what double precision leaves of the frequency, at most
 * |pos| (|f| 2^-52 + (f < 0) 2^-51) radians (2.2e-10 at position 10^6, f = 1);
 * sine and cosine are within 1.9e-7 of that angle's.  Products and sums are fp32,
 * rounded once to dtype.
 *   q [B, H, N, d], k [B, Hkv, N, d] in dtype (FA_BF16 or FA_FP32), d 64 or 128;
 *     k = k_out = NULL with Hkv = 0 rotates q alone.
 *   q_out, k_out  out: the inputs themselves (same pointer, same strides) or
 *     memory that overlaps no input.
 *   strides       NULL = all contiguous, or a HOST array of 12: the (batch,
 *     head, token) strides in elements of q, k, q_out and k_out, so that heads can
 *     be read out of a projection's [B, N, heads, d] output.  d is contiguous;
 *     every stride is >= 0 and a multiple of 16 bytes.  Rows of an output must
 *     not overlap one another.
 *   positions     device int32 [n_axes, B, N], or [n_axes, N] with pos_shared = 1
 *     (the same for every batch entry); any value, negative ones too.
 *   freqs         device float64 [rot/2], radians per position, finite.
 *   axes          device int32 [rot/2]: axis(i) in 0 .. n_axes - 1, or NULL: axis 0.
 *     A pair whose entry is out of range becomes NaN, and
 *     fa_check_device_error reports FA_ERR_INVALID_ARG.
 *   n_axes 1 .. 8; rot a multiple of 16, 16 <= rot <= d; (H + Hkv) * d < 2^31; B * N < 2^31 - 1024.
 * No workspace.  Returns FA_OK or an fa_status code.
 */
int fa_rope(const void* q, const void* k, void* q_out, void* k_out, const long long* strides,
            int B, int H, int Hkv, int N, int d, int dtype, const int* positions, int pos_shared,
            const double* freqs, const int* axes, int n_axes, int rot, int interleaved, int inverse,
            fa_stream_t stream);

/*
 * fa_norm_rope -- fa_rope on heads that are normed first, in the same pass: for a head x of d elements with
 * the weights w (q_weight for every query head, k_weight for every key head),
 *   y = R(w x / sqrt(mean(x^2) + eps)),  R fa_rope's rotation,
 * in fp32, rounded once to dtype.
 *   q_weight, k_weight  device [d] in weight_dtype (FA_BF16 or FA_FP32, whatever dtype is); k_weight
 *                       NULL with Hkv = 0.  eps finite, >= 0.
 *   positions, freqs    NULL with rot = 0: norms alone.
 * Other arguments and rules as in fa_rope.
 */
int fa_norm_rope(const void* q, const void* k, void* q_out, void* k_out, const long long* strides,
                 int B, int H, int Hkv, int N, int d, int dtype, const void* q_weight, const void* k_weight,
                 int weight_dtype, float eps, const int* positions, int pos_shared, const double* freqs,
                 const int* axes, int n_axes, int rot, int interleaved, fa_stream_t stream);

/*
 * fa_norm_rope_bwd -- the backward pass of fa_norm_rope: from the gradients dq, dk of its outputs and its
 * inputs q, k the gradients of those inputs and of the weights,
 *   g = R^-1 dy, u = x / sqrt(mean(x^2) + eps):  dx = (w g - u mean(w g u)) / sqrt(mean(x^2) + eps),
 *   dw = sum of g u over all tokens and heads.
 *   dq_in, dk_in          out, in dtype: dq, dk or q, k themselves (same pointer, same strides) or memory that
 *                         overlaps no input
 *   dq_weight, dk_weight  out, device fp32 [d] (dk_weight NULL with Hkv = 0)
 *   strides               NULL = all contiguous, or a HOST array of 18: the (batch, head, token) strides of
 *                         dq, dk, dq_in, dk_in, q and k
 *   workspace             device buffer of at least fa_norm_rope_bwd_workspace_bytes(d) bytes, 16-byte aligned,
 *                         or NULL to allocate it stream-ordered on `stream`; calls that may overlap on the GPU
 *                         must not share one
 * Sums are fp32 in a fixed order, without atomics: repeated calls on one GPU give identical bits.  Other
 * arguments as in fa_norm_rope.
 */
int fa_norm_rope_bwd(const void* dq, const void* dk, const void* q, const void* k, void* dq_in, void* dk_in,
                     float* dq_weight, float* dk_weight, const long long* strides, int B, int H, int Hkv,
                     int N, int d, int dtype, const void* q_weight, const void* k_weight, int weight_dtype,
                     float eps, const int* positions, int pos_shared, const double* freqs, const int* axes,
                     int n_axes, int rot, int interleaved, void* workspace, size_t workspace_bytes,
                     fa_stream_t stream);

/* Bytes of workspace fa_norm_rope_bwd needs on the current device; 0 on bad arguments or without an sm_103 GPU. */
size_t fa_norm_rope_bwd_workspace_bytes(int d);

/*
 * fa_paged_append -- writes the keys and values of T new tokens into a paged
 * cache, rotating the keys (and the tokens' queries) on the way.
 *
 * The cache is a pool of num_pages pages of page_size rows: k_cache and v_cache
 * [num_pages, Hkv, page_size, d] bf16, or any layout with d contiguous given by
 * cache_strides (a HOST array: the page, head and row strides in elements, used
 * for both caches; NULL = contiguous).  Token t goes to slots[t]:
 * page slots[t] / page_size, row slots[t] % page_size.
 *   k, v     [T, Hkv, d] bf16      q [T, H, d] bf16, or NULL with H = 0
 *   q_out    [T, H, d] bf16 contiguous, out (may be q itself if that is contiguous)
 *   in_strides  NULL = contiguous, or a HOST array of 6: (token, head) strides in
 *            elements of k, v and q (slices of one projection's output).
 *   slots    device int64 [T].  A negative slot stores nothing: a batch padded to a
 *            fixed size marks its unused places so.  A slot past the cache stores
 *            nothing and makes fa_check_device_error report FA_ERR_INVALID_ARG.
 *            Two tokens must not name one slot in a call (that slot would hold
 *            parts of either); no other slot is touched.
 *   positions, freqs, axes, n_axes, rot, interleaved  as in fa_rope, with positions
 *            int32 [n_axes, T]; rot = 0 with positions = freqs = NULL stores the keys
 *            and copies the queries as they are.  q_out is written for every token,
 *            those with a negative slot too.
 * All strides are multiples of 8 elements; (H + 2 * Hkv) * d < 2^31.  T = 0 is a step without new tokens.
 * Returns FA_OK or an fa_status code.
 */
int fa_paged_append(const void* k, const void* v, const void* q, void* q_out, void* k_cache, void* v_cache,
                    const long long* in_strides, const long long* cache_strides, const long long* slots,
                    int T, int H, int Hkv, int d, int num_pages, int page_size,
                    const int* positions, const double* freqs, const int* axes, int n_axes, int rot,
                    int interleaved, fa_stream_t stream);

/*
 * fa_decode_paged -- attention of one bf16 query per head over a paged cache:
 * sequence b sees its seq_lens[b] rows, row i being row i % page_size of page
 * page_table[b][i / page_size].  Lengths stay on the device; long tables' work is
 * spread evenly over the GPU whatever they are, and short tables' sequences each
 * have CTAs of their own (the results may differ in the last bit).
 *
 *   q, o       [B, H, d] bf16 (o is written); query head h reads key/value head
 *              h / (H / Hkv), any group size H / Hkv.
 *   k_cache, v_cache, cache_strides, num_pages, page_size   as in fa_paged_append.
 *   page_table device int32 [B, max_pages], rows table_stride entries apart; entries
 *              past a sequence's last page are not read.
 *   seq_lens   device int32 [B].  A sequence without keys (seq_lens[b] <= 0) gets
 *              o = 0 and lse = -inf.
 *   scale      finite score scale (finite in log2 units too: |scale| < 2.3e38).
 *   lse        fp32 [B, H] out (natural log, scaled-score units), or NULL.
 *   workspace  device buffer of at least fa_decode_paged_workspace_bytes(B, H, Hkv,
 *              d, page_size, 0) bytes, 16-byte aligned, or NULL to allocate it stream-ordered on
 *              `stream`.  It needs no clearing; calls that may overlap on the GPU must
 *              not share one.
 * A sequence with a page outside the cache or more keys than max_pages * page_size
 * gets NaN in o and lse, and fa_check_device_error reports FA_ERR_INVALID_ARG; the
 * others are not affected.  Accumulation and softmax statistics are fp32; P goes into
 * P V as two bf16 terms, together within 2^-15 of it.  No atomics: repeated calls on one GPU give identical
 * bits.  max_pages * page_size < 2^30, B * H * d < 2^31, and B * H *
 * (max_pages * page_size / 64 + 3) <= 2^39 (FA_ERR_INVALID_ARG otherwise).  Returns
 * FA_OK or an fa_status code.
 */
int fa_decode_paged(const void* q, const void* k_cache, const void* v_cache, void* o, const int* page_table,
                    long long table_stride, const int* seq_lens, int B, int H, int Hkv, int d,
                    int num_pages, int page_size, int max_pages, const long long* cache_strides, float scale,
                    void* workspace, size_t workspace_bytes, float* lse, fa_stream_t stream);

/*
 * fa_decode_paged_prefix -- fa_decode_paged for a batch whose sequences all begin
 * with the same prefix_len keys, which are read and multiplied once for the whole
 * batch.  Sequence b sees the prefix, then its own seq_lens[b] rows:
 * page_table and seq_lens describe the own rows alone.
 *   prefix_pages  device int32 [ceil(prefix_len / page_size)]: the pages of the
 *                 prefix, whose last one may be partly used.
 *   prefix_len    >= 0; 0 is fa_decode_paged (prefix_pages may then be NULL).
 *   seq_lens      0 = a sequence that sees the prefix alone; negative = an unused place
 *                 of a padded batch, which sees nothing (o = 0, lse = -inf).
 *   workspace     fa_decode_paged_workspace_bytes(B, H, Hkv, d, page_size, prefix_len)
 *                 bytes.
 * A prefix page outside the cache gives NaN in every sequence that sees the prefix.
 * Other arguments and rules as in fa_decode_paged.
 */
int fa_decode_paged_prefix(const void* q, const void* k_cache, const void* v_cache, void* o,
                           const int* prefix_pages, int prefix_len, const int* page_table,
                           long long table_stride, const int* seq_lens, int B, int H, int Hkv, int d,
                           int num_pages, int page_size, int max_pages, const long long* cache_strides,
                           float scale, void* workspace, size_t workspace_bytes, float* lse,
                           fa_stream_t stream);

/* Bytes of workspace fa_decode_paged (prefix_len = 0) and fa_decode_paged_prefix need on the current
 * device; 0 on bad arguments or without an sm_103 GPU. */
size_t fa_decode_paged_workspace_bytes(int B, int H, int Hkv, int d, int page_size, int prefix_len);

/* Bytes of workspace that a call with tables of max_pages pages uses: those, or 0 where it uses none (no prefix and
 * tables of a few thousand keys at most), so that its workspace can be NULL without an allocation. */
size_t fa_decode_paged_call_bytes(int B, int H, int Hkv, int d, int page_size, int max_pages, int prefix_len);

/*
 * fa_paged_append_norm -- fa_paged_append with the norms of fa_norm_rope: keys (and queries) are normed, rotated
 * and rounded once on their way; values are copied.  q_weight is NULL with H = 0.
 */
int fa_paged_append_norm(const void* k, const void* v, const void* q, void* q_out, void* k_cache, void* v_cache,
                         const long long* in_strides, const long long* cache_strides, const long long* slots,
                         int T, int H, int Hkv, int d, int num_pages, int page_size, const void* q_weight,
                         const void* k_weight, int weight_dtype, float eps, const int* positions,
                         const double* freqs, const int* axes, int n_axes, int rot, int interleaved,
                         fa_stream_t stream);

/*
 * fa_paged_slots -- a step's bookkeeping from its request lengths, on the GPU: what fa_paged_append, fa_fwd_paged
 * and fa_decode_paged take.  Sequence b has ctx_lens[b] tokens in the cache and gets new_lens[b] more, which follow
 * one another in the step's tokens, sequence by sequence.
 *   ctx_lens, new_lens  device int32 [B]; new_lens[b] <= 0: no new tokens (a place that is unused may have
 *                       a negative ctx_lens[b] too)
 *   page_table          device int32 [B, max_pages], rows table_stride entries apart: a sequence's new pages are
 *                       added behind the ceil(ctx_lens[b] / page_size) that it has
 *   free_pages          device int32 [n_free], free_count device int32 [1]: a stack of free pages, of which the top
 *                       ones are dealt, to the sequences in order: first free_pages[free_count - 1]
 *   T                   places for new tokens
 *   cu_seqlens          out, device int32 [B + 1]: sequence b's tokens are cu_seqlens[b] .. cu_seqlens[b + 1] - 1
 *   positions, slots    out, device int32 and int64 [T]: position and page * page_size + row of each token; 0 and -1
 *                       in places behind the last token
 *   seq_lens            out, device int32 [B]: ctx_lens[b] plus the new tokens; may be ctx_lens itself
 *   free_left           out, device int32 [1]: the free pages that are left; may be free_count itself
 * A sequence fails where ctx_lens[b] is negative, its tokens pass max_pages * page_size or the T places, or the free pages
 * do not reach for it and those before it: it gets no page, seq_lens[b] = -1 and slots of -1 (positions of 0), and
 * fa_check_device_error reports FA_ERR_INVALID_ARG.  The others are not affected.  (fa_fwd_paged gives a failed
 * sequence's tokens NaN.)  No other output may overlap an input.  max_pages * page_size < 2^30; B <= 16384
 * (FA_ERR_UNSUPPORTED above); B = 0 and T = 0 are steps without sequences or tokens.
 */
int fa_paged_slots(const int* ctx_lens, const int* new_lens, int* page_table, long long table_stride,
                   const int* free_pages, int n_free, const int* free_count, int B, int T, int page_size,
                   int max_pages, int* cu_seqlens, int* positions, long long* slots, int* seq_lens,
                   int* free_left, fa_stream_t stream);

/*
 * fa_fwd_paged -- attention of a ragged batch's new tokens (prompts, parts of prompts, drafts, single tokens) over a
 * paged cache that holds their keys and values already.  Sequence b has the tokens cu_seqlens[b] .. cu_seqlens[b + 1]
 * - 1 of q, n_b of them, the last of its seq_lens[b] keys: token i stands at position p = seq_lens[b] - n_b + i and
 * sees the keys 0 .. p (causal), or with window > 0 those of them with j > p - window or j < sinks.
 *
 *   q, o       [T, H, d] bf16 (o is written, contiguous); query head h reads key/value head h / (H / Hkv).
 *   q_strides  NULL = contiguous, or a HOST array of 2: the token and head strides of q in elements,
 *              multiples of 8; heads lie within a token (d <= head stride <= token stride).
 *   k_cache, v_cache, cache_strides, num_pages, page_size, page_table, table_stride   as in fa_decode_paged.  Pages
 *              that no token sees, behind a window, are not read: their entries may hold anything.
 *   cu_seqlens device int32 [B + 1], ascending, cu_seqlens[B] <= T.  Rows of o and lse behind cu_seqlens[B] are left
 *              as they were.
 *   seq_lens   device int32 [B], the new tokens included.
 *   window     0: none.       sinks  first keys that stay visible behind the window.
 *   scale, lse as in fa_decode_paged; lse [T, H].
 *   workspace  device buffer of at least fa_fwd_paged_workspace_bytes(T, B, H, Hkv, d) bytes, 16-byte aligned, or
 *              NULL to allocate it stream-ordered on `stream`.  It needs no clearing; calls that may overlap on the
 *              GPU must not share one.  A call that uses none (fa_fwd_paged_call_bytes) allocates none either, and
 *              takes a buffer of any size.
 * A sequence with seq_lens[b] below its new tokens or above max_pages * page_size gets NaN in o and lse, one
 * with a page outside the cache NaN in the tokens that the page reaches (and others near them); offsets that do
 * not ascend make their sequence's tokens stay unwritten, and give tokens that others then share unspecified values
 * or none.  fa_check_device_error then reports FA_ERR_INVALID_ARG.
 * Accumulation and softmax statistics are fp32.  No atomics on results: repeated calls on one GPU give identical bits
 * (other sizes of the call, a wider table, say, may change the last one).
 * H / Hkv <= 128, B <= 16384 (FA_ERR_UNSUPPORTED otherwise); max_pages * page_size < 2^30, T * (H / Hkv) <= 2^30 and
 * (T * (H / Hkv) / 128 + B + 1) * (max_pages * page_size / 64 + 3) < 2^31 (FA_ERR_INVALID_ARG otherwise).
 */
int fa_fwd_paged(const void* q, const void* k_cache, const void* v_cache, void* o, const int* page_table,
                 long long table_stride, const int* cu_seqlens, const int* seq_lens, int T, int B, int H,
                 int Hkv, int d, int num_pages, int page_size, int max_pages, const long long* q_strides,
                 const long long* cache_strides, float scale, int window, int sinks, void* workspace,
                 size_t workspace_bytes, float* lse, fa_stream_t stream);

/* Bytes of workspace that fa_fwd_paged needs on the current device at most, whatever its table and window are; 0 on bad
 * arguments or without an sm_103 GPU. */
size_t fa_fwd_paged_workspace_bytes(int T, int B, int H, int Hkv, int d);

/* What a call with tables of max_pages pages and this window uses of its workspace: all of it, or nothing (0: small calls,
 * whose units' states are joined on chip; 0 too on bad arguments or without an sm_103 GPU). */
size_t fa_fwd_paged_call_bytes(int T, int B, int H, int Hkv, int d, int page_size, int max_pages, int window, int sinks);

/*
 * fa_check_device_error -- reads and clears the library's device error word
 * on the current device (synchronises that device).  Returns FA_OK, or
 * FA_ERR_TIMEOUT if a kernel gave up on a wait since the last check (its
 * outputs are then undefined), or FA_ERR_INVALID_ARG if a kernel met an index
 * outside its range in device memory (a page, slot, length or axis of the entry
 * points above that say so), or FA_ERR_CUDA if the read itself failed.
 */
int fa_check_device_error(void);

/* Static, human-readable name of a status code. */
const char* fa_status_string(int status);

/*
 * fa_last_cuda_error -- the CUDA error behind the calling host thread's last
 * FA_ERR_CUDA (a cudaError_t value, or 100000 + a CUresult from tensor-map
 * encoding); 0 if none.  fa_last_cuda_error_string gives its static text.
 */
int fa_last_cuda_error(void);
const char* fa_last_cuda_error_string(void);

/*
 * fa_debug_set_fault -- TEST ONLY.  Arms a host-side fault for the next
 * fa_fwd / fa_fwd_ex or fa_bwd call on this process (whichever comes first):
 * mode 1 makes the load warp of the forward kernel skip its first key-tile
 * copy, or the load warp of the backward's dK/dV kernel skip its key/value
 * copy (and the expected-byte count), so the consumers' bounded waits run
 * out, the kernel abandons its work, records FA_ERR_TIMEOUT and returns.
 * An fp32 fa_bwd call disarms it without effect (its kernels have no waits).
 * mode 0 disarms.  Returns FA_OK or FA_ERR_INVALID_ARG.
 */
int fa_debug_set_fault(int mode);

#ifdef __cplusplus
}
#endif

#endif /* FA_H_ */
