// fa_internal.h -- launch interfaces between the C ABI (fa_api.cu) and the
// kernel translation units.  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <utility>

#include <nvtx3/nvToolsExt.h>

namespace fa {

// NVTX range over one C ABI call, named after the entry point, for timeline tools (Nsight Systems and
// the like).  Header-only NVTX: without an attached tool a push or pop is a cheap no-op.
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

// Launch with programmatic stream serialization: the kernel may start before the previous kernel in
// the stream has completed, once every CTA of that kernel has executed griddepcontrol.launch_dependents.
template <typename... KArgs, typename... Args>
cudaError_t launch_dependent(void (*kernel)(KArgs...), dim3 grid, int threads, int smem, cudaStream_t stream,
                             Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// The same in clusters of `cluster` CTAs (a divisor of the grid; above 8 the kernel has to allow it).
template <typename... KArgs, typename... Args>
cudaError_t launch_dependent_clusters(void (*kernel)(KArgs...), dim3 grid, int cluster, int threads, int smem,
                                      cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// The C ABI's per-device check for the current device: FA_OK on an sm_103 GPU (after fetching the
// library's device error word), FA_ERR_UNSUPPORTED on any other device, FA_ERR_CUDA when a runtime
// call fails.  Allocates nothing.
int current_device_status();

// The same with what the launch code needs: the device's error word and SM count.
int current_device_info(int** err, int* sms);

// Lets `kernel` have more than 48 KB of dynamic shared memory on the current device: set at its first launch there.
template <auto kernel>
cudaError_t allow_shared_memory(int bytes) {
  static std::atomic<unsigned long long> done{0};  // one bit a device (fa_api.cu takes up to 64)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (done.load(std::memory_order_acquire) >> dev & 1u)) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(1ull << dev, std::memory_order_release);
  return e;
}

// Records a CUDA error for fa_last_cuda_error() and returns FA_ERR_CUDA.
int report_cuda_error(cudaError_t e);

// Division of numbers below 2^31 by a fixed one.
struct FastDiv {
  unsigned mul, shift, d;
  explicit FastDiv(unsigned n) : mul(0), shift(0), d(n) {
    if (n <= 1) return;
    unsigned l = 0;
    while ((1u << l) < n) ++l;
    mul = static_cast<unsigned>((1ull << (31 + l)) / n + 1);
    shift = l - 1;
  }
  FastDiv() : FastDiv(1) {}
  __device__ __forceinline__ int div(int x) const {
    return d <= 1 ? x : static_cast<int>(__umulhi(static_cast<unsigned>(x), mul) >> shift);
  }
};

// Rotation of position pairs shared by fa_rope and fa_paged_append (fa_rope.cu).
struct Rotary {
  const double* freqs = nullptr;  // device [rot / 2], radians per position
  const int* axes = nullptr;      // device [rot / 2], position axis of each pair; nullptr: axis 0
  const int* pos = nullptr;       // device int32 positions: pos[axis * axis_stride + b * batch_stride + n]
  long long axis_stride = 0, batch_stride = 0;
  int n_axes = 1;
  int rot = 0;                    // elements rotated at the start of a head: a multiple of 16, <= d; 0: none
  int interleaved = 0;            // pairs (2i, 2i+1) instead of (i, i + rot/2)
  int inverse = 0;                // rotate by the negative angle (the gradient's rotation)
};

// Element strides of one [B, heads, N, d] operand (d contiguous).
struct RowStrides {
  long long b, h, n;
};

struct RopeLaunch {
  const void* q;
  const void* k;        // nullptr with Hkv = 0
  void* q_out;
  void* k_out;
  RowStrides sq, sk, sqo, sko;
  int B, H, Hkv, N, d;
  int bf16;
  Rotary r;
  int* err;
  int sms;
  cudaStream_t stream;
};
cudaError_t launch_rope(const RopeLaunch& a);

struct AppendLaunch {
  const void* q;        // nullptr with H = 0
  const void* k;
  const void* v;
  void* q_out;          // [T, H, d] contiguous
  void* k_cache;
  void* v_cache;
  long long q_tok, q_head, k_tok, k_head, v_tok, v_head;  // element strides of the new tokens
  long long c_page, c_head, c_row;                        // element strides of both caches
  const long long* slots;                                 // device [T]
  int T, H, Hkv, d, page_size;
  long long n_slots;    // num_pages * page_size
  Rotary r;
  int* err;
  int sms;
  cudaStream_t stream;
};
cudaError_t launch_append(const AppendLaunch& a);

// Norms of query and key heads ahead of the rotation (fa_norm_rope.cu).
struct HeadNorm {
  const void* wq;  // [d]
  const void* wk;  // [d]; nullptr without key heads
  int fp32;        // the weights' type: fp32, or bf16
  float eps;
};
cudaError_t launch_norm_rope(const RopeLaunch& a, const HeadNorm& nm);
cudaError_t launch_norm_append(const AppendLaunch& a, const HeadNorm& nm);

// The backward pass: q, k of the RopeLaunch are the outputs' gradients, q_out, k_out the inputs' ones.
struct NormBwd {
  const void* q;        // the forward pass's inputs
  const void* k;
  RowStrides sq, sk;
  float* dwq;           // [d]
  float* dwk;
  float* parts;         // workspace: [norm_bwd_parts(sms)][2][d]
};
int norm_bwd_parts(int sms);
cudaError_t launch_norm_rope_bwd(const RopeLaunch& a, const NormBwd& b, const HeadNorm& nm);

// Step bookkeeping (fa_slots.cu).
constexpr int SLOTS_MAX_B = 16384;  // sequences whose tables fit a CTA's shared memory
struct SlotsLaunch {
  const int* ctx_lens;      // [B]
  const int* new_lens;      // [B]
  int* page_table;          // [B, max_pages], rows table_stride apart
  const int* free_pages;    // [n_free]
  const int* free_count;    // [1]
  int* cu_seqlens;          // [B + 1]
  int* positions;           // [T]
  long long* slots;         // [T]
  int* seq_lens;            // [B]
  int* free_left;           // [1]
  long long table_stride;
  int B, T, n_free, page_size, max_pages;
  int* err;
  cudaStream_t stream;
};
cudaError_t launch_slots(const SlotsLaunch& a);

// Attention of a ragged batch's new tokens over the paged cache (fa_fwd_paged.cu).
constexpr int FWD_PAGED_MAX_B = 16384;  // sequences whose block counts fit the tile ring's shared memory
constexpr int FWD_PAGED_MAX_G = 128;    // query heads of a key/value head: rows of a query tile
struct FwdPagedLaunch {
  const void* q;            // [T, H, d] bf16, strides q_tok, q_head
  const void* k_cache;
  const void* v_cache;
  void* o;                  // [T, H, d] bf16
  float* lse;               // [T, H] or nullptr
  long long q_tok, q_head;
  long long c_page, c_head, c_row;  // element strides of both caches
  const int* table;         // [B, max_pages], rows table_stride apart
  const int* cu;            // [B + 1]
  const int* lens;          // [B]
  int T, B, H, Hkv, d, num_pages, page_size, max_pages;
  long long table_stride;
  int window, sinks;        // window 0: every key up to the token's own
  float c;                  // scale * log2(e)
  char* ws;                 // fwd_paged_workspace(...) bytes where the call is dealt to ranges
  int* err;
  int sms;
  cudaStream_t stream;
};
// How a call is split, by its sizes (T to max_pages, window, sinks) and the SM count alone.
struct FwdPagedForm {
  int cl;    // CTAs of each unit's cluster; 0: dealt to ranges, which take the workspace
  int wide;  // clusters with key tiles of 128 (d = 128)
};
FwdPagedForm fwd_paged_form(const FwdPagedLaunch& a);
size_t fwd_paged_workspace(int T, int H, int Hkv, int d, int sms);
cudaError_t launch_fwd_paged(const FwdPagedLaunch& a, FwdPagedForm form);

struct PagedLaunch {
  const void* q;            // [B, H, d] bf16
  const void* k_cache;
  const void* v_cache;
  void* o;                  // [B, H, d] bf16
  float* lse;               // [B, H] or nullptr
  long long c_page, c_head, c_row;  // element strides of both caches
  const int* table;         // [B, max_pages], rows table_stride apart
  const int* lens;          // [B]
  const int* prefix_pages;  // [ceil(prefix_len / page_size)]
  int B, H, Hkv, d, num_pages, page_size, max_pages;
  long long table_stride;
  int prefix_len;
  float c;                  // scale * log2(e)
  char* ws;                 // paged_plan(...).total bytes
  int* err;
  int sms;
  cudaStream_t stream;
};
// Work split and workspace layout (byte offsets) of a paged decode.
struct PagedPlan {
  int n_cta = 0;                                      // CTAs that share the sequences' own keys
  int cl = 0;                                         // or CTAs of each unit; without a prefix those need no workspace
  size_t part_ml = 0, part_o = 0, infos = 0;          // states of units shared by warps (fa_paged.cu)
  // with a shared prefix:
  int n_split = 0, kv_per_split = 0, wide = 0;        // the prefix's key splits; wide: two query tiles per CTA
  size_t pre_ml = 0, pre_o = 0, unit_ml = 0, unit_o = 0;
  int gather_len = 0, gather_rows = 0;                // pages (of gather_rows rows) the prefix is first copied into; 0: none
  size_t gather_k = 0, gather_v = 0, gather_pages = 0;
  size_t total = 0;
};
// max_pages: of a sequence's table; 0: any.
PagedPlan paged_plan(int B, int H, int Hkv, int d, int page_size, int max_pages, int prefix_len, int sms);
cudaError_t launch_decode_paged(const PagedLaunch& a, const PagedPlan& pl);

struct FwdLaunch {
  const CUtensorMap* tm_q;  // 3-D maps over [B*H, N, d] (innermost d), 128-byte swizzle
  const CUtensorMap* tm_k;
  const CUtensorMap* tm_v;
  void* o;                  // [B, H, Nq, d], same dtype as the inputs
  float* lse;               // [B, H, Nq] or nullptr
  int* err;                 // device error word
  int BH, Nq, Nk;
  int H, Hkv;               // query heads per batch, key/value heads per batch (H % Hkv == 0)
  int kv_per_split;         // keys per split, a multiple of the key tile (Nk rounded up when not split)
  int n_split;              // key splits; > 1 writes partial states to ws_o / ws_ml for fa_fwd_merge
  float* ws_o;              // [n_split][BH][Nq][d] fp32 unnormalised O
  float* ws_ml;             // [n_split][BH][Nq][2] fp32 (m in log2 units, l)
  int causal;               // 1: query row i sees keys j <= i + Nk - Nq (requires Nq <= Nk)
  float c;                  // scale * log2(e)
  float tau;                // lazy-rescale threshold in log2 units (0 = rescale whenever m grows)
  int fault;                // test-only fault injection mode (0 = none)
  cudaStream_t stream;
  int dependent = 0;        // 1: the fp32 prep kernel precedes it on `stream` (programmatic dependent launch)
  // Key-split CTAs (bf16, d = 64, no mask, n_split == 1; ks_half = 0: none): the grid is ks_whole usual
  // CTAs (units 0 .. ks_whole - 1) and then ks_count CTAs of one 128-row query tile each (tiles
  // ks_tile0 .. of the head-major list of 128-row tiles), whose two tile slots take the keys [0, ks_half)
  // and [ks_half, Nk) and merge (fa_fwd_kernel.cuh, FwdParams).
  int ks_whole = 0, ks_tile0 = 0, ks_count = 0, ks_half = 0;
  // Paged keys and a decode batch's queries (fa_fwd_kernel.cuh, FwdPagedParams); tm_q is not used.
  const void* paged_q = nullptr;  // [B, Hkv * G, d]
  const int* pages = nullptr;
  int G = 0, num_pages = 0, page_size = 0, box_rows = 0, heads_inner = 0;
};

// Tile geometry the tensor maps must be encoded with, per instantiation.
struct FwdGeometry {
  int box_cols;     // elements per 128-byte row segment (64 bf16, 32 fp32)
  int q_rows;       // rows per Q box (128)
  int kv_rows;      // rows per K box (the KV tile, Bc)
  int v_kmajor;     // 1: V is read from a key-major copy [BH, d, Nk_pad] with boxes (32 keys, d rows)
  int rows_per_cta; // query rows one CTA covers
  int ctas_per_sm;  // CTAs of this instantiation resident per SM
};

FwdGeometry fwd_geometry(int dtype_is_bf16, int d);
FwdGeometry fwd_geometry_bf16(int d);

// Merge of per-split partial states into O (dtype of the forward) and LSE:
// O = sum_s o_s 2^(m_s - M) / sum_s l_s 2^(m_s - M), M = max_s m_s; LSE = (M + log2 L) ln 2.
// `order`: nullptr (index order) or a device int32 permutation of 0 .. n_split - 1.
cudaError_t launch_fwd_merge(const float* ws_o, const float* ws_ml, void* o, float* lse, long long rows, int d,
                             int n_split, int out_bf16, cudaStream_t stream, const int* order = nullptr);

// fp32 prep pass: qr = tf32(q), kr = tf32(k) (round to nearest), and the key-major copy
// vt[bh][c][j] = tf32(v[bh][j][c]) for j < Nk, 0 for Nk <= j < Nk_pad.
cudaError_t launch_prep_fp32(const float* q, const float* k, const float* v, float* qr, float* kr, float* vt,
                             int BH, int BHkv, int Nq, int Nk, int Nk_pad, int d, cudaStream_t stream);
cudaError_t launch_fwd_bf16_d64(const FwdLaunch& a);
cudaError_t launch_fwd_bf16_d128(const FwdLaunch& a);
cudaError_t launch_fwd_fp32_d64(const FwdLaunch& a);
cudaError_t launch_fwd_fp32_d128(const FwdLaunch& a);
// bf16 forward shaped for grouped-query decode (one query tile per CTA); see fa_fwd_decode.cu
// `sms`: the device's SM count (picks the d = 64 configuration whose CTAs start in one wave, if any)
cudaError_t launch_fwd_decode(const FwdLaunch& a, int d, int sms);
FwdGeometry fwd_geometry_decode(int d);

// Attention of all a decode batch's queries over the shared prefix's pages (fa_paged_prefix.cu): partial states
// [n_split][Hkv][B * G] into the workspace.
void plan_prefix(int B, int G, int Hkv, int d, int page_size, int prefix_len, int sms, PagedPlan* pl);
cudaError_t launch_prefix(const PagedLaunch& a, const PagedPlan& pl);

// 4-D tensor map over a paged cache: dims (d, page_size, Hkv, num_pages) with boxes of (64, box_rows, 1, 1), or with
// rows and heads exchanged (heads_inner); 128-byte swizzle.
cudaError_t encode_paged_map(CUtensorMap* map, const void* base, int d, int page_size, int Hkv, int num_pages,
                             long long c_row, long long c_head, long long c_page, int box_rows, int heads_inner);

// 3-D tensor map over queries [T, H, d]: dims (d, H, T) with boxes of (64, G, tokens); 128-byte swizzle.
cudaError_t encode_heads_map(CUtensorMap* map, const void* base, int d, int H, int T, long long head, long long token, int G,
                             int tokens);

struct BwdLaunch {
  // maps for the dK/dV kernel: K, V boxes (64 cols, kv_keys rows); Q, dO boxes (64 cols, kv_qrows rows)
  const CUtensorMap* tm_k_kv;
  const CUtensorMap* tm_v_kv;
  const CUtensorMap* tm_q_kv;
  const CUtensorMap* tm_do_kv;
  // maps for the dQ kernel: Q, dO boxes (64 cols, q_rows rows); K, V boxes (64 cols, q_keys rows)
  const CUtensorMap* tm_q_q;
  const CUtensorMap* tm_do_q;
  const CUtensorMap* tm_k_q;
  const CUtensorMap* tm_v_q;
  const void* q;            // [BH, Nq, d] (read directly by the fp32 kernels; bf16 reads through the maps)
  const void* k;            // [BHkv, Nk, d]
  const void* v;
  const void* o;            // [BH, Nq, d] forward output, in the inputs' dtype
  const void* dout;         // [BH, Nq, d]
  const float* lse;         // [BH, Nq] natural-log LSE of the forward
  void* dq;                 // [BH, Nq, d]
  void* dk;                 // [BHkv, Nk, d]
  void* dv;
  float* rowv;              // bf16: workspace [BH][Nq_pad/2][4]: (-L log2 e, -D) interleaved by row pairs;
                            // fp32: [BH][Nq_pad] of -L log2 e
  float* rowv2;             // fp32: [BH][Nq_pad] of -D
  int* err;
  int BH, BHkv, H, Hkv, Nq, Nk, Nq_pad, d;
  int causal;
  float c;                  // scale * log2(e)
  float scale;
  int fault;                // test-only fault injection mode for the dK/dV kernel (0 = none)
  cudaStream_t stream;
};

struct BwdGeometry {
  int kv_keys;   // keys per dK/dV CTA
  int kv_qrows;  // query rows per dK/dV step
  int q_rows;    // query rows per dQ tile
  int q_keys;    // keys per dQ step
  int nq_align;  // Nq_pad is Nq rounded up to this
};

BwdGeometry bwd_geometry(int d);
// prep pass, then dK/dV, then dQ, in stream order
cudaError_t launch_bwd_bf16(const BwdLaunch& a);
// fp32 tensors, fp32 arithmetic on the CUDA cores (fa_bwd_fp32.cu); the same three launches.  Nq_pad
// must be a multiple of bwd_fp32_nq_align().
cudaError_t launch_bwd_fp32(const BwdLaunch& a);
int bwd_fp32_nq_align();

struct DecodeLaunch {
  const void* q;            // [BH, d] bf16
  const void* k;            // [BH, Nk, d] bf16
  const void* v;
  void* o;                  // [BH, d] bf16
  float* lse;               // [BH] or nullptr
  float* ws;                // workspace: m [BH*splits], l [BH*splits], o [BH*splits*d]
  const int* order;         // [splits] or nullptr
  int BH, Nk, d, splits;
  float c;                  // scale * log2(e)
  cudaStream_t stream;
};

cudaError_t launch_decode(const DecodeLaunch& a);

// Merge of per-(head, chunk) decode states in `order` (or 0..splits-1): o = sum w o_s / sum w l_s.
cudaError_t launch_decode_merge(const float* ws_m, const float* ws_l, const float* ws_o, const int* order, void* o,
                                float* lse, int BH, int splits, int d, cudaStream_t stream);

struct DecodeGqaLaunch {
  const void* q;            // [B, H, d] bf16
  const void* k;            // [B, Hkv, Nk, d] bf16
  const void* v;
  void* o;                  // [B, H, d] bf16
  float* lse;               // [B, H] or nullptr
  float* ws;                // m [B*H*splits], l [B*H*splits], o [B*H*splits*d]
  const int* order;         // [splits] or nullptr
  int* err;                 // device error word
  int B, H, Hkv, Nk, d, splits;
  float c;                  // scale * log2(e)
  cudaStream_t stream;
};

// 1 when one CTA can serve a group of this many query heads per key/value head (1, 2, 4 or a
// multiple of 8).
int decode_gqa_supported_group(int group);
cudaError_t launch_decode_gqa(const DecodeGqaLaunch& a);

}  // namespace fa
