// fa_paged_api.cu -- C ABI of the position and paged-cache entry points declared in include/fa.h:
// fa_rope, fa_norm_rope, fa_paged_append, fa_decode_paged, fa_decode_paged_prefix, fa_paged_slots, fa_fwd_paged.  Host
// code: argument validation, workspaces, launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "fa.h"
#include "fa_internal.h"

namespace {

constexpr long long kMaxElems = 1LL << 38;  // strides in bytes stay below the tensor maps' 2^40

constexpr long long kMaxTokens = (1LL << 31) - 1024;  // token indices of a block stay below 2^31

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Strides in elements whose rows must start on 16-byte boundaries; `unit` elements are 16 bytes.
bool good_strides(const long long* s, int n, int unit) {
  for (int i = 0; i < n; ++i)
    if (s[i] < 0 || s[i] > kMaxElems || s[i] % unit != 0) return false;
  return true;
}

// No dimension of several entries stands still.
bool distinct(const long long* s, int n0, int n1, int n2) {
  return (s[0] > 0 || n0 == 1) && (s[1] > 0 || n1 == 1) && (s[2] > 0 || n2 == 1);
}

bool good_cache(const long long* c, int num_pages, int Hkv, int page_size) {
  return good_strides(c, 3, 8) && distinct(c, num_pages, Hkv, page_size);
}

bool needs_workspace(const fa::PagedPlan& plan, int prefix_len) { return plan.cl == 0 || prefix_len > 0; }

// Arguments of a rotation; rot = 0 (no rotation) is the caller's business.
int check_rotation(const int* positions, const double* freqs, const int* axes, int n_axes, int rot, int interleaved,
                   int d) {
  if (!positions || !freqs || !aligned(positions, 4) || !aligned(freqs, 8) || (axes && !aligned(axes, 4)))
    return FA_ERR_INVALID_ARG;
  if (n_axes < 1 || rot < 1 || rot > d || (interleaved != 0 && interleaved != 1)) return FA_ERR_INVALID_ARG;
  if (n_axes > 8 || rot % 16 != 0) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// Norms' weights, of query heads and, where there are any, of key heads.
int check_norm(const void* wq, const void* wk, int heads_q, int heads_k, int weight_dtype, float eps) {
  if ((wq == nullptr) != (heads_q == 0) || (wk == nullptr) != (heads_k == 0)) return FA_ERR_INVALID_ARG;
  if (weight_dtype != FA_BF16 && weight_dtype != FA_FP32) return FA_ERR_UNSUPPORTED;
  const unsigned n = weight_dtype == FA_FP32 ? 4 : 2;
  if (!aligned(wq, n) || !aligned(wk, n)) return FA_ERR_INVALID_ARG;
  return std::isfinite(eps) && eps >= 0.f ? FA_OK : FA_ERR_INVALID_ARG;
}

// Checks and fills what fa_rope and fa_norm_rope share.  Their rotation may be left out where `norm` is given.
int rope_launch(fa::RopeLaunch* a, const void* q, const void* k, void* q_out, void* k_out, const long long* strides, int B,
                int H, int Hkv, int N, int d, int dtype, const int* positions, int pos_shared, const double* freqs,
                const int* axes, int n_axes, int rot, int interleaved, int inverse, bool norm) {
  if (!q || !q_out || (k == nullptr) != (k_out == nullptr) || (k == nullptr) != (Hkv == 0)) return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(q_out, 16) || !aligned(k, 16) || !aligned(k_out, 16)) return FA_ERR_INVALID_ARG;
  if (B < 1 || H < 1 || Hkv < 0 || N < 1) return FA_ERR_INVALID_ARG;
  if ((pos_shared != 0 && pos_shared != 1) || (inverse != 0 && inverse != 1)) return FA_ERR_INVALID_ARG;
  if (dtype != FA_BF16 && dtype != FA_FP32) return FA_ERR_UNSUPPORTED;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  int rc = FA_OK;
  if (!norm || rot != 0 || freqs || positions) rc = check_rotation(positions, freqs, axes, n_axes, rot, interleaved, d);
  if (rc != FA_OK) return rc;
  const long long heads = static_cast<long long>(H) + Hkv, tokens = static_cast<long long>(B) * N;
  if (tokens > kMaxTokens || heads > 0x7FFFFFFFLL / d || tokens > kMaxElems / (heads * d)) return FA_ERR_INVALID_ARG;
  long long s[12];
  for (int i = 0; i < 4; ++i) {
    const long long h = (i & 1) ? Hkv : H;
    s[3 * i] = strides ? strides[3 * i] : h * N * d;
    s[3 * i + 1] = strides ? strides[3 * i + 1] : static_cast<long long>(N) * d;
    s[3 * i + 2] = strides ? strides[3 * i + 2] : d;
  }
  if (!good_strides(s, 12, dtype == FA_BF16 ? 8 : 4)) return FA_ERR_INVALID_ARG;
  for (int i = 2; i < (k ? 4 : 3); ++i)  // an input may be broadcast, an output may not
    if (!distinct(s + 3 * i, B, i == 2 ? H : Hkv, N)) return FA_ERR_INVALID_ARG;
  if ((rc = fa::current_device_info(&a->err, &a->sms)) != FA_OK) return rc;
  a->q = q;
  a->k = k;
  a->q_out = q_out;
  a->k_out = k_out;
  a->sq = {s[0], s[1], s[2]};
  a->sk = {s[3], s[4], s[5]};
  a->sqo = {s[6], s[7], s[8]};
  a->sko = {s[9], s[10], s[11]};
  a->B = B;
  a->H = H;
  a->Hkv = Hkv;
  a->N = N;
  a->d = d;
  a->bf16 = dtype == FA_BF16;
  a->r.freqs = freqs;
  a->r.axes = axes;
  a->r.pos = positions;
  a->r.axis_stride = pos_shared ? N : tokens;
  a->r.batch_stride = pos_shared ? 0 : N;
  a->r.n_axes = n_axes;
  a->r.rot = rot;
  a->r.interleaved = rot ? interleaved : 0;
  a->r.inverse = inverse;
  return FA_OK;
}

// fa_paged_append, with norms where `nm` is given.
int append_call(const void* k, const void* v, const void* q, void* q_out, void* k_cache, void* v_cache,
                const long long* in_strides, const long long* cache_strides, const long long* slots, int T, int H, int Hkv,
                int d, int num_pages, int page_size, const int* positions, const double* freqs, const int* axes, int n_axes,
                int rot, int interleaved, fa_stream_t stream, const fa::HeadNorm* nm) {
  if (!k || !v || !k_cache || !v_cache || !slots) return FA_ERR_INVALID_ARG;
  if ((q == nullptr) != (q_out == nullptr) || (q == nullptr) != (H == 0)) return FA_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(q, 16) || !aligned(q_out, 16) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16) || !aligned(slots, 8))
    return FA_ERR_INVALID_ARG;
  if (T < 0 || H < 0 || Hkv < 1 || num_pages < 1 || page_size < 1) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (rot != 0 || freqs || positions) {
    const int rc = check_rotation(positions, freqs, axes, n_axes, rot, interleaved, d);
    if (rc != FA_OK) return rc;
  }
  const long long heads = static_cast<long long>(H) + 2LL * Hkv;
  if (T > kMaxTokens || heads > 0x7FFFFFFFLL / d || T > kMaxElems / (heads * d)) return FA_ERR_INVALID_ARG;
  long long s[6], c[3];
  for (int i = 0; i < 3; ++i) {
    s[2 * i] = in_strides ? in_strides[2 * i] : static_cast<long long>(i < 2 ? Hkv : H) * d;
    s[2 * i + 1] = in_strides ? in_strides[2 * i + 1] : d;
  }
  c[0] = cache_strides ? cache_strides[0] : static_cast<long long>(Hkv) * page_size * d;
  c[1] = cache_strides ? cache_strides[1] : static_cast<long long>(page_size) * d;
  c[2] = cache_strides ? cache_strides[2] : d;
  if (!good_strides(s, 6, 8) || !good_cache(c, num_pages, Hkv, page_size)) return FA_ERR_INVALID_ARG;
  fa::AppendLaunch a;
  const int rc = fa::current_device_info(&a.err, &a.sms);
  if (rc != FA_OK) return rc;
  if (T == 0) return FA_OK;  // a step without new tokens
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_out = q_out;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_tok = s[0];
  a.k_head = s[1];
  a.v_tok = s[2];
  a.v_head = s[3];
  a.q_tok = s[4];
  a.q_head = s[5];
  a.c_page = c[0];
  a.c_head = c[1];
  a.c_row = c[2];
  a.slots = slots;
  a.T = T;
  a.H = H;
  a.Hkv = Hkv;
  a.d = d;
  a.page_size = page_size;
  a.n_slots = static_cast<long long>(num_pages) * page_size;
  a.r.freqs = freqs;
  a.r.axes = axes;
  a.r.pos = positions;
  a.r.axis_stride = T;
  a.r.n_axes = n_axes;
  a.r.rot = rot;
  a.r.interleaved = rot ? interleaved : 0;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = nm ? fa::launch_norm_append(a, *nm) : fa::launch_append(a);
  return e == cudaSuccess ? FA_OK : fa::report_cuda_error(e);
}

}  // namespace

extern "C" {

int fa_rope(const void* q, const void* k, void* q_out, void* k_out, const long long* strides, int B, int H, int Hkv,
            int N, int d, int dtype, const int* positions, int pos_shared, const double* freqs, const int* axes,
            int n_axes, int rot, int interleaved, int inverse, fa_stream_t stream) {
  const fa::NvtxRange nvtx_range("fa_rope");
  fa::RopeLaunch a;
  const int rc = rope_launch(&a, q, k, q_out, k_out, strides, B, H, Hkv, N, d, dtype, positions, pos_shared, freqs, axes,
                             n_axes, rot, interleaved, inverse, false);
  if (rc != FA_OK) return rc;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = fa::launch_rope(a);
  return e == cudaSuccess ? FA_OK : fa::report_cuda_error(e);
}

int fa_paged_append(const void* k, const void* v, const void* q, void* q_out, void* k_cache, void* v_cache,
                    const long long* in_strides, const long long* cache_strides, const long long* slots, int T, int H,
                    int Hkv, int d, int num_pages, int page_size, const int* positions, const double* freqs,
                    const int* axes, int n_axes, int rot, int interleaved, fa_stream_t stream) {
  const fa::NvtxRange nvtx_range("fa_paged_append");
  return append_call(k, v, q, q_out, k_cache, v_cache, in_strides, cache_strides, slots, T, H, Hkv, d, num_pages, page_size,
                     positions, freqs, axes, n_axes, rot, interleaved, stream, nullptr);
}

int fa_paged_append_norm(const void* k, const void* v, const void* q, void* q_out, void* k_cache, void* v_cache,
                         const long long* in_strides, const long long* cache_strides, const long long* slots, int T, int H,
                         int Hkv, int d, int num_pages, int page_size, const void* q_weight, const void* k_weight,
                         int weight_dtype, float eps, const int* positions, const double* freqs, const int* axes,
                         int n_axes, int rot, int interleaved, fa_stream_t stream) {
  const fa::NvtxRange nvtx_range("fa_paged_append_norm");
  const int rc = check_norm(q_weight, k_weight, H, 1, weight_dtype, eps);
  if (rc != FA_OK) return rc;
  const fa::HeadNorm nm{q_weight, k_weight, weight_dtype == FA_FP32, eps};
  return append_call(k, v, q, q_out, k_cache, v_cache, in_strides, cache_strides, slots, T, H, Hkv, d, num_pages, page_size,
                     positions, freqs, axes, n_axes, rot, interleaved, stream, &nm);
}

int fa_norm_rope(const void* q, const void* k, void* q_out, void* k_out, const long long* strides, int B, int H, int Hkv,
                 int N, int d, int dtype, const void* q_weight, const void* k_weight, int weight_dtype, float eps,
                 const int* positions, int pos_shared, const double* freqs, const int* axes, int n_axes, int rot,
                 int interleaved, fa_stream_t stream) {
  const fa::NvtxRange nvtx_range("fa_norm_rope");
  int rc = check_norm(q_weight, k_weight, 1, Hkv, weight_dtype, eps);
  if (rc != FA_OK) return rc;
  fa::RopeLaunch a;
  rc = rope_launch(&a, q, k, q_out, k_out, strides, B, H, Hkv, N, d, dtype, positions, pos_shared, freqs, axes, n_axes, rot,
                   interleaved, 0, true);
  if (rc != FA_OK) return rc;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = fa::launch_norm_rope(a, fa::HeadNorm{q_weight, k_weight, weight_dtype == FA_FP32, eps});
  return e == cudaSuccess ? FA_OK : fa::report_cuda_error(e);
}

size_t fa_norm_rope_bwd_workspace_bytes(int d) {
  int* err = nullptr;
  int sms = 0;
  if ((d != 64 && d != 128) || fa::current_device_info(&err, &sms) != FA_OK) return 0;
  return static_cast<size_t>(fa::norm_bwd_parts(sms)) * 2 * d * sizeof(float);
}

int fa_norm_rope_bwd(const void* dq, const void* dk, const void* q, const void* k, void* dq_in, void* dk_in,
                     float* dq_weight, float* dk_weight, const long long* strides, int B, int H, int Hkv, int N, int d,
                     int dtype, const void* q_weight, const void* k_weight, int weight_dtype, float eps,
                     const int* positions, int pos_shared, const double* freqs, const int* axes, int n_axes, int rot,
                     int interleaved, void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  const fa::NvtxRange nvtx_range("fa_norm_rope_bwd");
  int rc = check_norm(q_weight, k_weight, 1, Hkv, weight_dtype, eps);
  if (rc != FA_OK) return rc;
  if (!q || (k == nullptr) != (Hkv == 0) || !dq_weight || (dk_weight == nullptr) != (Hkv == 0)) return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(dq_weight, 4) || !aligned(dk_weight, 4) || !aligned(workspace, 16))
    return FA_ERR_INVALID_ARG;
  const long long* const s = strides;  // of dq, dk, dq_in, dk_in, then of q and k
  if (s && !good_strides(s + 12, 6, dtype == FA_BF16 ? 8 : 4)) return FA_ERR_INVALID_ARG;
  fa::RopeLaunch a;
  rc = rope_launch(&a, dq, dk, dq_in, dk_in, strides, B, H, Hkv, N, d, dtype, positions, pos_shared, freqs, axes, n_axes,
                   rot, interleaved, 1, true);
  if (rc != FA_OK) return rc;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  const size_t need = static_cast<size_t>(fa::norm_bwd_parts(a.sms)) * 2 * d * sizeof(float);
  if (workspace && workspace_bytes < need) return FA_ERR_INVALID_ARG;
  void* ws = workspace;
  if (!workspace) {
    const cudaError_t ea = cudaMallocAsync(&ws, need, a.stream);
    if (ea != cudaSuccess) return fa::report_cuda_error(ea);
  }
  fa::NormBwd b;
  b.q = q;
  b.k = k;
  const long long h = static_cast<long long>(N) * d;
  b.sq = s ? fa::RowStrides{s[12], s[13], s[14]} : fa::RowStrides{H * h, h, d};
  b.sk = s ? fa::RowStrides{s[15], s[16], s[17]} : fa::RowStrides{Hkv * h, h, d};
  b.dwq = dq_weight;
  b.dwk = dk_weight;
  b.parts = static_cast<float*>(ws);
  cudaError_t e = fa::launch_norm_rope_bwd(a, b, fa::HeadNorm{q_weight, k_weight, weight_dtype == FA_FP32, eps});
  if (!workspace) {
    const cudaError_t e2 = cudaFreeAsync(ws, a.stream);
    if (e == cudaSuccess) e = e2;
  }
  return e == cudaSuccess ? FA_OK : fa::report_cuda_error(e);
}

int fa_paged_slots(const int* ctx_lens, const int* new_lens, int* page_table, long long table_stride,
                   const int* free_pages, int n_free, const int* free_count, int B, int T, int page_size, int max_pages,
                   int* cu_seqlens, int* positions, long long* slots, int* seq_lens, int* free_left, fa_stream_t stream) {
  const fa::NvtxRange nvtx_range("fa_paged_slots");
  if (B < 0 || T < 0 || n_free < 0 || page_size < 1 || max_pages < 1 || table_stride < max_pages) return FA_ERR_INVALID_ARG;
  if (!free_count || !cu_seqlens || !free_left || (n_free > 0 && !free_pages)) return FA_ERR_INVALID_ARG;
  if (B > 0 && (!ctx_lens || !new_lens || !page_table || !seq_lens)) return FA_ERR_INVALID_ARG;
  if (T > 0 && (!positions || !slots)) return FA_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(ctx_lens), static_cast<const void*>(new_lens),
                        static_cast<const void*>(page_table), static_cast<const void*>(free_pages),
                        static_cast<const void*>(free_count), static_cast<const void*>(cu_seqlens),
                        static_cast<const void*>(positions), static_cast<const void*>(seq_lens),
                        static_cast<const void*>(free_left)})
    if (!aligned(p, 4)) return FA_ERR_INVALID_ARG;
  if (!aligned(slots, 8)) return FA_ERR_INVALID_ARG;
  if (T > (1 << 30) || static_cast<long long>(max_pages) * page_size >= (1LL << 30)) return FA_ERR_INVALID_ARG;
  if (B > fa::SLOTS_MAX_B) return FA_ERR_UNSUPPORTED;
  fa::SlotsLaunch a;
  int sms = 0;
  const int rc = fa::current_device_info(&a.err, &sms);
  if (rc != FA_OK) return rc;
  a.ctx_lens = ctx_lens;
  a.new_lens = new_lens;
  a.page_table = page_table;
  a.free_pages = free_pages;
  a.free_count = free_count;
  a.cu_seqlens = cu_seqlens;
  a.positions = positions;
  a.slots = slots;
  a.seq_lens = seq_lens;
  a.free_left = free_left;
  a.table_stride = table_stride;
  a.B = B;
  a.T = T;
  a.n_free = n_free;
  a.page_size = page_size;
  a.max_pages = max_pages;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = fa::launch_slots(a);
  return e == cudaSuccess ? FA_OK : fa::report_cuda_error(e);
}

size_t fa_fwd_paged_call_bytes(int T, int B, int H, int Hkv, int d, int page_size, int max_pages, int window, int sinks) {
  if (page_size < 1 || max_pages < 1 || static_cast<long long>(max_pages) * page_size >= (1LL << 30) || window < 0 || sinks < 0)
    return 0;
  const size_t most = fa_fwd_paged_workspace_bytes(T, B, H, Hkv, d);
  fa::FwdPagedLaunch a = {};
  if (most == 0 || fa::current_device_info(&a.err, &a.sms) != FA_OK) return 0;
  a.T = T;
  a.B = B;
  a.H = H;
  a.Hkv = Hkv;
  a.d = d;
  a.page_size = page_size;
  a.max_pages = max_pages;
  a.window = window;
  a.sinks = sinks;
  return fa::fwd_paged_form(a).cl == 0 ? most : 0;
}

size_t fa_fwd_paged_workspace_bytes(int T, int B, int H, int Hkv, int d) {
  if (T < 1 || B < 1 || H < 1 || Hkv < 1 || H % Hkv != 0 || H / Hkv > fa::FWD_PAGED_MAX_G || B > fa::FWD_PAGED_MAX_B ||
      (d != 64 && d != 128) || static_cast<long long>(T) * H > kMaxElems / d)
    return 0;
  int* err = nullptr;
  int sms = 0;
  if (fa::current_device_info(&err, &sms) != FA_OK) return 0;
  return fa::fwd_paged_workspace(T, H, Hkv, d, sms);
}

int fa_fwd_paged(const void* q, const void* k_cache, const void* v_cache, void* o, const int* page_table,
                 long long table_stride, const int* cu_seqlens, const int* seq_lens, int T, int B, int H, int Hkv, int d,
                 int num_pages, int page_size, int max_pages, const long long* q_strides, const long long* cache_strides,
                 float scale, int window, int sinks, void* workspace, size_t workspace_bytes, float* lse,
                 fa_stream_t stream) {
  const fa::NvtxRange nvtx_range("fa_fwd_paged");
  if (!q || !k_cache || !v_cache || !o || !page_table || !cu_seqlens || !seq_lens) return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(o, 16) || !aligned(workspace, 16) ||
      !aligned(page_table, 4) || !aligned(cu_seqlens, 4) || !aligned(seq_lens, 4) || !aligned(lse, 4))
    return FA_ERR_INVALID_ARG;
  if (T < 0 || B < 0 || H < 1 || Hkv < 1 || H % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (num_pages < 1 || page_size < 1 || max_pages < 1 || table_stride < max_pages) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(max_pages) * page_size >= (1LL << 30)) return FA_ERR_INVALID_ARG;
  if (window < 0 || sinks < 0) return FA_ERR_INVALID_ARG;
  const float c2 = scale * 1.4426950408889634f;  // log2 units; the largest scales overflow here
  if (!std::isfinite(c2)) return FA_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || H / Hkv > fa::FWD_PAGED_MAX_G || B > fa::FWD_PAGED_MAX_B) return FA_ERR_UNSUPPORTED;
  // a key/value head's blocks of at least 128 rows and their tiles are counted in 32 bits, all heads' in 62
  if ((static_cast<long long>(T) * (H / Hkv) / 128 + B + 1) * (static_cast<long long>(max_pages) * page_size / 64 + 3) >
      0x7FFFFFFFLL)
    return FA_ERR_INVALID_ARG;
  if (H > (1 << 20) || static_cast<long long>(T) * H > (1LL << 36) ||
      static_cast<long long>(T) * (H / Hkv) > (1LL << 30))
    return FA_ERR_INVALID_ARG;
  long long qs[2], c[3];
  qs[0] = q_strides ? q_strides[0] : static_cast<long long>(H) * d;
  qs[1] = q_strides ? q_strides[1] : d;
  if (H == 1) qs[1] = d;  // never stepped over
  if (T <= 1) qs[0] = std::max(qs[1], static_cast<long long>(H) * d);
  if (!good_strides(qs, 2, 8) || qs[1] < d || qs[0] < qs[1]) return FA_ERR_INVALID_ARG;
  c[0] = cache_strides ? cache_strides[0] : static_cast<long long>(Hkv) * page_size * d;
  c[1] = cache_strides ? cache_strides[1] : static_cast<long long>(page_size) * d;
  c[2] = cache_strides ? cache_strides[2] : d;
  if (!good_cache(c, num_pages, Hkv, page_size)) return FA_ERR_INVALID_ARG;
  fa::FwdPagedLaunch a;
  const int rc = fa::current_device_info(&a.err, &a.sms);
  if (rc != FA_OK) return rc;
  if (T == 0 || B == 0) return FA_OK;  // a step without tokens
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.o = o;
  a.lse = lse;
  a.q_tok = qs[0];
  a.q_head = qs[1];
  a.c_page = c[0];
  a.c_head = c[1];
  a.c_row = c[2];
  a.table = page_table;
  a.cu = cu_seqlens;
  a.lens = seq_lens;
  a.T = T;
  a.B = B;
  a.H = H;
  a.Hkv = Hkv;
  a.d = d;
  a.num_pages = num_pages;
  a.page_size = page_size;
  a.max_pages = max_pages;
  a.table_stride = table_stride;
  a.window = window;
  a.sinks = sinks;
  a.c = c2;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  const fa::FwdPagedForm form = fa::fwd_paged_form(a);
  const size_t need = form.cl == 0 ? fa::fwd_paged_workspace(T, H, Hkv, d, a.sms) : 0;
  if (workspace && workspace_bytes < need) return FA_ERR_INVALID_ARG;
  void* ws = workspace;
  const bool own_ws = ws == nullptr && need > 0;
  if (own_ws) {
    const cudaError_t ea = cudaMallocAsync(&ws, need, a.stream);
    if (ea != cudaSuccess) return fa::report_cuda_error(ea);
  }
  a.ws = static_cast<char*>(ws);
  cudaError_t e = fa::launch_fwd_paged(a, form);
  if (own_ws) {
    const cudaError_t e2 = cudaFreeAsync(ws, a.stream);
    if (e == cudaSuccess) e = e2;
  }
  return e == cudaSuccess ? FA_OK : fa::report_cuda_error(e);
}

size_t fa_decode_paged_call_bytes(int B, int H, int Hkv, int d, int page_size, int max_pages, int prefix_len) {
  if (B < 1 || H < 1 || Hkv < 1 || H % Hkv != 0 || page_size < 1 || max_pages < 0 || prefix_len < 0 ||
      prefix_len >= (1 << 30) || (d != 64 && d != 128) || static_cast<long long>(B) * H > 0x7FFFFFFFLL / d)
    return 0;
  int* err = nullptr;
  int sms = 0;
  if (fa::current_device_info(&err, &sms) != FA_OK) return 0;
  const fa::PagedPlan plan = fa::paged_plan(B, H, Hkv, d, page_size, max_pages, prefix_len, sms);
  return needs_workspace(plan, prefix_len) ? plan.total : 0;
}

size_t fa_decode_paged_workspace_bytes(int B, int H, int Hkv, int d, int page_size, int prefix_len) {
  return fa_decode_paged_call_bytes(B, H, Hkv, d, page_size, 0, prefix_len);
}

int fa_decode_paged_prefix(const void* q, const void* k_cache, const void* v_cache, void* o, const int* prefix_pages,
                           int prefix_len, const int* page_table, long long table_stride, const int* seq_lens, int B,
                           int H, int Hkv, int d, int num_pages, int page_size, int max_pages,
                           const long long* cache_strides, float scale, void* workspace, size_t workspace_bytes,
                           float* lse, fa_stream_t stream) {
  const fa::NvtxRange nvtx_range("fa_decode_paged_prefix");
  if (!q || !k_cache || !v_cache || !o || !page_table || !seq_lens) return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(o, 16) || !aligned(workspace, 16) ||
      !aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(prefix_pages, 4) || !aligned(lse, 4))
    return FA_ERR_INVALID_ARG;
  if (B < 1 || H < 1 || Hkv < 1 || H % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (num_pages < 1 || page_size < 1 || max_pages < 1 || table_stride < max_pages) return FA_ERR_INVALID_ARG;
  if (prefix_len < 0 || prefix_len >= (1 << 30) || (prefix_len > 0 && !prefix_pages)) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(max_pages) * page_size >= (1LL << 30)) return FA_ERR_INVALID_ARG;
  // the tiles of a CTA's share are counted in 32 bits
  if (static_cast<long long>(max_pages) * page_size / 64 + 3 > (1LL << 39) / B / H) return FA_ERR_INVALID_ARG;
  const float c2 = scale * 1.4426950408889634f;  // log2 units; the largest scales overflow here
  if (!std::isfinite(c2)) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * H > 0x7FFFFFFFLL / d) return FA_ERR_INVALID_ARG;
  long long c[3];
  c[0] = cache_strides ? cache_strides[0] : static_cast<long long>(Hkv) * page_size * d;
  c[1] = cache_strides ? cache_strides[1] : static_cast<long long>(page_size) * d;
  c[2] = cache_strides ? cache_strides[2] : d;
  if (!good_cache(c, num_pages, Hkv, page_size)) return FA_ERR_INVALID_ARG;
  fa::PagedLaunch a;
  const int rc = fa::current_device_info(&a.err, &a.sms);
  if (rc != FA_OK) return rc;
  const fa::PagedPlan plan = fa::paged_plan(B, H, Hkv, d, page_size, max_pages, prefix_len, a.sms);
  if (workspace && workspace_bytes < plan.total) return FA_ERR_INVALID_ARG;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  void* ws = workspace;
  const bool own_ws = ws == nullptr && needs_workspace(plan, prefix_len);
  if (own_ws) {
    const cudaError_t ea = cudaMallocAsync(&ws, plan.total, a.stream);
    if (ea != cudaSuccess) return fa::report_cuda_error(ea);
  }
  a.ws = static_cast<char*>(ws);
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.o = o;
  a.lse = lse;
  a.c_page = c[0];
  a.c_head = c[1];
  a.c_row = c[2];
  a.table = page_table;
  a.lens = seq_lens;
  a.prefix_pages = prefix_pages;
  a.B = B;
  a.H = H;
  a.Hkv = Hkv;
  a.d = d;
  a.num_pages = num_pages;
  a.page_size = page_size;
  a.max_pages = max_pages;
  a.table_stride = table_stride;
  a.prefix_len = prefix_len;
  a.c = c2;
  cudaError_t e = fa::launch_decode_paged(a, plan);
  if (own_ws) {
    const cudaError_t e2 = cudaFreeAsync(ws, a.stream);
    if (e == cudaSuccess) e = e2;
  }
  return e == cudaSuccess ? FA_OK : fa::report_cuda_error(e);
}

int fa_decode_paged(const void* q, const void* k_cache, const void* v_cache, void* o, const int* page_table,
                    long long table_stride, const int* seq_lens, int B, int H, int Hkv, int d, int num_pages,
                    int page_size, int max_pages, const long long* cache_strides, float scale, void* workspace,
                    size_t workspace_bytes, float* lse, fa_stream_t stream) {
  return fa_decode_paged_prefix(q, k_cache, v_cache, o, nullptr, 0, page_table, table_stride, seq_lens, B, H, Hkv, d,
                                num_pages, page_size, max_pages, cache_strides, scale, workspace, workspace_bytes, lse,
                                stream);
}

}  // extern "C"
