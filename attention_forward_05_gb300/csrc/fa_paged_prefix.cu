// fa_paged_prefix.cu -- one query per head over a paged key/value cache behind a shared prefix.
//
// Sequence b sees the keys of the shared prefix (if any), then its own len_b cache rows through its row
// of the page table: o = softmax(scale q K^T) V and the natural-log LSE, by the online-softmax
// recurrence in log2 units.
//
// One CTA per (sequence, query head); each warp takes every eighth key, and the warps' partial states
// (m, l, o) merge at the end.
#include <cuda_bf16.h>

#include "fa_internal.h"
#include "sm103_ptx.cuh"

namespace fa {

namespace {
constexpr int PG_WARPS = 8;
enum : int { W_PAGE = 0x30, W_LEN };  // sites recorded with DEV_BAD_INDEX
}  // namespace

template <int D>
__global__ void __launch_bounds__(32 * PG_WARPS) fa_decode_paged_simple(const PagedLaunch a) {
  constexpr int E = D / 32;
  __shared__ float sm_m[PG_WARPS], sm_l[PG_WARPS], sm_o[PG_WARPS][D];
  const int b = blockIdx.x / a.H, h = blockIdx.x % a.H;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hk = h / (a.H / a.Hkv);
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (static_cast<long long>(b) * a.H + h) * D;
  float qf[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qf[e] = __bfloat162float(q[lane * E + e]) * a.c;
    o[e] = 0.f;
  }
  int len = a.lens[b];
  const bool idle = len < 0;
  bool bad = false;
  if (len > static_cast<long long>(a.max_pages) * a.page_size) bad = true;
  if (idle || bad) len = 0;
  const int total = idle ? 0 : a.prefix_len + len;
  float m = -INFINITY, l = 0.f;
  for (int j = warp; j < total && !bad; j += PG_WARPS) {
    const int i = j < a.prefix_len ? j : j - a.prefix_len;
    const int page = j < a.prefix_len ? a.prefix_pages[i / a.page_size] : a.table[b * a.table_stride + i / a.page_size];
    if (page < 0 || page >= a.num_pages) {
      bad = true;
      break;
    }
    const long long off = page * a.c_page + hk * a.c_head + i % a.page_size * a.c_row + lane * E;
    const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(a.k_cache) + off;
    const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v_cache) + off;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(qf[e], __bfloat162float(k[e]), s);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    const float m_new = fmaxf(m, s);
    const float ref = m_new == -INFINITY ? 0.f : m_new;
    const float alpha = ex2_approx(m - ref), p = ex2_approx(s - ref);
    l = l * alpha + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * alpha + p * __bfloat162float(v[e]);
    m = m_new;
  }
  if (bad) l = __int_as_float(0x7fc00000);
  if (lane == 0) {
    sm_m[warp] = m;
    sm_l[warp] = l;
    if (bad) record_bad_index(a.err, W_PAGE);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) sm_o[warp][lane * E + e] = o[e];
  __syncthreads();
  if (threadIdx.x < D) {
    float M = -INFINITY;
    for (int w = 0; w < PG_WARPS; ++w) M = fmaxf(M, sm_m[w]);
    const float ref = M == -INFINITY ? 0.f : M;
    float L = 0.f, O = 0.f;
    for (int w = 0; w < PG_WARPS; ++w) {
      const float wt = ex2_approx(sm_m[w] - ref);
      L += sm_l[w] * wt;
      O += sm_o[w][threadIdx.x] * wt;
    }
    const long long row = static_cast<long long>(b) * a.H + h;
    const bool nothing = total == 0 && !bad;
    static_cast<__nv_bfloat16*>(a.o)[row * D + threadIdx.x] = __float2bfloat16_rn(nothing ? 0.f : O / L);
    if (a.lse != nullptr && threadIdx.x == 0) a.lse[row] = nothing ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
  }
}

cudaError_t launch_decode_prefix(const PagedLaunch& a) {
  const unsigned grid = static_cast<unsigned>(a.B * a.H);
  if (a.d == 64) fa_decode_paged_simple<64><<<grid, 32 * PG_WARPS, 0, a.stream>>>(a);
  else fa_decode_paged_simple<128><<<grid, 32 * PG_WARPS, 0, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace fa
