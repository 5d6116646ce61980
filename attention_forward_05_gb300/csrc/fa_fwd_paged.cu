// fa_fwd_paged.cu -- attention of a ragged batch's new tokens over a paged key/value cache.
//
// Token i of sequence b's n_b new ones stands at position p = len_b - n_b + i and sees the keys 0 .. p, or with a sliding
// window w the keys p - w + 1 .. p and the first `sinks` ones: o = softmax(scale q K^T) V over those, and the LSE.
//
// One warp a (token, head): its lanes hold d / 32 elements each, every key costs a sum over the warp.
#include <cuda_bf16.h>

#include "fa_internal.h"
#include "sm103_ptx.cuh"

namespace fa {

namespace {

enum : int { W_FWD_PAGED = 0x48 };  // site recorded with DEV_BAD_INDEX

template <int D>
__global__ void __launch_bounds__(128) fa_fwd_paged_kernel(const FwdPagedLaunch a) {
  using bf = __nv_bfloat16;
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long w = static_cast<long long>(blockIdx.x) * 4 + threadIdx.x / 32;
  const int t = static_cast<int>(w / a.H), h = static_cast<int>(w % a.H), kvh = h / (a.H / a.Hkv);
  if (t >= a.T) return;
  int b = -1;
  for (int i = lane; i < a.B; i += 32) {
    const int from = a.cu[i], to = a.cu[i + 1];
    if (from < 0 || from > to || to > a.T) {
      if (w == 0) record_bad_index(a.err, W_FWD_PAGED);
    } else if (from <= t && t < to) {
      b = i;
    }
  }
  b = __reduce_max_sync(0xffffffffu, b);
  if (b < 0) return;
  const int first = a.cu[b], n = a.cu[b + 1] - first;
  const int len = a.lens[b], p = len - n + t - first;
  bool bad = len < n || len > static_cast<long long>(a.max_pages) * a.page_size;
  float q[E], o[E] = {}, m = -INFINITY, l = 0.f;
  for (int i = 0; i < E; ++i)
    q[i] = __bfloat162float(static_cast<const bf*>(a.q)[t * a.q_tok + h * a.q_head + lane * E + i]);
  const int from = a.window > 0 ? max(0, p - a.window + 1) : 0;
  for (int j = 0; !bad && j <= p; ++j) {
    if (j >= a.sinks && j < from) j = from;
    const int pg = a.table[b * a.table_stride + j / a.page_size];
    if (pg < 0 || pg >= a.num_pages) {
      bad = true;
      break;
    }
    const long long row = pg * a.c_page + kvh * a.c_head + j % a.page_size * a.c_row + lane * E;
    float s = 0.f;
    for (int i = 0; i < E; ++i) s = fmaf(q[i], __bfloat162float(static_cast<const bf*>(a.k_cache)[row + i]), s);
    for (int i = 1; i < 32; i *= 2) s += __shfl_xor_sync(0xffffffffu, s, i);
    s *= a.c;
    const float mn = fmaxf(m, s), al = exp2f(m - mn), e = exp2f(s - mn);
    m = mn;
    l = l * al + e;
    for (int i = 0; i < E; ++i) o[i] = o[i] * al + e * __bfloat162float(static_cast<const bf*>(a.v_cache)[row + i]);
  }
  if (bad) {
    record_bad_index(a.err, W_FWD_PAGED);
    l = __int_as_float(0x7fc00000);
  }
  const long long out = (static_cast<long long>(t) * a.H + h);
  for (int i = 0; i < E; ++i) static_cast<bf*>(a.o)[out * D + lane * E + i] = __float2bfloat16(o[i] / l);
  if (a.lse && lane == 0) a.lse[out] = (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace

size_t fwd_paged_workspace(int, int, int, int, int, int) { return 0; }

cudaError_t launch_fwd_paged(const FwdPagedLaunch& a) {
  const long long warps = static_cast<long long>(a.T) * a.H, grid = (warps + 3) / 4;
  if (a.d == 64)
    fa_fwd_paged_kernel<64><<<static_cast<unsigned>(grid), 128, 0, a.stream>>>(a);
  else
    fa_fwd_paged_kernel<128><<<static_cast<unsigned>(grid), 128, 0, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace fa
