// fa_paged_prefix.cu -- a decode batch's attention over the prefix that all its sequences share.
//
// With one query per head, a sequence's products with a key are few; but the B sequences of a batch share the
// prefix's keys, so for each key/value head the B * G queries that read it are the rows of a prefill over those
// keys: the forward kernel's tensor-core tiles (fa_fwd_kernel.cuh), with K and V copied out of the cache's pages
// and partial states (m, l, unnormalised O) as its result.  The prefix is read once a key split instead of once
// a sequence, and for large batches the work is bound by the matrix rate.  The sequences' own keys follow in
// fa_paged_kernel (fa_paged.cu), whose clusters, or fa_paged_join_kernel behind it, join the states.
//
// Measured, the whole call: 16384 shared keys, 256 sequences (d = 128, 32 heads on 8) 96 us, 720 TFLOP/s of the formula's
// products (P V is done twice, FwdCfg::TWO), of which this kernel takes 74; 8192 shared keys, 32 sequences (d = 64) 15 us;
// 1000 and 5 7.5 us.  With P rounded to bf16 once: 78, 14 and 7.5 us, and o up to 40 % further from the formula.
//
// Configurations (fa_fwd_bf16.cu and fa_fwd_decode.cu have the same tiles): two 128-row query tiles per CTA, or
// one where the B * G rows of a head fit in it.
#include <cuda_bf16.h>

#include <cmath>

#include "fa_fwd_kernel.cuh"

namespace fa {

namespace {

using WideD64 = FwdCfg<__nv_bfloat16, 64, 64, 2, 4, 2, false, true>;
using WideD128 = FwdCfg<__nv_bfloat16, 128, 128, 2, 2, 1, true, true>;
using NarrowD64 = FwdCfg<__nv_bfloat16, 64, 64, 1, 3, 3, false, true>;
using NarrowD128 = FwdCfg<__nv_bfloat16, 128, 64, 1, 2, 2, false, true>;

constexpr int GATHER_PAGE = 64;  // rows of a gathered page
constexpr float kPrefixTau = 32.f;  // fa_api.cu, kLazyTau

// Rows of the largest copy that stays in one page and starts on a swizzle boundary: a power of two that divides
// the page size, at most the key tile.  Under 8 rows there is none.
int box_rows_of(int page_size, int bc) {
  int r = page_size & -page_size;
  return r > bc ? bc : r;
}

// The prefix's rows copied into whole pages of GATHER_PAGE rows, [pages][Hkv][GATHER_PAGE][d], for page sizes whose
// rows cannot be copied in boxes.  One thread moves 16 bytes of K and of V; a bad page makes its keys NaN.
// (No read-only loads here and in fa_paged_kernel: they are launched while their inputs may still be written.)
__global__ void __launch_bounds__(256) gather_prefix_kernel(const uint4* k, const uint4* v, uint4* gk, uint4* gv,
                                                            int* ids, const int* pages, int n, int Hkv, int pieces,
                                                            int num_pages, int page_size, long long c_page,
                                                            long long c_head, long long c_row, int* err) {
  griddep_launch_dependents();
  griddep_wait();
  const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (i < (n + GATHER_PAGE - 1) / GATHER_PAGE) ids[i] = static_cast<int>(i);
  const int pc = static_cast<int>(i % pieces);
  const long long r = i / pieces;  // (key, head)
  const int h = static_cast<int>(r % Hkv);
  const long long key = r / Hkv;
  if (key >= n) return;
  const long long dst =
      ((key / GATHER_PAGE * Hkv + h) * GATHER_PAGE + key % GATHER_PAGE) * pieces + pc;
  const int pg = pages[key / page_size];
  if (pg < 0 || pg >= num_pages) {
    record_bad_index(err, W_PREFIX_PAGE);
    gk[dst] = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
    gv[dst] = make_uint4(0, 0, 0, 0);
    return;
  }
  const long long src = (pg * c_page + h * c_head + key % page_size * c_row) / 8 + pc;
  gk[dst] = k[src];
  gv[dst] = v[src];
}

template <class C>
void plan_cfg(int rows, int Hkv, int prefix_len, int sms, PagedPlan* pl) {
  const int tiles = (prefix_len + C::BC - 1) / C::BC;
  const double ctas = static_cast<double>(Hkv) * ((rows + C::BR * C::NQT - 1) / (C::BR * C::NQT));
  const double slots = static_cast<double>(sms) * C::MINB;
  // Key splits: the waves of CTAs times a CTA's key tiles, plus about three tiles' time to start and end a CTA,
  // plus the splits' states written and read (in units of a tile's time, 1.2 us).
  const double merge = static_cast<double>(rows) * Hkv * C::D * 8 / 4e6 / 1.2;
  double best = 0;
  for (int n = 1, last = 0; n <= 64 && n <= tiles; ++n) {
    const int per = (tiles + n - 1) / n, used = (tiles + per - 1) / per;
    if (used == last) continue;
    last = used;
    const double t = std::ceil(ctas * used / slots) * (per + 3) + used * merge;
    if (n == 1 || t < best) {
      best = t;
      pl->n_split = used;
      pl->kv_per_split = per * C::BC;
    }
  }
}

template <class C>
cudaError_t launch_cfg(const PagedLaunch& a, const PagedPlan& pl) {
  const int G = a.H / a.Hkv;
  FwdLaunch f = {};
  const void *kc = a.k_cache, *vc = a.v_cache;
  long long c_page = a.c_page, c_head = a.c_head, c_row = a.c_row;
  f.pages = a.prefix_pages;
  f.num_pages = a.num_pages;
  f.page_size = a.page_size;
  f.dependent = 1;
  if (box_rows_of(a.page_size, C::BC) < 8) {
    uint4* gk = reinterpret_cast<uint4*>(a.ws + pl.gather_k);
    uint4* gv = reinterpret_cast<uint4*>(a.ws + pl.gather_v);
    int* ids = reinterpret_cast<int*>(a.ws + pl.gather_pages);
    const int pieces = C::D / 8;
    const long long threads = static_cast<long long>(a.prefix_len) * a.Hkv * pieces;
    if (threads > 0x7FFFFFFFLL * 256) return cudaErrorInvalidValue;
    const cudaError_t e = launch_dependent(
        gather_prefix_kernel, dim3(static_cast<unsigned>((threads + 255) / 256)), 256, 0, a.stream,
        static_cast<const uint4*>(kc), static_cast<const uint4*>(vc), gk, gv, ids, a.prefix_pages, a.prefix_len, a.Hkv,
        pieces, a.num_pages, a.page_size, c_page, c_head, c_row, a.err);
    if (e != cudaSuccess) return e;
    kc = gk;
    vc = gv;
    f.pages = ids;
    f.num_pages = (a.prefix_len + GATHER_PAGE - 1) / GATHER_PAGE;
    f.page_size = GATHER_PAGE;
    c_row = C::D;
    c_head = GATHER_PAGE * C::D;
    c_page = c_head * a.Hkv;
  }
  f.box_rows = box_rows_of(f.page_size, C::BC);
  f.heads_inner = c_row > c_head;
  CUtensorMap tk, tv;
  cudaError_t e = encode_paged_map(&tk, kc, C::D, f.page_size, a.Hkv, f.num_pages, c_row, c_head, c_page, f.box_rows,
                                   f.heads_inner);
  if (e == cudaSuccess)
    e = encode_paged_map(&tv, vc, C::D, f.page_size, a.Hkv, f.num_pages, c_row, c_head, c_page, f.box_rows,
                         f.heads_inner);
  if (e != cudaSuccess) return e;
  f.tm_q = &tk;
  f.tm_k = &tk;
  f.tm_v = &tv;
  f.err = a.err;
  f.BH = a.Hkv;
  f.H = a.Hkv;
  f.Hkv = a.Hkv;
  f.Nq = a.B * G;
  f.Nk = a.prefix_len;
  f.kv_per_split = pl.kv_per_split;
  f.n_split = pl.n_split;
  f.ws_o = reinterpret_cast<float*>(a.ws + pl.pre_o);
  f.ws_ml = reinterpret_cast<float*>(a.ws + pl.pre_ml);
  f.c = a.c;
  f.tau = kPrefixTau;
  f.paged_q = a.q;
  f.G = G;
  f.stream = a.stream;
  return launch_fwd<C>(f);
}

}  // namespace

void plan_prefix(int B, int G, int Hkv, int d, int page_size, int prefix_len, int sms, PagedPlan* pl) {
  const int rows = B * G;
  pl->wide = rows > 128;
  if (d == 64)
    pl->wide ? plan_cfg<WideD64>(rows, Hkv, prefix_len, sms, pl) : plan_cfg<NarrowD64>(rows, Hkv, prefix_len, sms, pl);
  else
    pl->wide ? plan_cfg<WideD128>(rows, Hkv, prefix_len, sms, pl) : plan_cfg<NarrowD128>(rows, Hkv, prefix_len, sms, pl);
  if (box_rows_of(page_size, 64) < 8) {
    pl->gather_len = (prefix_len + GATHER_PAGE - 1) / GATHER_PAGE;
    pl->gather_rows = GATHER_PAGE;
  }
}

cudaError_t launch_prefix(const PagedLaunch& a, const PagedPlan& pl) {
  if (a.d == 64) return pl.wide ? launch_cfg<WideD64>(a, pl) : launch_cfg<NarrowD64>(a, pl);
  return pl.wide ? launch_cfg<WideD128>(a, pl) : launch_cfg<NarrowD128>(a, pl);
}

}  // namespace fa
