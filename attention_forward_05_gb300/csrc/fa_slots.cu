// fa_slots.cu -- a step's bookkeeping from its request lengths: the sequences' offsets among the new tokens, the tokens'
// positions and cache slots, page tables extended from the free pages.
//
// Sequence b has ctx_b tokens in the cache and n_b new ones.  Two prefix sums over the sequences give everything: of n_b
// (where a sequence's tokens begin) and of the pages it needs, ceil((ctx_b + n_b) / P) - ceil(ctx_b / P) (how far down the
// stack of free pages its own begin).  A token then finds its sequence by bisection and its slot by itself.
//
// One cluster of up to 16 CTAs.  Every CTA forms both sums over all sequences in its shared memory (12 bytes a sequence)
// and takes its pieces of the tokens, so no CTA waits for another's sums; the cluster's barrier stands between the last
// read of the lengths and the free pages' count and the writes of the new ones, which may go to the same memory.
// A few thousand bytes: bound by the launch and four dependent round trips to memory (237 sequences of a token: 3.9 us in a
// graph); with many tokens by the rate at which one SM writes (67961 tokens, 0.8 MB: 7.7 us; by clusters of 8 10.3).
#include "fa_internal.h"
#include "sm103_ptx.cuh"

namespace fa {

namespace {

constexpr int THREADS = 1024;
constexpr int MAX_CTAS = 16;  // of the cluster (above 8 it has to be asked for); one of the 8 processor clusters has 19 SMs at least
enum : int { W_STEP = 0x40 };  // site recorded with DEV_BAD_INDEX

// Exclusive prefix sums of the threads' values, and the total; `tmp` is shared, [THREADS / 32 + 1].
__device__ __forceinline__ long long block_scan(long long v, long long* tmp, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int i = 1; i < 32; i *= 2) {
    const long long y = __shfl_up_sync(0xffffffffu, x, i);
    if (lane >= i) x += y;
  }
  __syncthreads();  // tmp may still be read
  if (lane == 31) tmp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    const long long s = tmp[lane];
    long long y = s;
#pragma unroll
    for (int i = 1; i < 32; i *= 2) {
      const long long z = __shfl_up_sync(0xffffffffu, y, i);
      if (lane >= i) y += z;
    }
    tmp[lane] = y - s;
    if (lane == 31) tmp[32] = y;
  }
  __syncthreads();
  *total = tmp[32];
  return tmp[warp] + x - v;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

template <int RUN>
__global__ void __launch_bounds__(THREADS) fa_slots_kernel(const SlotsLaunch a, const FastDiv by_page, int ctas) {
  extern __shared__ int tables[];
  int* const s_start = tables;             // first token of each sequence (its new length until the first sum)
  int* const s_ctx = tables + a.B;
  int* const s_base = tables + 2 * a.B;    // free pages dealt before its own; -1: the sequence failed
  __shared__ long long tmp[THREADS / 32 + 1];
  __shared__ int s_taken, s_bad;
  const int tid = threadIdx.x, rank = blockIdx.x;
  griddep_wait();
  if (tid == 0) s_taken = s_bad = 0;
  int free_count = *a.free_count;
  for (int b = tid; b < a.B; b += THREADS) {
    s_ctx[b] = a.ctx_lens[b];
    s_start[b] = max(0, a.new_lens[b]);
  }
  if (free_count < 0 || free_count > a.n_free) free_count = -1;  // no page can be dealt
  __syncthreads();
  cluster_arrive();  // the inputs that outputs may lie in have been read
  const int per = (a.B + THREADS - 1) / THREADS, b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  const long long room = static_cast<long long>(a.max_pages) * a.page_size;
  const auto pages_of = [&](int n) { return n > 0 ? by_page.div(n - 1) + 1 : 0; };
  const auto fits = [&](int b, int n, long long end) {
    return s_ctx[b] >= 0 && end <= a.T && static_cast<long long>(s_ctx[b]) + n <= room;
  };
  long long total, deal_total, mine = 0;
  for (int b = b0; b < b1; ++b) mine += s_start[b];
  const long long start = block_scan(mine, tmp, &total);
  long long at = start;
  mine = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = s_start[b];
    at += n;
    if (n > 0 && fits(b, n, at)) mine += pages_of(s_ctx[b] + n) - pages_of(s_ctx[b]);
  }
  long long dealt = block_scan(mine, tmp, &deal_total);
  at = start;
  int taken = 0, bad = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = s_start[b], ctx = s_ctx[b];
    const int begin = static_cast<int>(min(at, static_cast<long long>(a.T)));
    at += n;
    int base = 0;
    if (n > 0) {
      bool ok = fits(b, n, at);
      if (ok) {
        const int need = pages_of(ctx + n) - pages_of(ctx);
        ok = need == 0 || dealt + need <= free_count;
        base = static_cast<int>(min(dealt, 0x7FFFFFFFLL));
        dealt += need;
        if (ok && need > 0) taken = static_cast<int>(dealt);
      }
      if (!ok) base = -1, bad = 1;
    }
    s_start[b] = begin;
    s_base[b] = base;
  }
  if (taken > 0) atomicMax(&s_taken, taken);
  if (bad) s_bad = 1;
  __syncthreads();
  cluster_wait();
  const int tokens = static_cast<int>(min(total, static_cast<long long>(a.T)));
  if (rank == 0) {
    for (int b = tid; b < a.B; b += THREADS) {
      const int n = max(0, (b + 1 < a.B ? s_start[b + 1] : tokens) - s_start[b]);
      a.cu_seqlens[b] = s_start[b];
      a.seq_lens[b] = s_base[b] < 0 ? -1 : s_ctx[b] + n;
    }
    if (tid == 0) {
      a.cu_seqlens[a.B] = tokens;
      *a.free_left = max(free_count, 0) - s_taken;
      if (s_bad || free_count < 0) record_bad_index(a.err, W_STEP);
    }
  }
  // The last sequence that begins at or before token t: those without tokens begin where the next one does.
  const auto sequence_of = [&](int t) {
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_start[mid] <= t) lo = mid;
      else hi = mid;
    }
    return lo;
  };
  // Page pi of sequence b, which has `held` already; a new one also goes into its table where `mine`.
  const auto page_of = [&](int b, int pi, int held, bool mine) {
    int* const entry = a.page_table + b * a.table_stride + pi;
    if (pi < held) return *entry;
    const int page = a.free_pages[free_count - 1 - (s_base[b] + pi - held)];
    if (mine) *entry = page;
    return page;
  };
  const auto slot_of = [&](int page, int row) { return page < 0 ? -1LL : static_cast<long long>(page) * a.page_size + row; };
  const auto one = [&](int t) {
    int pos = 0;
    long long slot = -1;
    if (t < tokens) {
      const int b = sequence_of(t);
      if (s_base[b] >= 0) {
        pos = s_ctx[b] + (t - s_start[b]);
        const int pi = by_page.div(pos), row = pos - pi * a.page_size;
        slot = slot_of(page_of(b, pi, pages_of(s_ctx[b]), row == 0), row);  // a page whose first row is a new token's is new
      }
    }
    a.positions[t] = pos;
    a.slots[t] = slot;
  };
  if (RUN == 1) {
    for (int t = rank * THREADS + tid; t < a.T; t += ctas * THREADS) one(t);
  } else {
    // RUN neighbouring tokens a thread: of one sequence, they lie in two pages at most.
    const bool wide =
        ((reinterpret_cast<unsigned long long>(a.positions) | reinterpret_cast<unsigned long long>(a.slots)) & 15) == 0;
    for (int t = (rank * THREADS + tid) * RUN; t < a.T; t += ctas * THREADS * RUN) {
      const int b = t < tokens ? sequence_of(t) : 0;
      const int end = t >= tokens ? 0 : b + 1 < a.B ? s_start[b + 1] : tokens;
      if (!wide || t + RUN > end || s_base[b] < 0) {
        for (int e = 0; e < RUN && t + e < a.T; ++e) one(t + e);
        continue;
      }
      const int pos = s_ctx[b] + (t - s_start[b]), pi = by_page.div(pos), row = pos - pi * a.page_size, held = pages_of(s_ctx[b]);
      const bool second = row + RUN > a.page_size;
      const int page0 = page_of(b, pi, held, row == 0), page1 = second ? page_of(b, pi + 1, held, true) : 0;
      long long slot[RUN];
#pragma unroll
      for (int e = 0; e < RUN; ++e)
        slot[e] = row + e < a.page_size ? slot_of(page0, row + e) : slot_of(page1, row + e - a.page_size);
#pragma unroll
      for (int e = 0; e < RUN; e += 4) {
        *reinterpret_cast<int4*>(a.positions + t + e) = make_int4(pos + e, pos + e + 1, pos + e + 2, pos + e + 3);
        reinterpret_cast<longlong2*>(a.slots + t + e)[0] = make_longlong2(slot[e], slot[e + 1]);
        reinterpret_cast<longlong2*>(a.slots + t + e)[1] = make_longlong2(slot[e + 2], slot[e + 3]);
      }
    }
  }
}

}  // namespace

template <int RUN>
static cudaError_t launch_run(const SlotsLaunch& a) {
  const int need = (a.T + RUN * THREADS - 1) / (RUN * THREADS), ctas = need < 1 ? 1 : need > MAX_CTAS ? MAX_CTAS : need;
  cudaError_t e = allow_shared_memory<fa_slots_kernel<RUN>>(12 * SLOTS_MAX_B);
  if (e == cudaSuccess && ctas > 8)
    e = cudaFuncSetAttribute(fa_slots_kernel<RUN>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  return launch_dependent_clusters(fa_slots_kernel<RUN>, static_cast<unsigned>(ctas), ctas, THREADS, 12 * a.B, a.stream, a,
                                   FastDiv(static_cast<unsigned>(a.page_size)), ctas);
}

// One token a thread as long as the cluster has threads for it; then four, whose pages are looked up once, where four rows lie
// in two pages at most.
cudaError_t launch_slots(const SlotsLaunch& a) {
  return a.T <= MAX_CTAS * THREADS || a.page_size < 4 ? launch_run<1>(a) : launch_run<4>(a);
}

}  // namespace fa
