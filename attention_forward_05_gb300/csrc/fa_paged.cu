// fa_paged.cu -- one query per head over a paged key/value cache (split-KV decode of a ragged batch).
//
// Sequence b sees len_b cache rows through its row of the page table: o = softmax(scale q K^T) V and the
// natural-log LSE, by the online-softmax recurrence in log2 units.  All G = H / Hkv query heads of a
// key/value head go through one pass over its keys, so each key and value is read from device memory once:
// the kernel is bound by those bytes.
//
// Products.  Both are computed transposed, by warp-level matrix instructions: S^T = K Q^T with 16 keys as the
// rows and 8 heads as the columns, O^T += V^T P^T with 16 dimensions as the rows.  Keys and values then fill the
// 16-row side, and a group of up to 8 heads wastes no product; S^T turns into the operand P^T by one transposing
// move a 16-key block.  (With the heads as the 16 rows a tile step took 630 instructions an 8 KB of K and V
// instead of about 200, and the issue slots, not the bytes, bound short contexts.)  A thread holds two heads'
// columns, so maxima, sums and rescaling are its own; the running maximum moves only when a score passes it by
// more than 2^PG_TAU.  The instruction takes both operands in one 16-bit type and V is bf16, so P goes in as two bf16
// terms (two_terms: together within 2^-15 of P), each multiplied with the same fragment of V; with P rounded to bf16
// alone o was up to 40 % further from the formula than its own rounding is.  The row sums add P itself, in fp32 like
// everything else.
//
// Work split.  A unit is one (sequence, group of query heads); its keys are cut into tiles of TILE (32 KB of K
// and V).  The tiles of all units, in order, are dealt evenly to the CTAs, one contiguous range each, whatever
// the lengths are (they stay in device memory; every CTA sums them itself).  A CTA's range covers whole units,
// which it finishes, and at most two parts of units at its ends, which it leaves as partial states (m, l,
// unnormalised O) for fa_paged_join_kernel.  (Ranges of single warps left four times as many parts to join:
// 28 instead of 21 us on one sequence of 32768 keys.)
//
// Where no sequence can be long (its table says how long), a unit has a cluster of 1 to 8 CTAs of its own instead
// (CLUSTER, cluster_size): nothing is planned, and the cluster joins its states through its shared memory, with the
// prefix's, so there is no join kernel behind it.
//
// Inside a CTA each warp takes its own KW keys of every tile through its own ring of asynchronous 16-byte
// copies, with no barrier between the warps until a unit ends; then their states merge in shared memory.  The
// lanes look up their keys' pages one step ahead.  Page sizes that are multiples of 16 rows copy 16 rows from
// one base address; others pass every row's offset around by shuffles.
//
// Measured, device time: 32 sequences of 32768 keys (d = 64, groups of 4) 305 to 308 us, 7.0 TB/s (floor 322 us at the copy's
// rate); 61 sequences of 0 to 32768 keys (d = 128, groups of 8) 69.7 us, 5.9 TB/s; one of 777 keys 5.6 us (8.0 by ranges).
#include <cuda_bf16.h>

#include "fa_internal.h"
#include "sm103_ptx.cuh"

namespace fa {

namespace {

enum : int { W_PAGE = 0x30, W_LEN };  // sites recorded with DEV_BAD_INDEX
constexpr float PG_TAU = 8.f;
// A unit's end (merging the warps' states, fetching the next queries) takes a CTA about as long as PG_END tiles:
// the ranges are cut as if every unit had that many tiles more.
constexpr int PG_END = 2;

template <int D_, int NT_>
struct PgCfg {
  static constexpr int D = D_;
  static constexpr int NT = NT_;                 // 8-column tiles of query heads
  static constexpr int GR = 8 * NT;              // query heads a unit holds
  static constexpr int NW = 4;
  static constexpr int KW = D == 128 ? 16 : 32;  // keys of one warp step: 8 KB of K and V
  static constexpr int TILE = NW * KW;
  static constexpr int CTAS = NT == 4 ? 2 : 3;   // per SM
  static constexpr int STAGES = NT == 4 ? 3 : 2;
  static constexpr int ROW_BYTES = D * 2;
  static constexpr int K_BYTES = KW * ROW_BYTES;
  static constexpr int STAGE_BYTES = 2 * K_BYTES;
  static constexpr int OFF_Q = NW * STAGES * STAGE_BYTES;
  static constexpr int OFF_ML = OFF_Q + GR * ROW_BYTES;         // float2 [NW][GR]
  static constexpr int OFF_PLAN = OFF_ML + NW * GR * 8;
  static constexpr int SMEM = OFF_PLAN + 64;
  static constexpr int FIT = STAGE_BYTES / (GR * D * 4) > 0 ? NT : STAGE_BYTES / (8 * D * 4);  // head tiles whose O fits a stage
  static_assert(NT % FIT == 0, "whole rounds");
  static_assert(SMEM * CTAS <= 227 * 1024 - CTAS * 1024, "shared memory");
};

struct PgParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* kc;
  const __nv_bfloat16* vc;
  __nv_bfloat16* o;
  float* lse;
  const int* table;
  const int* lens;
  long long c_page, c_head, c_row, table_stride;
  int B, H, Hkv, G, ngrp, U;      // U = Hkv * ngrp units a sequence
  int num_pages, page_size;
  FastDiv by_page;
  int runs16;                     // page_size is a multiple of 16
  int cap;                        // max_pages * page_size
  int n_cta;
  float c;
  int* err;
  float* part_ml;                 // float2 (m, l) [2 * n_cta][GR] of the CTAs' first (0) and last (1) unfinished units
  float* part_o;                  // [2 * n_cta][GR][D] unnormalised
  int2* infos;                    // [B * U]: slot of the unit's first part (-1: it has one, in unit_ml / unit_o), and its
                                  // parts (0: no own keys; -1: an unused place; -2: a bad length)
  // with a shared prefix every unit's own state stays a state, and the join adds the prefix's:
  int prefix;
  float* unit_ml;                 // float2 [B * H]: units that one CTA covers
  float* unit_o;                  // [B * H][D]
  const float* pre_ml;            // float2 [pre_split][Hkv][B * G]
  const float* pre_o;
  int pre_split;
  int cl;                         // CTAs of a unit in the form without ranges (CLUSTER); 0: the other one
};

// Tiles of sequence b: 0 for a sequence without keys or with a length past its table.
template <int TILE>
__device__ __forceinline__ int seq_tiles(const PgParams& p, int b, int* len) {
  const int n = p.lens[b];
  *len = n;
  return n <= 0 || n > p.cap ? 0 : (n + TILE - 1) / TILE;
}

// CTAs that share `total` tiles, the first tile of CTA c, and the CTA of tile t.
__device__ __forceinline__ long long cta_count(long long total, int n_cta) { return total < n_cta ? total : n_cta; }
__device__ __forceinline__ long long cta_first(long long c, long long total, long long n) { return c * total / n; }
__device__ __forceinline__ long long cta_of(long long t, long long total, long long n) {
  return ((t + 1) * n - 1) / total;
}

// ---- thread-block clusters

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// The shared-memory address `addr` of this CTA in CTA `rank` of its cluster.
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, int rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}
__device__ __forceinline__ float2 load_peer8(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 load_peer16(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// A place in a CTA's range: tile `tile` of unit (b, u), at position v of the range.
template <class C>
struct Cursor {
  int b, u, tile, nt, len, v;
  __device__ __forceinline__ void next(const PgParams& p) {
    ++v;
    if (++tile < nt) return;
    v += PG_END;
    tile = 0;
    if (++u < p.U) return;
    u = 0;
    do {
      if (++b >= p.B) {  // past the last unit, and so past every range
        v = 0x7fffffff;
        return;
      }
      nt = seq_tiles<C::TILE>(p, b, &len);
    } while (nt == 0);
  }
};

// (M, L, acc) += states (x, v), by the online-softmax recurrence.  An empty state is (-inf, 0, 0); a state of NaN keys
// (-inf, NaN, NaN).
template <int W>
__device__ __forceinline__ void add_states(const float2 (&x)[W], const float4 (&v)[W], float& M, float& L, float4& acc) {
  float m_new = M;
#pragma unroll
  for (int i = 0; i < W; ++i) m_new = fmaxf(m_new, x[i].x);
  const float ref = m_new == -INFINITY ? 0.f : m_new;
  const float alpha = ex2_approx(M - ref);
  M = m_new;
  L *= alpha;
  acc.x *= alpha, acc.y *= alpha, acc.z *= alpha, acc.w *= alpha;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const float w = ex2_approx(x[i].x - ref);
    L = fmaf(x[i].y, w, L);
    acc.x = fmaf(v[i].x, w, acc.x);
    acc.y = fmaf(v[i].y, w, acc.y);
    acc.z = fmaf(v[i].z, w, acc.z);
    acc.w = fmaf(v[i].w, w, acc.w);
  }
}

// The end of the form in which a unit has a cluster of its own: joins the states of the cluster's CTAs, which lie in their
// shared memory, and those of the prefix, and writes the unit's outputs.  The output's 16-byte pieces are dealt to the
// CTAs; inside one, groups of threads take every (number of groups)-th state, eight in flight, and are added up in order.
template <class C, typename RowOf>
__device__ __forceinline__ void join_cluster(const PgParams& p, int b, int len, int rows, int hk, int g0, long long head0,
                                             int rank, uint8_t* smem, RowOf state_row) {
  constexpr int D = C::D, THREADS = 32 * C::NW, W = 8;
  if (p.cl > 1) cluster_sync();
  if (p.prefix) griddep_wait();
  const bool bad = len > p.cap, none = bad || len < 0 || (len == 0 && !p.prefix);
  if (bad && rank == 0 && threadIdx.x == 0) record_bad_index(p.err, W_LEN);
  const int pieces = rows * (D / 4), share = (pieces + p.cl - 1) / p.cl;
  const int wide = share >= THREADS ? THREADS : 1 << (32 - __clz(share - 1));  // pieces side by side
  const int groups = THREADS / wide, grp = threadIdx.x / wide, at = threadIdx.x % wide;
  const int pre = p.prefix ? p.pre_split : 0, parts = none ? 0 : pre + p.cl;
  const long long pstep = static_cast<long long>(p.B) * p.H;
  const uint32_t base = smem_u32(smem);
  float4* const sum_o = reinterpret_cast<float4*>(smem);  // the warps' own states, done with
  float2* const sum_ml = reinterpret_cast<float2*>(smem + THREADS * 16);
  for (int e0 = 0; e0 < share; e0 += wide) {
    const int e = rank * share + e0 + at;
    const bool mine = e0 + at < share && e < pieces;
    const int row = e / (D / 4), pc = e % (D / 4);
    const long long prow = (static_cast<long long>(hk) * p.B + b) * p.G + g0 + row;
    float M = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = grp; mine && s0 < parts; s0 += W * groups) {
      float2 x[W];
      float4 v[W];
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const int s = s0 + i * groups;
        x[i] = make_float2(-INFINITY, 0.f);
        v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (s < pre) {
          x[i] = reinterpret_cast<const float2*>(p.pre_ml)[s * pstep + prow];
          v[i] = reinterpret_cast<const float4*>(p.pre_o + (s * pstep + prow) * D)[pc];
        } else if (s < parts) {
          x[i] = load_peer8(peer_addr(base + C::OFF_Q + row * 8, s - pre));
          v[i] = load_peer16(peer_addr(base + state_row(row) + pc * 16, s - pre));
        }
      }
      add_states(x, v, M, L, acc);
    }
    if (groups > 1) {
      sum_o[threadIdx.x] = acc;
      sum_ml[threadIdx.x] = make_float2(M, L);
      __syncthreads();
      if (grp == 0) {
        M = -INFINITY;
        L = 0.f;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int g = 0; g < groups; g += 4) {  // a power of two; two groups are padded with empty states
          float2 x[4];
          float4 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool in = g + i < groups;
            x[i] = in ? sum_ml[(g + i) * wide + at] : make_float2(-INFINITY, 0.f);
            v[i] = in ? sum_o[(g + i) * wide + at] : make_float4(0.f, 0.f, 0.f, 0.f);
          }
          add_states(x, v, M, L, acc);
        }
      }
    }
    if (mine && grp == 0) {
      const float nan = __int_as_float(0x7fc00000), inv = bad ? nan : none ? 0.f : 1.f / L;
      *reinterpret_cast<uint2*>(p.o + (head0 + row) * D + pc * 4) =
          make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
      if (p.lse != nullptr && pc == 0)
        p.lse[head0 + row] = bad ? nan : none ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
    }
  }
  if (p.cl > 1) cluster_sync();  // a CTA's shared memory is there while others read it
}

}  // namespace

template <class C, bool CLUSTER>
__global__ void __launch_bounds__(32 * C::NW, C::CTAS) fa_paged_kernel(const PgParams p) {
  extern __shared__ __align__(256) uint8_t smem[];  // pieces are found by xor on address bits 4 to 7
  constexpr int D = C::D, KW = C::KW, NW = C::NW, S = C::STAGES;
  constexpr int CPR = D / 8;        // 16-byte pieces of a row
  constexpr int RPP = 32 / CPR;     // rows one warp-wide copy covers
  constexpr int NP = KW / RPP;      // copies of K (and of V) a step
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_launch_dependents();
  // After the prefix's kernel, which waited for everything before it and whose states this kernel does not read, it
  // may run beside that kernel; each CTA then waits at its end, so that this grid's completion implies that one's.
  if (!p.prefix) griddep_wait();

  auto leave = [&]() {
    if (p.prefix) griddep_wait();
  };
  Cursor<C> cur;
  int range;
  long long t0 = 0, total = 0, n = 0;
  const int rank = CLUSTER ? static_cast<int>(blockIdx.x) % p.cl : 0;
  if constexpr (CLUSTER) {  // the unit's CTAs share its tiles evenly; some may have none
    const int unit = static_cast<int>(blockIdx.x) / p.cl;
    cur.b = unit / p.U;
    cur.u = unit - cur.b * p.U;
    cur.nt = seq_tiles<C::TILE>(p, cur.b, &cur.len);
    cur.tile = cur.nt * rank / p.cl;
    cur.v = 0;
    range = cur.nt * (rank + 1) / p.cl - cur.tile;
  } else {
    // ---- plan: total tiles, this CTA's range, the unit it starts in
    long long* plan = reinterpret_cast<long long*>(smem + C::OFF_PLAN);  // [0..3] warp sums, [4] tiles before, [5] b
    const int per = (p.B + 32 * NW - 1) / (32 * NW);
    const int b_lo = min(p.B, static_cast<int>(threadIdx.x) * per), b_hi = min(p.B, b_lo + per);
    long long mine = 0;
    int len_tmp;
    for (int b = b_lo; b < b_hi; ++b) {
      const int nt = seq_tiles<C::TILE>(p, b, &len_tmp);
      if (nt > 0) mine += nt + PG_END;
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) plan[warp] = incl;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (w < warp) incl += plan[w];
      total += plan[w];
    }
    total *= p.U;
    // outputs of sequences without keys, and of those whose length passes their table
    for (int b = blockIdx.x; b < p.B; b += p.n_cta) {
      int len;
      if (seq_tiles<C::TILE>(p, b, &len) > 0) continue;
      const bool bad = len > 0;
      if (bad && threadIdx.x == 0) record_bad_index(p.err, W_LEN);
      for (int u = threadIdx.x; u < p.U; u += 32 * NW)
        p.infos[static_cast<long long>(b) * p.U + u] = make_int2(-1, bad ? -2 : len < 0 ? -1 : 0);
      if (p.prefix) continue;  // the join writes their outputs
      const long long row0 = static_cast<long long>(b) * p.H;
      for (int e = threadIdx.x; e < p.H * CPR; e += 32 * NW)
        reinterpret_cast<uint4*>(p.o + row0 * D)[e] = bad ? make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu)
                                                          : make_uint4(0, 0, 0, 0);
      if (p.lse != nullptr)
        for (int h = threadIdx.x; h < p.H; h += 32 * NW) p.lse[row0 + h] = bad ? __int_as_float(0x7fc00000) : -INFINITY;
    }
    n = cta_count(total, p.n_cta);
    if (static_cast<long long>(blockIdx.x) >= n) return leave();  // the whole CTA (n = 0 without keys)
    t0 = cta_first(blockIdx.x, total, n);
    const long long t1 = cta_first(blockIdx.x + 1, total, n);
    {
      long long before = (incl - mine) * p.U;
      if (t0 >= before && t0 < incl * p.U) {
        for (int b = b_lo;; ++b) {
          const int tiles = seq_tiles<C::TILE>(p, b, &len_tmp);
          const long long nt = tiles > 0 ? static_cast<long long>(tiles + PG_END) * p.U : 0;
          if (t0 < before + nt) {
            plan[4] = before;
            plan[5] = b;
            break;
          }
          before += nt;
        }
      }
    }
    __syncthreads();
    cur.b = static_cast<int>(plan[5]);
    cur.nt = seq_tiles<C::TILE>(p, cur.b, &cur.len);
    cur.u = static_cast<int>((t0 - plan[4]) / (cur.nt + PG_END));
    cur.tile = static_cast<int>((t0 - plan[4]) % (cur.nt + PG_END));
    cur.v = 0;
    range = static_cast<int>(t1 - t0);
    if (cur.tile >= cur.nt) {  // the range begins behind a unit's last tile
      cur.v = cur.nt - 1 - cur.tile;
      cur.tile = cur.nt - 1;
      cur.next(p);
    }
    if (cur.v >= range) return leave();  // no tile of its own (the whole CTA)
  }

  // ---- loads: `ld` is the step whose pages are being looked up; lane r holds the page of key r of its KW
  const uint32_t ring = smem_u32(smem) + warp * S * C::STAGE_BYTES;
  Cursor<C> ld = cur;
  int ld_stage = 0;
  const int r_l = lane % KW, piece = lane % CPR;
  const long long lane_off = static_cast<long long>(lane / CPR) * p.c_row + piece * 8;
  const long long pass_off = RPP * p.c_row;
  // piece `piece` of row r of a stage lies at r * ROW_BYTES + ((piece ^ (r & 7)) << 4); pass i has r = i * RPP + lane / CPR
  const uint32_t dst_lane = ring + lane / CPR * C::ROW_BYTES + ((piece ^ (lane / CPR)) << 4);
  int pid = 0;
  auto lookup = [&]() {
    const int key = ld.tile * C::TILE + warp * KW + r_l;
    if (ld.v < range && key < ld.len) pid = p.table[ld.b * p.table_stride + p.by_page.div(key)];
  };
  auto load_step = [&]() {  // copies of step ld into ring stage ld_stage, then the next step's lookup
    if (ld.v < range) {
      const int key = ld.tile * C::TILE + warp * KW + r_l;
      const bool good = pid >= 0 && pid < p.num_pages;
      long long off = pid * p.c_page + (p.ngrp == 1 ? ld.u : ld.u / p.ngrp) * p.c_head +
                      (key - p.by_page.div(key) * p.page_size) * p.c_row;
      const uint32_t dst0 = dst_lane + ld_stage * C::STAGE_BYTES;
      if (p.runs16 && __all_sync(0xffffffffu, key < ld.len && good)) {
#pragma unroll
        for (int h = 0; h < KW / 16; ++h) {
          const long long base = __shfl_sync(0xffffffffu, off, 16 * h) + lane_off;
          const __nv_bfloat16 *kp = p.kc + base, *vp = p.vc + base;
#pragma unroll
          for (int j = 0; j < 16 / RPP; ++j) {
            const int i = h * (16 / RPP) + j;
            const uint32_t dst = (dst0 ^ ((i * RPP & 7) << 4)) + i * RPP * C::ROW_BYTES;
            cp_async16(dst, kp);
            cp_async16(dst + C::K_BYTES, vp);
            kp += pass_off;
            vp += pass_off;
          }
        }
      } else {
        if (key >= ld.len) {
          off = -1;  // zeros
        } else if (!good) {
          off = -2;  // a NaN key: the sequence's outputs become NaN
          record_bad_index(p.err, W_PAGE);
        }
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const long long ro = __shfl_sync(0xffffffffu, off, i * RPP + lane / CPR);
          const uint32_t dst = (dst0 ^ ((i * RPP & 7) << 4)) + i * RPP * C::ROW_BYTES;
          const long long src = ro < 0 ? 0 : ro + piece * 8;
          if (ro == -2 && piece == 0)
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst), "r"(0x7fff7fffu) : "memory");
          else
            cp_async16(dst, p.kc + src, ro < 0 ? 0 : 16);
          cp_async16(dst + C::K_BYTES, p.vc + src, ro < 0 ? 0 : 16);
        }
      }
      if constexpr (CLUSTER)
        ++ld.v, ++ld.tile;
      else
        ld.next(p);
      lookup();
    }
    cp_async_commit();
    ld_stage = ld_stage + 1 == S ? 0 : ld_stage + 1;
  };
  lookup();

  // ---- queries: fetched into registers, handed over through shared memory (sign flipped for a negative scale, so
  // that the largest score is the largest product)
  uint8_t* sq = smem + C::OFF_Q;
  constexpr int QN = (C::GR * CPR + 32 * NW - 1) / (32 * NW);  // 16-byte pieces of Q a thread carries
  uint4 qv[QN];
  const float c = fmaxf(fabsf(p.c), 1e-30f);  // a zero scale: every score 0, without 0 * inf in masked places
  const uint32_t flip = p.c < 0.f ? 0x80008000u : 0u;
  auto fetch_q = [&](int b, int u) {
    const int g0 = u % p.ngrp * C::GR, rows = min(C::GR, p.G - g0);
    const __nv_bfloat16* src = p.q + (static_cast<long long>(b) * p.H + u / p.ngrp * p.G + g0) * D;
#pragma unroll
    for (int i = 0; i < QN; ++i) {
      const int e = i * 32 * NW + threadIdx.x;
      qv[i] = e / CPR < rows ? reinterpret_cast<const uint4*>(src)[e] : make_uint4(flip, flip, flip, flip);
    }
  };
  auto store_q = [&]() {
#pragma unroll
    for (int i = 0; i < QN; ++i) {
      const int e = i * 32 * NW + threadIdx.x, row = e / CPR;
      if (row < C::GR)
        *reinterpret_cast<uint4*>(sq + row * C::ROW_BYTES + ((e % CPR ^ (row & 7)) << 4)) =
            make_uint4(qv[i].x ^ flip, qv[i].y ^ flip, qv[i].z ^ flip, qv[i].w ^ flip);
    }
  };
  fetch_q(cur.b, cur.u);
#pragma unroll
  for (int i = 0; i < S - 1; ++i) load_step();
  store_q();
  __syncthreads();

  // ---- fragments (mat, l7: the 8x8 matrix and its row whose address a lane gives)
  const int l7 = lane & 7, mat = lane >> 3, gid = lane >> 2, tig = lane & 3;
  const uint32_t q_addr = smem_u32(sq) + l7 * C::ROW_BYTES + ((mat ^ l7) << 4);   // B: heads l7, two k steps' halves
  const uint32_t k_lane = ring + ((mat & 1) * 8 + l7) * C::ROW_BYTES + (((mat >> 1) ^ l7) << 4);                // A: keys, k halves
  const uint32_t v_lane = ring + C::K_BYTES + ((mat >> 1) * 8 + l7) * C::ROW_BYTES + (((mat & 1) ^ l7) << 4);  // A: dims, keys
  uint32_t qf[C::NT][D / 32][4];  // [head tile][two k steps]: B fragments (b0, b1) of the one, then of the other
  auto load_qf = [&]() {
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
      for (int k2 = 0; k2 < D / 32; ++k2) ldmatrix_x4((q_addr ^ (k2 << 6)) + nt * 8 * C::ROW_BYTES, qf[nt][k2]);
  };
  load_qf();
  float o[C::NT][D / 16][4];       // O^T: dims 16 dp + gid (+ 8) x heads 2 tig, 2 tig + 1
  float m_ref[C::NT][2], l[C::NT][2];
  auto reset = [&]() {
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt) {
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][j][e] = 0.f;
      m_ref[nt][0] = m_ref[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }
  };
  reset();
  bool first_unit = true;
  int stage = 0;

  while (true) {
    const int seg_tile0 = cur.tile;  // first tile of the unit that this CTA covers
    const int tiles = min(cur.nt - cur.tile, range - cur.v);
    for (int i = 0; !CLUSTER || i < tiles; ++i) {
      load_step();  // into the stage of the step before this one
      cp_async_wait<S - 1>();
      __syncwarp();
      const int valid = cur.len - ((seg_tile0 + i) * C::TILE + warp * KW);
      const uint32_t ks0 = k_lane + stage * C::STAGE_BYTES, vs0 = v_lane + stage * C::STAGE_BYTES;
      if (valid > 0) {
        float s[C::NT][KW / 16][4];  // S^T: keys 16 kb + gid (+ 8) x heads 2 tig, 2 tig + 1
#pragma unroll
        for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
          for (int kb = 0; kb < KW / 16; ++kb)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nt][kb][e] = 0.f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
          for (int kb = 0; kb < KW / 16; ++kb) {
            uint32_t a[4];
            ldmatrix_x4((ks0 ^ (ks << 5)) + kb * 16 * C::ROW_BYTES, a);
#pragma unroll
            for (int nt = 0; nt < C::NT; ++nt)
              mma_16816(s[nt][kb], a, qf[nt][ks / 2][ks % 2 * 2], qf[nt][ks / 2][ks % 2 * 2 + 1]);
          }
        if (valid < KW) {
#pragma unroll
          for (int kb = 0; kb < KW / 16; ++kb)
#pragma unroll
            for (int r = 0; r < 2; ++r)
              if (kb * 16 + r * 8 + gid >= valid)
#pragma unroll
                for (int nt = 0; nt < C::NT; ++nt) s[nt][kb][2 * r] = s[nt][kb][2 * r + 1] = -INFINITY;
        }
        uint32_t pf[C::NT][KW / 16][2], pr[C::NT][KW / 16][2];  // P^T's two terms: B operands of V^T P^T
#pragma unroll
        for (int nt = 0; nt < C::NT; ++nt) {
          float mx[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            mx[x] = fmaxf(s[nt][0][x], s[nt][0][2 + x]);
#pragma unroll
            for (int kb = 1; kb < KW / 16; ++kb) mx[x] = max3f(mx[x], s[nt][kb][x], s[nt][kb][2 + x]);
            mx[x] *= c;
          }
          if (__any_sync(0xffffffffu, mx[0] > m_ref[nt][0] + PG_TAU || mx[1] > m_ref[nt][1] + PG_TAU)) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
              for (int off = 4; off < 32; off <<= 1) mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], off));
              if (mx[x] > m_ref[nt][x] + PG_TAU) {
                const float alpha = ex2_approx(m_ref[nt][x] - mx[x]);  // 0 on the first keys
                m_ref[nt][x] = mx[x];
                l[nt][x] *= alpha;
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                  o[nt][j][x] *= alpha;
                  o[nt][j][2 + x] *= alpha;
                }
              }
            }
          }
          const float n0 = m_ref[nt][0] == -INFINITY ? 0.f : -m_ref[nt][0];
          const float n1 = m_ref[nt][1] == -INFINITY ? 0.f : -m_ref[nt][1];
#pragma unroll
          for (int kb = 0; kb < KW / 16; ++kb) {
            const float p0 = ex2_approx(fmaf(s[nt][kb][0], c, n0)), p1 = ex2_approx(fmaf(s[nt][kb][1], c, n1));
            const float p2 = ex2_approx(fmaf(s[nt][kb][2], c, n0)), p3 = ex2_approx(fmaf(s[nt][kb][3], c, n1));
            l[nt][0] += p0 + p2;
            l[nt][1] += p1 + p3;
            uint32_t h0, h1, r0, r1;
            two_terms(p0, p1, h0, r0);
            two_terms(p2, p3, h1, r1);
            pf[nt][kb][0] = movmatrix_trans(h0);
            pf[nt][kb][1] = movmatrix_trans(h1);
            pr[nt][kb][0] = movmatrix_trans(r0);
            pr[nt][kb][1] = movmatrix_trans(r1);
          }
        }
#pragma unroll
        for (int kb = 0; kb < KW / 16; ++kb)
#pragma unroll
          for (int dp = 0; dp < D / 16; ++dp) {
            uint32_t a[4];
            ldmatrix_x4_trans((vs0 ^ (dp << 5)) + kb * 16 * C::ROW_BYTES, a);
#pragma unroll
            for (int nt = 0; nt < C::NT; ++nt) {
              mma_16816(o[nt][dp], a, pf[nt][kb][0], pf[nt][kb][1]);
              mma_16816(o[nt][dp], a, pr[nt][kb][0], pr[nt][kb][1]);
            }
          }
      }
      __syncwarp();  // every lane has read the stage
      if (i + 1 == tiles) break;
      stage = stage + 1 == S ? 0 : stage + 1;
    }

    // ---- the unit's part in this CTA ends: merge the warps' states
    if (CLUSTER) stage = 0;  // nothing is in flight; the merged state's place is the same in every CTA
    Cursor<C> nx = cur;
    bool more = false, whole = false;
    if constexpr (!CLUSTER) {
      cur.tile += tiles - 1;
      cur.v += tiles - 1;
      nx = cur;
      nx.next(p);
      more = nx.v < range;
      if (more) fetch_q(nx.b, nx.u);  // in flight during the merge
      whole = seg_tile0 == 0 && cur.tile + 1 == cur.nt;
    }
    const int slot = 2 * blockIdx.x + (first_unit ? 0 : 1);
    const int hk = cur.u / p.ngrp, g0 = cur.u % p.ngrp * C::GR;
    const int rows = min(C::GR, p.G - g0);
    const long long head0 = static_cast<long long>(cur.b) * p.H + hk * p.G + g0;
    float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
    // CLUSTER: row r of the merged state is in the second stage of warp r / (rows that fit)
    auto state_row = [&](int r) {
      constexpr int FITS = C::STAGE_BYTES / (D * 4);
      return (r / FITS * S + 1) * C::STAGE_BYTES + r % FITS * (D * 4);
    };
    auto stage_of = [&](int w) { return reinterpret_cast<float*>(smem + (w * S + stage) * C::STAGE_BYTES); };
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt) {
      // Every warp leaves (m, l) and its O in its own stage, row by head, 8-element runs swapped by the head pair so that
      // a store's 32 elements use all banks; then each thread adds up one 16-byte piece over the warps.
      float* const mine_o = stage_of(warp) + nt % C::FIT * 8 * D;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float sum = l[nt][x];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (gid == 0) ml[warp * C::GR + nt * 8 + 2 * tig + x] = make_float2(m_ref[nt][x], sum);
        float* dst = mine_o + (2 * tig + x) * D + gid;
#pragma unroll
        for (int dp = 0; dp < D / 16; ++dp) {
          dst[16 * dp ^ (tig << 3)] = o[nt][dp][x];
          dst[(16 * dp + 8) ^ (tig << 3)] = o[nt][dp][2 + x];
        }
      }
      if (nt % C::FIT != C::FIT - 1) continue;
      __syncthreads();
      const int row_lo = (nt + 1 - C::FIT) * 8, row_hi = min(rows, (nt + 1) * 8);
      for (int e = threadIdx.x; e < (row_hi - row_lo) * (D / 4); e += 32 * NW) {
        const int row = e / (D / 4), pc = e % (D / 4), grow = row_lo + row;
        float2 x[NW];
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          x[w] = ml[w * C::GR + grow];
          M = fmaxf(M, x[w].x);
        }
        const float ref = M == -INFINITY ? 0.f : M;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < NW; ++w) {  // an empty state is (-inf, 0, 0); a state of NaN keys (-inf, NaN, NaN)
          const float wt = ex2_approx(x[w].x - ref);
          L = fmaf(x[w].y, wt, L);
          const float4 y = *reinterpret_cast<const float4*>(stage_of(w) + row * D + ((4 * pc) ^ ((row >> 1 & 3) << 3)));
          acc.x = fmaf(y.x, wt, acc.x);
          acc.y = fmaf(y.y, wt, acc.y);
          acc.z = fmaf(y.z, wt, acc.z);
          acc.w = fmaf(y.w, wt, acc.w);
        }
        if constexpr (CLUSTER) {
          *reinterpret_cast<float4*>(smem + state_row(grow) + pc * 16) = acc;
          if (pc == 0) reinterpret_cast<float2*>(smem + C::OFF_Q)[grow] = make_float2(M, L);
        } else if (whole && !p.prefix) {
          const float inv = 1.f / L;
          *reinterpret_cast<uint2*>(p.o + (head0 + grow) * D + pc * 4) =
              make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
          if (p.lse != nullptr && pc == 0) p.lse[head0 + grow] = (M + log2f(L)) * 0.6931471805599453f;
        } else {
          const long long at = whole ? head0 + grow : static_cast<long long>(slot) * C::GR + grow;
          *reinterpret_cast<float4*>((whole ? p.unit_o : p.part_o) + at * D + pc * 4) = acc;
          if (pc == 0) reinterpret_cast<float2*>(whole ? p.unit_ml : p.part_ml)[at] = make_float2(M, L);
        }
      }
      if (nt == C::NT - 1) {
        if (!CLUSTER && seg_tile0 == 0 && threadIdx.x == 0) {  // begun here: what will be found where
          const long long last = t0 + cur.v - cur.tile + cur.nt - 1;
          p.infos[static_cast<long long>(cur.b) * p.U + cur.u] =
              make_int2(whole ? -1 : slot, static_cast<int>(cta_of(last, total, n) - blockIdx.x + 1));
        }
        if (more) store_q();  // every warp is past its products with the unit's queries
      }
      __syncthreads();
    }
    if constexpr (CLUSTER) {
      join_cluster<C>(p, cur.b, cur.len, rows, hk, g0, head0, rank, smem, state_row);
      return;
    }
    if (!more) break;
    first_unit = false;
    load_qf();
    reset();
    cur = nx;
    stage = stage + 1 == S ? 0 : stage + 1;
  }
  cp_async_wait<0>();
  leave();
}

// Joins the parts of units that several CTAs share, and with a shared prefix the prefix's states and every
// sequence's own, and writes the outputs.  A team of WPR warps takes every (number of teams)-th (sequence, query
// head): its warps take every WPR-th state, eight states' rows in flight, with the online-softmax recurrence, and add
// up in warp order.  Bound by latency, a handful of dependent loads, so WPR goes with the states a row is likely to
// have (join_warps).  (It does not let the next kernel start early: CTAs of the next call's fa_paged_kernel placed
// between these were spread unevenly over the SMs, and its time on 32 sequences of 32768 keys went from 304 to 325 us.)
template <int D, int GR, int WPR>
__global__ void __launch_bounds__(WPR == 1 ? 128 : 32 * WPR) fa_paged_join_kernel(const PgParams p) {
  constexpr int E = D / 32, TEAMS = WPR == 1 ? 4 : 1;
  __shared__ float sm_o[WPR][D];
  __shared__ float2 sm_ml[WPR];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % WPR;  // the warp's place in its team
  const long long heads = static_cast<long long>(p.B) * p.H;
  const long long team = static_cast<long long>(blockIdx.x) * TEAMS + (threadIdx.x >> 5) / WPR;
  const long long teams = static_cast<long long>(gridDim.x) * TEAMS;
  const float nan = __int_as_float(0x7fc00000);
  for (long long k0 = team; k0 < heads; k0 += 32 * teams) {
    // this team's next 32 rows: what there is to do for each
    const long long mine = k0 + lane * teams;
    int2 info = make_int2(-1, 1);
    if (mine < heads) {
      const int h = static_cast<int>(mine % p.H);
      info = p.infos[mine / p.H * p.U + h / p.G * p.ngrp + h % p.G / GR];
    }
    unsigned todo = __ballot_sync(0xffffffffu, mine < heads && (p.prefix || info.y > 1));
    while (todo != 0) {
      const int k = __ffs(todo) - 1;
      todo &= todo - 1;
      const long long head = k0 + k * teams;
      const int slot = __shfl_sync(0xffffffffu, info.x, k), own = __shfl_sync(0xffffffffu, info.y, k);
      const int b = static_cast<int>(head / p.H), h = static_cast<int>(head - static_cast<long long>(b) * p.H);
      const int hk = h / p.G, g = h - hk * p.G;
      const long long pstep = heads;
      const long long prow = (static_cast<long long>(hk) * p.B + b) * p.G + g;
      const int pre = own < 0 ? 0 : p.pre_split;
      const int parts = own < 0 ? 0 : pre + own;
      float M = -INFINITY, L = 0.f, acc[E];
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = 0.f;
      for (int s0 = warp; s0 < parts; s0 += 8 * WPR) {
        float2 x[8];
        float v[8][E];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int s = s0 + i * WPR;
          x[i] = make_float2(-INFINITY, 0.f);
#pragma unroll
          for (int e = 0; e < E; ++e) v[i][e] = 0.f;
          if (s >= parts) continue;
          const float2* ml;
          const float* o;
          if (s < pre) {
            ml = reinterpret_cast<const float2*>(p.pre_ml) + s * pstep + prow;
            o = p.pre_o + (s * pstep + prow) * D;
          } else if (slot < 0) {
            ml = reinterpret_cast<const float2*>(p.unit_ml) + head;
            o = p.unit_o + head * D;
          } else {  // the first part's slot, then slot 0 of the CTAs after that one
            const long long at = static_cast<long long>(s == pre ? slot : 2 * (slot / 2 + s - pre)) * GR + g % GR;
            ml = reinterpret_cast<const float2*>(p.part_ml) + at;
            o = p.part_o + at * D;
          }
          x[i] = *ml;
          if constexpr (E == 4) {
            const float4 y = *reinterpret_cast<const float4*>(o + lane * E);
            v[i][0] = y.x, v[i][1] = y.y, v[i][2] = y.z, v[i][3] = y.w;
          } else {
            const float2 y = *reinterpret_cast<const float2*>(o + lane * E);
            v[i][0] = y.x, v[i][1] = y.y;
          }
        }
        float m_new = M;
#pragma unroll
        for (int i = 0; i < 8; ++i) m_new = fmaxf(m_new, x[i].x);
        const float ref = m_new == -INFINITY ? 0.f : m_new;
        const float alpha = ex2_approx(M - ref);
        M = m_new;
        L *= alpha;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] *= alpha;
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // an empty state is (-inf, 0, 0); a state of NaN keys (-inf, NaN, NaN)
          const float w = ex2_approx(x[i].x - ref);
          L = fmaf(x[i].y, w, L);
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] = fmaf(v[i][e], w, acc[e]);
        }
      }
      if constexpr (WPR > 1) {
#pragma unroll
        for (int e = 0; e < E; ++e) sm_o[warp][lane * E + e] = acc[e];
        if (lane == 0) sm_ml[warp] = make_float2(M, L);
        __syncthreads();
        M = -INFINITY;
#pragma unroll
        for (int w = 0; w < WPR; ++w) M = fmaxf(M, sm_ml[w].x);
        const float ref = M == -INFINITY ? 0.f : M;
        L = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
        for (int w = 0; w < WPR; ++w) {
          const float wt = ex2_approx(sm_ml[w].x - ref);
          L = fmaf(sm_ml[w].y, wt, L);
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] = fmaf(sm_o[w][lane * E + e], wt, acc[e]);
        }
        __syncthreads();
      }
      if (warp == 0) {
        const float inv = own == -2 ? nan : parts == 0 ? 0.f : 1.f / L;
        uint32_t* out = reinterpret_cast<uint32_t*>(p.o + head * D) + lane * (E / 2);
#pragma unroll
        for (int e = 0; e < E; e += 2) out[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
        if (p.lse != nullptr && lane == 0)
          p.lse[head] = own == -2 ? nan : parts == 0 ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
      }
    }
  }
}

namespace {

constexpr size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// CTAs of a unit in the form where every unit has a cluster of its own, or 0 for even ranges of tiles.  `tiles`: of the
// longest sequence that its table can hold; n_cta: CTAs that may run at once.  As many as there is room for, less the
// places that clusters of this size leave free in each of the GPU's 8 processor clusters (3000 keys in 56 clusters of 8:
// 16.0 us, of 7: 9.9); behind a prefix, whose CTAs want room too, a power of two and two CTAs a SM (96 units in clusters
// of 3: 14.0 us, of 2: 11.0).  A CTA takes about 0.45 us a tile, so at eight tiles a CTA the launch and the join that the clusters save (2 to
// 4 us) are used up, whatever the real lengths are; behind a prefix, whose states are joined too, at sixteen.  Clusters
// against ranges, device time at 32 heads on 8 of 128: 1 sequence of 2000 keys 6.1 and 8.1 us, 4000: 8.2 and 9.2, 8000:
// 12.1 and 10.2; 16 of 300: 6.1 and 8.9, 1500: 14.4 and 14.1; 48 of 400: 9.3 and 13.1; 100 of 400: 29.7 and 32.4; behind a
// prefix 48 of 60: 17.3 and 24.6, 64 of 800: 48 and 56, 64 of 1 to 1500: 34.1 and 33.6.  Where the units are a little more than
// the CTAs that may run at once, sequences that fill their tables leave the second wave nearly empty, others do not (512
// units of 384 keys: 16.9 and 15.1; of 1 to 384: 11.5 and 13.2); the lengths are not known here.
// Many units of one or two tiles, without a prefix, are left to the ranges: a unit's start and end are most of its time, and
// a CTA of a range fetches the next unit's keys meanwhile.  Clusters and ranges: 32 heads on 8 of 128, 456 sequences of 64
// keys 36 and 30 us, of 128 46 and 49, of 1 to 128 38 and 34, of 192 61 and 66, of 1 to 192 43 and 41; 300 of 64 20.2 and
// 20.0, of 128 32 and 35; 32 on 8 of 64, 600 of 128 45 and 35, of 256 60 and 57.
int cluster_size(long long units, long long tiles, int n_cta, int sms, bool prefix) {
  if (!prefix && tiles <= 2 && units > 6LL * n_cta) return 0;
  const long long most = tiles > 2 ? (tiles < 8 ? tiles : 8) : 1;
  long long cl = 1;
  if (prefix)
    while (cl * 2 <= 8 && cl < most && units * cl <= sms) cl *= 2;
  else
    while (cl < most && units * (cl + 1) <= n_cta - 8 * cl) ++cl;
  return tiles <= (prefix ? 16 : 8) * cl && units * cl <= 0x7FFFFFFF ? static_cast<int>(cl) : 0;
}

template <class C>
PagedPlan plan_of(int B, int H, int Hkv, int page_size, int max_pages, int prefix_len, int sms) {
  PagedPlan pl;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += round256(bytes);
    return here;
  };
  pl.n_cta = sms * C::CTAS;
  const long long groups = (H / Hkv + C::GR - 1) / C::GR, cap = static_cast<long long>(max_pages) * page_size;
  if (max_pages > 0)
    pl.cl = cluster_size(groups * B * Hkv, (cap + C::TILE - 1) / C::TILE, pl.n_cta, sms, prefix_len > 0);
  const size_t slots = static_cast<size_t>(2) * pl.n_cta, heads = static_cast<size_t>(B) * H;
  pl.part_ml = take(slots * C::GR * 8);
  pl.part_o = take(slots * C::GR * C::D * 4);
  pl.infos = take(static_cast<size_t>(B) * Hkv * groups * 8);
  if (prefix_len > 0) {
    const int G = H / Hkv;
    plan_prefix(B, G, Hkv, C::D, page_size, prefix_len, sms, &pl);
    pl.pre_ml = take(heads * pl.n_split * 8);
    pl.pre_o = take(heads * pl.n_split * C::D * 4);
    pl.unit_ml = take(heads * 8);
    pl.unit_o = take(heads * C::D * 4);
    const size_t rows = static_cast<size_t>(pl.gather_len) * pl.gather_rows * Hkv;
    pl.gather_k = take(rows * C::D * 2);
    pl.gather_v = take(rows * C::D * 2);
    pl.gather_pages = take(static_cast<size_t>(pl.gather_len) * 4);
  }
  pl.total = at;
  return pl;
}

// Warps that join a row's states, at eight states a warp in flight.  A unit has about n_cta / units + 1 own parts and
// at most one a tile (the lengths, and so the parts, are not known here), and the prefix's splits.  One warp a row where
// that is at most eight and the rows alone fill the GPU (2048 rows of 64 equal sequences: 28 instead of 32 us with
// four), four otherwise, because a ragged batch's longest sequence has many more (320 rows: 17 instead of 20 us with
// one); sixteen for a few rows of very many states (one sequence of 32768 keys: 19 instead of 20 us with four).
int join_warps(long long units, long long heads, long long tiles, const PagedPlan& pl, int sms) {
  const long long share = pl.n_cta / units, parts = (share < tiles ? share : tiles) + 1 + pl.n_split;
  if (parts > 32 && heads <= sms) return 16;
  return parts > 8 || heads <= 8LL * sms ? 4 : 1;
}

template <class C>
cudaError_t launch_paged(const PagedLaunch& a, const PagedPlan& pl) {
  PgParams p = {};
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.kc = static_cast<const __nv_bfloat16*>(a.k_cache);
  p.vc = static_cast<const __nv_bfloat16*>(a.v_cache);
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.lse = a.lse;
  p.table = a.table;
  p.lens = a.lens;
  p.c_page = a.c_page;
  p.c_head = a.c_head;
  p.c_row = a.c_row;
  p.table_stride = a.table_stride;
  p.B = a.B;
  p.H = a.H;
  p.Hkv = a.Hkv;
  p.G = a.H / a.Hkv;
  p.ngrp = (p.G + C::GR - 1) / C::GR;
  p.U = a.Hkv * p.ngrp;
  p.num_pages = a.num_pages;
  p.page_size = a.page_size;
  p.runs16 = a.page_size % 16 == 0;
  p.by_page = FastDiv(static_cast<unsigned>(a.page_size));
  p.cap = a.max_pages * a.page_size;
  p.n_cta = pl.n_cta;
  p.c = a.c;
  p.err = a.err;
  p.part_ml = reinterpret_cast<float*>(a.ws + pl.part_ml);
  p.part_o = reinterpret_cast<float*>(a.ws + pl.part_o);
  p.infos = reinterpret_cast<int2*>(a.ws + pl.infos);
  const long long units = static_cast<long long>(a.B) * p.U;
  p.cl = pl.cl;
  cudaError_t e = p.cl > 0 ? allow_shared_memory<fa_paged_kernel<C, true>>(C::SMEM)
                           : allow_shared_memory<fa_paged_kernel<C, false>>(C::SMEM);
  if (e != cudaSuccess) return e;
  if (a.prefix_len > 0) {
    p.prefix = 1;
    p.unit_ml = reinterpret_cast<float*>(a.ws + pl.unit_ml);
    p.unit_o = reinterpret_cast<float*>(a.ws + pl.unit_o);
    p.pre_ml = reinterpret_cast<const float*>(a.ws + pl.pre_ml);
    p.pre_o = reinterpret_cast<const float*>(a.ws + pl.pre_o);
    p.pre_split = pl.n_split;
    if ((e = launch_prefix(a, pl)) != cudaSuccess) return e;
  }
  // programmatic dependents: a launch overlaps the end of the kernel before it
  if (p.cl > 0)
    return launch_dependent_clusters(fa_paged_kernel<C, true>, static_cast<unsigned>(units * p.cl), p.cl, 32 * C::NW, C::SMEM,
                                     a.stream, p);
  if ((e = launch_dependent(fa_paged_kernel<C, false>, pl.n_cta, 32 * C::NW, C::SMEM, a.stream, p)) != cudaSuccess) return e;
  const long long heads = static_cast<long long>(a.B) * a.H, most = static_cast<long long>(a.sms) * 16;
  const unsigned rows = static_cast<unsigned>(heads < most ? heads : most);
  switch (join_warps(units, heads, p.cap / C::TILE + 1, pl, a.sms)) {
    case 16: return launch_dependent(fa_paged_join_kernel<C::D, C::GR, 16>, rows, 512, 0, a.stream, p);
    case 4: return launch_dependent(fa_paged_join_kernel<C::D, C::GR, 4>, rows, 128, 0, a.stream, p);
    default: {
      const long long ctas = (heads + 3) / 4;
      return launch_dependent(fa_paged_join_kernel<C::D, C::GR, 1>, static_cast<unsigned>(ctas < most ? ctas : most), 128, 0,
                              a.stream, p);
    }
  }
}

// Query heads a unit holds: 8, 16 or 32, whichever the group fits.  Larger groups take several units of 32, which read K and V
// again: 32 sequences of 8192 keys, 32 heads on each of 4 of 128 take 108 us, 64 heads 205.
template <typename F>
auto with_config(int G, int d, F&& f) {
  if (d == 64) return G <= 8 ? f(PgCfg<64, 1>{}) : G <= 16 ? f(PgCfg<64, 2>{}) : f(PgCfg<64, 4>{});
  return G <= 8 ? f(PgCfg<128, 1>{}) : G <= 16 ? f(PgCfg<128, 2>{}) : f(PgCfg<128, 4>{});
}

}  // namespace

PagedPlan paged_plan(int B, int H, int Hkv, int d, int page_size, int max_pages, int prefix_len, int sms) {
  return with_config(H / Hkv, d,
                     [&](auto c) { return plan_of<decltype(c)>(B, H, Hkv, page_size, max_pages, prefix_len, sms); });
}

cudaError_t launch_decode_paged(const PagedLaunch& a, const PagedPlan& pl) {
  return with_config(a.H / a.Hkv, a.d, [&](auto c) { return launch_paged<decltype(c)>(a, pl); });
}

}  // namespace fa
