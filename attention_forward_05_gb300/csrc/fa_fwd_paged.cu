// fa_fwd_paged.cu -- attention of a ragged batch's new tokens over a paged key/value cache.
//
// Token i of sequence b's n_b new ones stands at position p = len_b - n_b + i and sees the keys 0 .. p, or with a sliding
// window w the keys p - w + 1 .. p and the first `sinks` ones: o = softmax(scale q K^T) V over those, and the LSE.
//
// Products.  The rows of a tile are the (token, head of the group) pairs of one key/value head, so a key is read and
// multiplied once for the whole group.  A block is two tiles of up to 128 rows (whole tokens); its keys come in tiles of BC.
// The pipeline is the forward kernel's (fa_fwd_kernel.cuh): S = Q K^T and O += P V on tcgen05 with S, P and O in tensor
// memory, a softmax warpgroup a tile with a thread a row, P over S, O rescaled only when a maximum moves by more than 2^tau.
// P is rounded to bf16 for P V, as there (the sums add P itself).  In two terms, as the paged decode has it, P V takes two
// products: 8191 tokens, 32 heads on 8 of 128, 487 us instead of 354, single tokens behind windows of 4096 97 instead of 75.  One
// puts o up to 40 % further from the formula than o's own rounding does (relative RMS error 0.0019 to 0.0023, in two terms 0.0017);
// fa_decode_paged has single tokens without that.
//
// The CTAs stay (one a SM at d = 128, two at 64) and walk through units of work; the load warp runs ahead into the next
// unit, and its first Q K^T is issued while the last one's epilogue is still writing.
//
// Work split.  A unit is (key/value head, block): its keys cut into tiles.  The tiles of all units, in order, are dealt
// evenly to the CTAs, one contiguous range each, whatever the lengths are (they stay in device memory; every CTA sums them
// itself, 3.5 us).  A range covers whole units, which the CTA finishes, and at most two parts of units at its ends, whose states
// (m, l, unnormalised O) it leaves in the workspace; fa_fwd_paged_join_kernel joins those in the order of the keys.  Where
// ranges of whole units are hardly longer, no unit is cut (256 units of 19 tiles, d = 64: 34 us, cut into 304 ranges 44).
//
// Small calls are not dealt (CLUSTER, cluster_size): where the units, then of one row tile, are few and short enough, each has a
// cluster of 1 to 16 CTAs, two an SM, with even shares of its tiles, and the cluster joins its states through its shared memory.
//
// No atomics on results: a token's depend on its sequence's queries and keys, the lengths, the call's sizes and the SM count alone.
//
// Keys and values come out of the pages by TMA boxes of as many rows as divide the page size (8 at least: a swizzle
// period), or, where no such box exists, by 16-byte asynchronous copies.  Keys that no row of the block sees are not read
// (their pages may be gone); their values are zeros.  A value that some rows see and others do not may be infinite or NaN,
// and 0 * inf would reach the others: the load warp sets such values aside (zeros in their place), and the epilogue
// adds them to the rows that see them.
//
// What bounds it, measured (one pass among others): prompts the matrix products: 8191 tokens, 32 heads on 8 of 128, 355 us, 1546
// TFLOP/s of the formula's products (the dense causal forward 348 us, 1580), in rows of its own under the power cap 375 to 385
// (dense 363).  At d = 64 the exponentials' latency, as in the dense forward: 37 sequences of up to 512 tokens over up to 8192
// keys, 32 heads on 4, 79 us, 700 TFLOP/s with start, ends and masked tiles.  Few tokens over long contexts device memory: 24
// sequences of 3 to 7 tokens, 1.41 GB, 220 us, 6.4 TB/s.  Small calls latency: 23 tokens behind 1000 keys 9.2 us (dealt 13.2: 3
// for the plan, 3 to the first scores, 3 to the states, 4 for the join).
#include <cuda_bf16.h>

#include <algorithm>

#include "fa_fwd_kernel.cuh"

namespace fa {

namespace {

enum : int { W_OFFSETS = 0x48, W_LENGTH, W_PAGE, W_DESC, W_DESC_FREE, W_QFREE };  // sites recorded

constexpr float kTau = 32.f;  // fa_api.cu, kLazyTau

constexpr int MAX_CLUSTER = 16;  // above 8 it has to be asked for

// CLUSTER: no dealing, each unit has a cluster of CTAs.  Its units have one row tile, so with key tiles of 64 at d = 128 too two
// CTAs fit on an SM.
template <int D_, bool GATHER_, bool CLUSTER_, int BC_>
struct ChunkCfg {
  static constexpr int D = D_;
  static constexpr bool GATHER = GATHER_, CLUSTER = CLUSTER_;
  static constexpr int BC = BC_;
  static constexpr int STAGES = D == 128 ? 2 : 4;
  static constexpr int MINB = BC == 128 ? 1 : 2;  // CTAs per SM
  static constexpr bool PV2 = BC == 128;          // P handed over in two halves (FwdCfg)
  static constexpr int BR = 128, TILES = CLUSTER ? 1 : 2;  // rows of a tile, row tiles of a block
  static constexpr int NCH = D / 64;             // 128-byte segments of a row
  static constexpr int Q_CH_BYTES = BR * 128, KV_CH_BYTES = BC * 128;
  static constexpr int Q_BYTES = NCH * Q_CH_BYTES, KV_BYTES = NCH * KV_CH_BYTES;
  static constexpr int OFF_Q = 0, OFF_K = TILES * Q_BYTES, OFF_V = OFF_K + STAGES * KV_BYTES, OFF_BAR = OFF_V + STAGES * KV_BYTES;
  static constexpr int UNITS = 4;                // units announced at a time
  static constexpr int NBAR = 4 * STAGES + 2 * UNITS + 12;
  static constexpr int OFF_UNITS = OFF_BAR + NBAR * 8;
  static constexpr int OUT_COLS = D == 128 ? 32 : 16;  // columns of the outputs that a softmax warp has on their way at a time
  static constexpr int STAGE_BYTES = 32 * OUT_COLS * 2;
  static constexpr int OFF_STAGE = OFF_UNITS + UNITS * 64;
  static constexpr int OFF_MISC = OFF_STAGE + 4 * TILES * STAGE_BYTES;
  static constexpr int SMEM_BYTES = OFF_MISC + 160 + (32 * 11 + 2) * 8 + 1024;  // plan's scratch; slack to align the base to 1024
  static constexpr int OFF_STATE = OFF_K, OFF_ML = OFF_Q;  // CLUSTER: the rows' O, and m and l, once all products are done
  static constexpr int O_COL0 = TILES * BC;      // TMEM: S_t at t * BC, O_t at O_COL0 + t * D
  static constexpr int TMEM_COLS = TILES * (BC + D) <= 128 ? 128 : TILES * (BC + D) <= 256 ? 256 : 512;
  // The values have a load warp of their own at d = 128 (FwdCfg::SPLIT_LOADS); it comes free of registers there.
  static constexpr int LOAD_WARP = 4 * TILES, MMA_WARP = LOAD_WARP + 1, LOADV_WARP = D == 128 ? LOAD_WARP + 2 : LOAD_WARP;
  static constexpr int NWARPS = LOAD_WARP + (D == 128 ? 3 : 2), NTHREADS = 32 * NWARPS;
  static constexpr int CONSUMERS = NWARPS - 1;   // warps that read the announced units
  static constexpr int WARPS_PER_SUBPART = (NWARPS * MINB + 3) / 4;
  static constexpr int MAXREG = WARPS_PER_SUBPART <= 2 ? 248 : (16384 / (WARPS_PER_SUBPART * 32)) / 8 * 8;
  static_assert(TILES * (BC + D) <= TMEM_COLS && TMEM_COLS * MINB <= 512, "tensor memory");
  static_assert(SMEM_BYTES * MINB <= 227 * 1024, "shared memory");
  static_assert(BR * D * 4 <= 2 * STAGES * KV_BYTES, "a cluster's states lie where keys and values were");
  static_assert((FWD_PAGED_MAX_B + 1) * 4 <= OFF_BAR, "the plan's block counts lie where the tiles will");
};

template <int D, bool GATHER>
using Ranges = ChunkCfg<D, GATHER, false, D>;
template <int D, bool GATHER, int BC = 64>
using Cluster = ChunkCfg<D, GATHER, true, BC>;

// The dealing counts key tiles.  A unit's start and end take about as long as this many of them, whether it has one row tile or
// two (a step of one is bound by its chain of products and exponentials, or by the tile's bytes).  A prompt of 8191 tokens,
// d = 128, with 2, 3, 4: 371, 357, 362 us; a mixed batch, d = 64: 88, 83, 79.
constexpr int cost_unit(int d) { return d == 128 ? 3 : 4; }

// Cutting units costs their states, written and read again, and a start and an end more: so no unit is cut where the
// longest range of whole units is at most this much longer than an even share.
constexpr int COST_CUT = 6;

struct ChunkParams {
  __nv_bfloat16* o;
  float* lse;
  const __nv_bfloat16* k;  // the caches, for copies of single rows
  const __nv_bfloat16* v;
  long long c_page, c_head, c_row;
  const int* table;
  const int* cu;
  const int* lens;
  long long table_stride;
  int* err;
  float4* part_o;    // [CTA][continued, begun][row tile][D / 4][part_rows]
  float2* part_ml;   // [CTA][continued, begun][row tile][part_rows]
  struct Shared* shared;  // [CTA]
  FastDiv by_g, by_page, by_block;
  int T, B, H, Hkv, G, tile_tokens, part_rows, part_tiles;
  int cl;  // CTAs of a unit, where each unit has a cluster
  int num_pages, page_size, max_pages, box_rows, heads_inner;
  int window, sinks;
  float c, tau, p_lim;
};

// What the join has to know of a unit that several CTAs share: the one that this CTA begins, or else the one whose middle it has.
struct __align__(16) Shared {
  int first, parts;  // the CTA that begins it, and how many have a part; parts 0: this CTA shares none
  int h, q0, ntok;
};

// Key tiles before place w of a unit that begins at `start` and takes `extra` tiles' time besides its tiles.
__device__ __forceinline__ int cut(long long w, long long start, int tiles, int extra) {
  const long long x = w - start - extra;
  return x <= 0 ? 0 : x >= tiles ? tiles : static_cast<int>(x);
}
// a / b of numbers >= 0, which are nearly always short.
__device__ __forceinline__ long long divide(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<unsigned>(a) / static_cast<unsigned>(b);
  return static_cast<long long>(static_cast<unsigned long long>(a) / static_cast<unsigned long long>(b));
}
__device__ __forceinline__ long long range_begin(long long total, int c, int ranges) { return divide(total * c, ranges); }
// The range that place w lies in.
__device__ __forceinline__ int range_of(long long total, int ranges, long long w) {
  return static_cast<int>(divide((w + 1) * ranges - 1, total));
}

// A sequence's new tokens, as far as its offsets and length make sense.
struct __align__(16) Seq {
  int q0, n, pos0;  // first row of q, tokens, the first one's position
  bool bad;         // its length does not fit: its tokens become NaN
};
__device__ __forceinline__ Seq load_seq(const ChunkParams& p, int b) {
  Seq s{0, 0, 0, false};
  if (b >= p.B) return s;
  const int from = p.cu[b], to = p.cu[b + 1], len = p.lens[b];
  if (from < 0 || to < from || to > p.T) return s;
  s.q0 = from;
  s.n = to - from;
  s.bad = s.n > 0 && (len < s.n || len > static_cast<long long>(p.max_pages) * p.page_size);
  s.pos0 = s.bad ? 0 : len - s.n;
  return s;
}

// Keys of a block of tokens at positions pos0 .. pos0 + ntok - 1, as tiles: the sinks' ones, then those from the window's
// first on.
struct Span {
  int lo, hi;         // keys that the window shows to some token: lo .. hi - 1
  int ns, w0, tiles;  // tiles 0 .. ns - 1, then w0 ..; how many in all
};
template <int BC>
__device__ __forceinline__ Span span_of(const ChunkParams& p, int pos0, int ntok) {
  Span s;
  s.hi = pos0 + ntok;
  s.lo = p.window > 0 ? max(0, pos0 - p.window + 1) : 0;
  s.w0 = s.lo / BC;
  s.ns = min(p.sinks / BC + (p.sinks % BC != 0), s.w0);
  s.tiles = s.ns + (s.hi + BC - 1) / BC - s.w0;
  return s;
}
// Key tiles of a sequence's i-th block; a bad sequence's block counts as one.
template <int BC>
__device__ __forceinline__ int block_tiles(const ChunkParams& p, const Seq& s, int i) {
  if (s.bad) return 1;
  const int first = i * 2 * p.tile_tokens;
  return span_of<BC>(p, s.pos0 + first, min(2 * p.tile_tokens, s.n - first)).tiles;
}

// A unit as the load warp announces it.
enum : int { UNIT_WHOLE = 0, UNIT_BEGUN = 1, UNIT_CONTINUED = 2, UNIT_BAD = 3, UNIT_NONE = 4 };
struct __align__(16) Unit {
  int kind, h, b, q0;
  int ntok, pos0, jb, je;  // tiles jb .. je - 1 of the block's
  int ns, w0, lo, hi;
  int bad_page, set_aside;  // set while its tiles are loaded
  int pad[2];
};
static_assert(sizeof(Unit) == 64, "OFF_MISC");

__device__ __forceinline__ int key_tile(const Unit& u, int j) { return j < u.ns ? j : u.w0 + j - u.ns; }

// Steps of row tile t in this part: it needs no tiles past its own last token.
template <int BC>
__device__ __forceinline__ int steps_of(const volatile Unit& u, int t, int tile_tokens) {
  if (t * tile_tokens >= u.ntok || u.kind >= UNIT_BAD) return 0;
  const int hi = u.pos0 + min((t + 1) * tile_tokens, u.ntok);
  return max(0, min(u.je, u.ns + (hi + BC - 1) / BC - u.w0) - u.jb);
}

// Bits of columns 0 .. n - 1.
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }

// Nonzero halves' sign bits where a bf16 is infinite or NaN.
__device__ __forceinline__ uint32_t not_finite(uint32_t w) { return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }

__device__ __forceinline__ int blocks_of(const ChunkParams& p, int n) { return n > 0 ? p.by_block.div(n - 1) + 1 : 0; }

// The last of 0 .. n - 1 that is 0 or below(i), which holds up to some i.  As many steps for every thread.
template <typename F>
__device__ __forceinline__ int last_below(int n, F below) {
  int at = 0;
  for (int step = n > 1 ? 1 << (31 - __clz(n - 1)) : 0; step > 0; step >>= 1)
    if (at + step < n && below(at + step)) at += step;
  return at;
}

// The last sequence that begins at or before block x: those without blocks begin where the next one does.
__device__ __forceinline__ int seq_of_block(const int* nblk, int B, int x) {
  return last_below(B, [&](int b) { return nblk[b] <= x; });
}

// Exclusive prefix sums of the threads' values, and their total.
template <int NT, typename T>
__device__ __forceinline__ T scan(T v, T* tmp, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int i = 1; i < 32; i *= 2) {
    const T y = __shfl_up_sync(0xffffffffu, x, i);
    if (lane >= i) x += y;
  }
  __syncthreads();  // tmp may still be read
  if (lane == 31) tmp[warp] = x;
  __syncthreads();
  T before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    const T t = tmp[w];
    if (w < warp) before += t;
    all += t;
  }
  *total = all;
  return before + x - v;
}

// Adds the values set aside (infinities, NaN) of the keys that the token at `pos` sees to its row of O, whose element e lies at
// o + e / run * stride + e % run, or with SWAP, stride the row, in 16-byte pieces swapped by it: rare, so it reads back what the
// epilogue has just written.
template <class C, bool SWAP, typename T>
__device__ __noinline__ void add_aside(const ChunkParams& p, const volatile Unit& u, int pos, T* o, int run, long long stride) {
  const int last_lo = p.window > 0 ? max(0, u.pos0 + u.ntok - p.window) : 0;
  for (int j = u.jb; j < u.je; ++j) {
    const int key0 = (j < u.ns ? j : u.w0 + j - u.ns) * C::BC;
    if (key0 + C::BC <= u.pos0 + 1 && key0 >= last_lo) continue;
    for (int key = key0; key < min(key0 + C::BC, u.hi); ++key) {
      if (key <= u.pos0 && key >= last_lo) continue;  // every row sees it: left in the products
      if (key > pos || (p.window > 0 && key <= pos - p.window && key >= p.sinks)) continue;
      const int pi = p.by_page.div(key), pg = p.table[u.b * p.table_stride + pi];
      if (pg < 0 || pg >= p.num_pages) continue;
      const __nv_bfloat16* const v = p.v + pg * p.c_page + u.h * p.c_head + (key - pi * p.page_size) * p.c_row;
      for (int e = 0; e < C::D; ++e) {
        const float x = __bfloat162float(v[e]);
        if (!(fabsf(x) < INFINITY)) {
          T& y = SWAP ? o[((e / 4) ^ (static_cast<int>(stride) & (C::D / 4 - 1))) * 4 + e % 4] : o[e / run * stride + e % run];
          y = static_cast<T>(static_cast<float>(y) + x);
        }
      }
    }
  }
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

// Joins a unit's states, which lie in its cluster's shared memory; a CTA has every cl-th row, a thread four columns of one, four
// states on their way.  (Slices of the rows pushed to the CTAs that join them by bulk copies instead: 23 tokens behind 1000 keys
// 1.3 us more; eight states at a time, or two rows a thread, 0.1 and 0.4 us.)
template <class C>
__device__ __forceinline__ void join_cluster(const ChunkParams& p, const Unit& u, uint32_t sbase) {
  constexpr int PCS = C::D / 4, PER = C::NTHREADS / PCS, N = 4;
  const int rows = u.ntok * p.G, pc = threadIdx.x % PCS;
  if (threadIdx.x >= PER * PCS) return;
  for (int row = threadIdx.x / PCS * p.cl + blockIdx.x; row < rows; row += PER * p.cl) {
    float m = -INFINITY, l = 0.f, o[4] = {};
    for (int c0 = 0; c0 < p.cl; c0 += N) {
      float2 ml[N];
      float4 x[N];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        ml[k] = make_float2(-INFINITY, 0.f);
        x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c0 + k < p.cl) {
          const int c = c0 + k + blockIdx.x;  // from its own on, so that not all read the same one
          const uint32_t peer = peer_addr(sbase, c < p.cl ? c : c - p.cl);
          ml[k] = load_peer8(peer + C::OFF_ML + row * 8);
          x[k] = load_peer16(peer + C::OFF_STATE + row * (C::D * 4) + ((pc ^ (row & (PCS - 1))) << 4));
        }
      }
      float m_new = m;
#pragma unroll
      for (int k = 0; k < N; ++k) m_new = fmaxf(m_new, ml[k].x);
      const float m_use = m_new == -INFINITY ? 0.f : m_new;  // no part so far sees a key of this row: weights of 0
      const float old = ex2_approx(m - m_use);
      l *= old;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] *= old;
      m = m_new;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const float w = ex2_approx(ml[k].x - m_use);
        l = fmaf(w, ml[k].y, l);
        o[0] = fmaf(w, x[k].x, o[0]);
        o[1] = fmaf(w, x[k].y, o[1]);
        o[2] = fmaf(w, x[k].z, o[2]);
        o[3] = fmaf(w, x[k].w, o[3]);
      }
    }
    const int tok = p.by_g.div(row), g = row - tok * p.G;
    const float inv = 1.f / l;
    const size_t out = static_cast<size_t>(u.q0 + tok) * p.H + u.h * p.G + g;
    *reinterpret_cast<uint2*>(p.o + out * C::D + pc * 4) =
        make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
    if (p.lse != nullptr && pc == 0) p.lse[out] = (m + log2f(l)) * 0.6931471805599453f;
  }
}

// CLUSTER: a cluster's CTAs take even shares of its unit's tiles; the grid is the cluster's CTAs, key/value heads, blocks.
template <class C>
__global__ void __maxnreg__(C::MAXREG)
    fa_fwd_paged_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const ChunkParams p) {
  constexpr int D = C::D, BC = C::BC, STAGES = C::STAGES;
  constexpr bool CLUSTER = C::CLUSTER;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (sbase - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;

  const uint32_t bar0 = sbase + C::OFF_BAR;
  const auto bar_kf = [&](int s) { return bar0 + 8u * s; };
  const auto bar_vf = [&](int s) { return bar0 + 8u * (STAGES + s); };
  const auto bar_ke = [&](int s) { return bar0 + 8u * (2 * STAGES + s); };
  const auto bar_ve = [&](int s) { return bar0 + 8u * (3 * STAGES + s); };
  const auto bar_uf = [&](int i) { return bar0 + 8u * (4 * STAGES + i); };             // unit announced
  const auto bar_ue = [&](int i) { return bar0 + 8u * (4 * STAGES + C::UNITS + i); };  // and read by all
  const uint32_t bar1 = bar0 + 8u * (4 * STAGES + 2 * C::UNITS);
  const uint32_t bar_q = bar1, bar_qe = bar1 + 8, bar_tail = bar1 + 16, bar_drain = bar1 + 24;
  const auto bar_sf = [&](int t) { return bar1 + 8u * (4 + t); };
  const auto bar_ph = [&](int t) { return bar1 + 8u * (6 + t); };
  const auto bar_pf = [&](int t) { return bar1 + 8u * (8 + t); };
  const auto bar_od = [&](int t) { return bar1 + 8u * (10 + t); };
  Unit* const units = reinterpret_cast<Unit*>(smem + C::OFF_UNITS);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  int* const plan_start = reinterpret_cast<int*>(smem + C::OFF_MISC + 8);             // head, block, ranges, extra, whole, sequence
  long long* const plan_at = reinterpret_cast<long long*>(smem + C::OFF_MISC + 32);   // start, total, range
  Seq* const plan_seq = reinterpret_cast<Seq*>(plan_at);                              // CLUSTER: the unit's
  int* const plan_tmp = reinterpret_cast<int*>(smem + C::OFF_MISC + 64);              // 12 64-bit numbers
  long long* const plan_place = reinterpret_cast<long long*>(smem + C::OFF_MISC + 160);

  griddep_launch_dependents();
  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(bar_kf(s), 1);
      mbar_init(bar_vf(s), 1);
      mbar_init(bar_ke(s), 1);
      mbar_init(bar_ve(s), 1);
    }
    for (int i = 0; i < C::UNITS; ++i) {
      mbar_init(bar_uf(i), 1);
      mbar_init(bar_ue(i), C::CONSUMERS);
    }
    mbar_init(bar_q, 1);
    mbar_init(bar_qe, 1);
    mbar_init(bar_tail, 1);
    mbar_init(bar_drain, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar_sf(t), 1);
      mbar_init(bar_ph(t), 4);  // one arrive per softmax warp of the tile
      mbar_init(bar_pf(t), 4);
      mbar_init(bar_od(t), 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == C::LOAD_WARP) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      if (!C::GATHER) {
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
      }
    }
  }
  griddep_wait();

  // ---------------------------------------------------------------- plan: this CTA's range of all units' tiles
  {
    constexpr int NT = C::NTHREADS;
    const auto report = [&](int b, const Seq& s) {
      if (blockIdx.x > 0) return;
      if (s.n == 0 && (p.cu[b] < 0 || p.cu[b] != p.cu[b + 1] || p.cu[b] > p.T)) record_bad_index(p.err, W_OFFSETS);
      if (s.bad) record_bad_index(p.err, W_LENGTH);
    };
    if (CLUSTER && p.B <= 32) {  // one warp finds the unit, a lane a sequence
      if (warp == C::LOAD_WARP) {
        const Seq s = load_seq(p, lane);
        if (lane < p.B) report(lane, s);
        const int nb = blocks_of(p, s.n), x = blockIdx.z;
        int upto = nb;
#pragma unroll
        for (int i = 1; i < 32; i *= 2) {
          const int y = __shfl_up_sync(0xffffffffu, upto, i);
          if (lane >= i) upto += y;
        }
        const bool here = x < upto && x >= upto - nb;
        const bool any = __any_sync(0xffffffffu, here);
        if (here) {
          plan_start[0] = blockIdx.y;
          plan_start[1] = x - (upto - nb);
          plan_start[5] = lane;
          *plan_seq = s;
        }
        if (lane == 0) {
          plan_start[2] = any;
          units[0].ntok = 0;
        }
      }
    } else {
      // Where the tiles will lie: blocks before each sequence, then the sequences, if they fit.
      int* const nblk = reinterpret_cast<int*>(smem);
      Seq* const seqs = reinterpret_cast<Seq*>(smem + (4 * p.B + 4 + 15) / 16 * 16);
      const bool kept = p.B <= C::OFF_BAR / 20 - 2;
      const auto seq_at = [&](int b) { return kept && b < p.B ? seqs[b] : load_seq(p, b); };
      const int per = (p.B + NT - 1) / NT, b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
      int mine = 0;
      for (int b = b0; b < b1; ++b) {
        const Seq s = load_seq(p, b);
        report(b, s);
        if (kept) seqs[b] = s;
        const int nb = blocks_of(p, s.n);
        if (per > 1) nblk[b] = nb;
        mine += nb;
      }
      // Offsets that do not ascend can give more blocks than T tokens have, which 32 bits need not hold: then there are none.
      const unsigned most = static_cast<unsigned>(blocks_of(p, p.T)) + p.B;
      unsigned sum;
      int at = static_cast<int>(scan<NT>(min(static_cast<unsigned>(mine), most + 1), reinterpret_cast<unsigned*>(plan_tmp), &sum));
      const int blocks = sum > most ? 0 : static_cast<int>(sum);
      if (per == 1) {
        if (b0 < b1) nblk[b0] = at;
      } else {
        for (int b = b0; b < b1; ++b) {
          const int nb = nblk[b];
          nblk[b] = at;
          at += nb;
        }
      }
      if (tid == 0) nblk[p.B] = blocks;
      __syncthreads();
      if constexpr (CLUSTER) {
        if (tid == 0) {
          const int x = blockIdx.z, b = x < blocks ? seq_of_block(nblk, p.B, x) : 0;
          plan_start[0] = blockIdx.y;
          plan_start[1] = x - nblk[b];
          plan_start[2] = x < blocks;
          plan_start[5] = b;
          *plan_seq = seq_at(b);
          units[0].ntok = 0;
        }
      } else {
        // A thread's blocks x0 .. x1 - 1 (of each key/value head), their tiles, and the tiles before them
        const int pb = (blocks + NT - 1) / NT, x0 = min(blocks, tid * pb), x1 = min(blocks, x0 + pb);
        int all_tiles, tiles = 0;  // of a key/value head: fewer than 2^31 (fa_fwd_paged's limit)
        if (x0 < x1) {
          int b = seq_of_block(nblk, p.B, x0);
          Seq s = seq_at(b);
          for (int x = x0; x < x1; ++x) {
            while (x >= nblk[b + 1]) s = seq_at(++b);
            tiles += block_tiles<BC>(p, s, x - nblk[b]);
          }
        }
        const int before = scan<NT>(tiles, plan_tmp, &all_tiles);
        // A unit's place in the order is the tiles before it and `extra` for each unit.  Up to two tiles a CTA are dealt evenly,
        // one or two each, and starts and ends do not count.
        const int extra = static_cast<long long>(all_tiles) * p.Hkv <= 2 * static_cast<long long>(gridDim.x) ? 0 : cost_unit(D);
        long long* const place = plan_place;  // of each thread's first block in its head
        place[tid] = before + static_cast<long long>(extra) * x0;
        const long long head = all_tiles + static_cast<long long>(extra) * blocks, total = head * p.Hkv;
        const int ranges = static_cast<int>(min(static_cast<long long>(min(static_cast<int>(gridDim.x), NT - 1)), total));
        __syncthreads();
        // Thread i looks up where ranges i and i + 1 begin: the unit that their first place lies in (or, with several blocks a
        // thread, the first one of that thread's).  Where a thread has one block at most, it also knows how long range i is if it
        // takes the units that begin in it, whole.
        long long from[2] = {0, 0}, w[2] = {0, 0}, next[2] = {0, 0};
        int h[2] = {0, 0}, at_block[2] = {0, 0};
        const bool mine_too = tid < ranges;
        if (mine_too) {
          long long in_head[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            w[k] = range_begin(total, tid + k, ranges);
            h[k] = static_cast<int>(static_cast<unsigned>(tid + k) * p.Hkv / ranges);  // w[k] / head: total is Hkv heads
            in_head[k] = w[k] - h[k] * head;
          }
          const int n = pb > 1 ? (blocks + pb - 1) / pb : blocks;
          int lo[2] = {0, 0};
          for (int step = n > 1 ? 1 << (31 - __clz(n - 1)) : 0; step > 0; step >>= 1) {  // last_below, both side by side
#pragma unroll
            for (int k = 0; k < 2; ++k)
              if (lo[k] + step < n && place[lo[k] + step] <= in_head[k]) lo[k] += step;
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            from[k] = h[k] * head + place[lo[k]];
            next[k] = lo[k] + 1 < n ? h[k] * head + place[lo[k] + 1] : (h[k] + 1LL) * head;
            at_block[k] = lo[k] * max(pb, 1);
          }
        }
        // the first unit that begins in a range or behind it
        const long long length = (w[1] == total ? total : w[1] == from[1] ? w[1] : next[1]) - (w[0] == from[0] ? w[0] : next[0]);
        const bool whole = __syncthreads_and(!mine_too || (pb <= 1 && length <= divide(total, ranges) + COST_CUT));
        if (tid == static_cast<int>(blockIdx.x) && mine_too) {
          const int b = seq_of_block(nblk, p.B, at_block[0]);
          plan_start[0] = h[0];
          plan_start[1] = at_block[0] - nblk[b];
          plan_start[5] = b;
          plan_at[0] = from[0];
          plan_at[1] = total;
          plan_at[2] = w[0];
          plan_at[3] = w[1];
        }
        if (tid == 0) {
          plan_start[2] = static_cast<int>(blockIdx.x) < ranges ? ranges : 0;
          plan_start[3] = extra;
          plan_start[4] = whole;
          p.shared[blockIdx.x].parts = 0;
        }
      }
      __syncthreads();
    }
    if (p.G * p.tile_tokens < C::BR) {  // rows of Q that no copy reaches (a tile holds whole tokens) are zeros
      for (int i = tid; i < C::TILES * C::Q_BYTES / 16; i += NT)
        *reinterpret_cast<uint4*>(smem + C::OFF_Q + i * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int ranges = plan_start[2];

  if (ranges == 0) {
    // nothing to do here
  } else if (warp == C::LOAD_WARP || warp == C::LOADV_WARP) {
    // ------------------------------------------------------------ loads
    const bool do_k = warp == C::LOAD_WARP, do_v = warp == C::LOADV_WARP;
    int n = 0, nq = 0, n_tail = 0;  // tiles, query blocks and edge tiles of values so far
    int nk = 0, nv = 0;             // tiles whose copies were issued
    const auto wait_all = [&](uint32_t bar, uint32_t parity, int where) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, p.err, where));
    };
    // the walk through the units (LOAD_WARP): lane i knows sequence base + i
    const long long total = plan_at[1];
    const long long w0 = plan_at[2], w1 = plan_at[3];
    long long at = plan_at[0];
    int h = plan_start[0], b = plan_start[5], blk = plan_start[1], base = -1;
    const int extra = plan_start[3];
    const bool whole = plan_start[4] != 0;
    Seq mine{};
    Unit u;
    long long cut_at = 0;  // place of a shared unit's first tile
    int cut_tiles = 0;
    bool ok = true;
    for (int iu = 0; ok; ++iu) {
      const int slot = iu % C::UNITS;
      if (do_k) {
        u.kind = UNIT_NONE;
        if constexpr (CLUSTER) {
          if (iu == 0) {
            const Seq s = *plan_seq;
            const int first = blk * p.tile_tokens;
            u.h = h;
            u.b = b;
            u.q0 = s.q0 + first;
            u.ntok = min(p.tile_tokens, s.n - first);
            u.pos0 = s.pos0 + first;
            u.bad_page = u.set_aside = 0;
            const Span sp = span_of<BC>(p, u.pos0, u.ntok);
            u.jb = s.bad ? 0 : sp.tiles * blockIdx.x / p.cl;  // fewer than 2^25 tiles
            u.je = s.bad ? 0 : sp.tiles * (blockIdx.x + 1) / p.cl;
            u.ns = sp.ns;
            u.w0 = sp.w0;
            u.lo = sp.lo;
            u.hi = sp.hi;
            u.kind = s.bad ? UNIT_BAD : p.cl == 1 ? UNIT_WHOLE : UNIT_BEGUN;
          }
        } else {
          // the next unit with work in this range
          while (at < w1) {
            if (base < 0 || b < base || b >= base + 32) {
              base = b;
              mine = load_seq(p, base + lane);
            }
            Seq s;
            s.q0 = __shfl_sync(0xffffffffu, mine.q0, b - base);
            s.n = __shfl_sync(0xffffffffu, mine.n, b - base);
            s.pos0 = __shfl_sync(0xffffffffu, mine.pos0, b - base);
            s.bad = __shfl_sync(0xffffffffu, static_cast<int>(mine.bad), b - base);
            const int first = blk * 2 * p.tile_tokens;
            if (first >= s.n) {  // past the sequence's last block
              blk = 0;
              if (++b >= p.B) {
                b = 0;
                ++h;
              }
              continue;
            }
            const long long start = at;
            at += block_tiles<BC>(p, s, blk) + extra;
            u.h = h;
            u.b = b;
            u.q0 = s.q0 + first;
            u.ntok = min(2 * p.tile_tokens, s.n - first);
            u.pos0 = s.pos0 + first;
            ++blk;
            u.bad_page = u.set_aside = 0;
            u.jb = u.je = u.ns = u.w0 = u.lo = u.hi = 0;
            if ((whole || s.bad) && start < w0) continue;  // the range that it begins in has it
            if (s.bad) {
              u.kind = UNIT_BAD;
              break;
            }
            const Span sp = span_of<BC>(p, u.pos0, u.ntok);
            u.jb = whole ? 0 : cut(w0, start, sp.tiles, extra);
            u.je = whole ? sp.tiles : cut(w1, start, sp.tiles, extra);
            if (u.jb >= u.je) continue;  // it lies before the range, or its first tile behind it
            u.ns = sp.ns;
            u.w0 = sp.w0;
            u.lo = sp.lo;
            u.hi = sp.hi;
            u.kind = u.jb > 0 ? UNIT_CONTINUED : u.je < sp.tiles ? UNIT_BEGUN : UNIT_WHOLE;
            if (u.kind != UNIT_WHOLE) cut_at = start + extra, cut_tiles = sp.tiles;
            break;
          }
        }
        if (iu >= C::UNITS) ok = wait_all(bar_ue(slot), (iu / C::UNITS - 1) & 1, W_DESC_FREE);
        if (!ok) break;
        if (lane == 0) {
          units[slot] = u;
          mbar_arrive(bar_uf(slot));
        }
        __syncwarp();
      } else {
        ok = wait_all(bar_uf(slot), (iu / C::UNITS) & 1, W_DESC);
        if (!ok) break;
        u = units[slot];
      }
      if (u.kind == UNIT_NONE) break;
      const int tiles = u.je - u.jb;
      if (tiles > 0) {
        // keys that some row of the block sees; of those, keys below `all` and from `edge` on are seen by every row
        const int sinks = p.window > 0 ? min(p.sinks, u.hi) : 0;
        const int last_lo = p.window > 0 ? max(0, u.pos0 + u.ntok - p.window) : 0;
        const auto used = [&](int key) { return key < u.hi && (key >= u.lo || key < sinks); };
        const auto note_bad = [&]() {
          *reinterpret_cast<volatile int*>(&units[slot].bad_page) = 1;
          record_bad_index(p.err, W_PAGE);
        };
        const int* const table = p.table + u.b * p.table_stride;
        // Sets values aside and zeroes those that no row sees, in the tile's rows that not every row of Q sees.
        const auto clean = [&](uint32_t dv, int key0) {
          constexpr int PIECES = C::NCH * 8;  // 16-byte pieces of a row, which lie in its 128-byte segments in some order
          uint8_t* const tile = smem + (dv - sbase);
          const auto at16 = [&](int i) {
            const int r = i / PIECES, pc = i % PIECES;
            return reinterpret_cast<uint4*>(tile + pc / 8 * C::KV_CH_BYTES + r * 128 + pc % 8 * 16);
          };
          const auto zero = [&](int r0, int r1) {
#pragma unroll 4
            for (int i = r0 * PIECES + lane; i < r1 * PIECES; i += 32) *at16(i) = make_uint4(0, 0, 0, 0);
          };
          const auto check = [&](int r0, int r1) {
#pragma unroll 1
            for (int i0 = r0 * PIECES + lane; i0 < r1 * PIECES; i0 += 128) {  // four loads on their way at a time
              uint4 w[4];
              uint32_t any = 0;
#pragma unroll
              for (int k = 0; k < 4; ++k) w[k] = i0 + 32 * k < r1 * PIECES ? *at16(i0 + 32 * k) : make_uint4(0, 0, 0, 0);
#pragma unroll
              for (int k = 0; k < 4; ++k) any |= not_finite(w[k].x) | not_finite(w[k].y) | not_finite(w[k].z) | not_finite(w[k].w);
              if (any == 0) continue;
              const auto keep = [](uint32_t x) {
                const uint32_t f = not_finite(x);
                return x & ~(((f & 0x8000u) ? 0xFFFFu : 0u) | ((f & 0x80000000u) ? 0xFFFF0000u : 0u));
              };
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (i0 + 32 * k < r1 * PIECES)
                  *at16(i0 + 32 * k) = make_uint4(keep(w[k].x), keep(w[k].y), keep(w[k].z), keep(w[k].w));
              *reinterpret_cast<volatile int*>(&units[slot].set_aside) = 1;
            }
          };
          const auto clip = [&](int key) { return min(BC, max(0, key - key0)); };
          const int s0 = clip(sinks), l0 = clip(u.lo), l1 = clip(last_lo), p0 = clip(u.pos0 + 1), p1 = clip(u.hi);
          if (s0 < l0) zero(s0, l0);                          // behind the sinks, before every window
          if (max(s0, l0) < l1) check(max(s0, l0), l1);       // in some tokens' windows
          check(p0, p1);                                      // the block's own tokens
          zero(p1, BC);                                       // behind the last one
        };
        const auto has_edge = [&](int key0) {
          return key0 + BC > u.pos0 + 1 || (key0 < last_lo && key0 + BC > sinks);
        };
        // TMA: lane i copies the i-th box of a tile, from the page that it looked up a tile ahead; boxes that no row sees and
        // boxes of a bad page are read past the last page: zeros.
        const int boxes = C::GATHER ? 0 : BC / p.box_rows;
        const auto page_of = [&](int j) {
          if (lane >= boxes || j >= u.je) return p.num_pages;
          const int key = key_tile(u, j) * BC + lane * p.box_rows;
          if (key >= u.hi || (key + p.box_rows <= u.lo && key >= sinks)) return p.num_pages;
          const int pg = table[p.by_page.div(key)];
          if (pg >= 0 && pg < p.num_pages) return pg;
          note_bad();
          return p.num_pages;
        };
        const auto copy_boxes = [&](const CUtensorMap* tm, uint32_t dst, uint32_t bar, int key0, int page) {
          __syncwarp();
          if (lane == 0) mbar_expect_tx(bar, C::KV_BYTES);
          __syncwarp();
          if (lane < boxes) {
            const int key = key0 + lane * p.box_rows, row = key - p.by_page.div(key) * p.page_size;
#pragma unroll
            for (int c = 0; c < C::NCH; ++c)
              tma_load_4d(dst + c * C::KV_CH_BYTES + lane * p.box_rows * 128, tm, bar, c * 64, p.heads_inner ? u.h : row,
                          p.heads_inner ? row : u.h, page);
          }
        };
        // Single rows: lane i knows where rows i, i + 32, ... of the tile are (-1: zeros).
        const auto copy_rows = [&](const __nv_bfloat16* cache, uint32_t dst, int key0) {
          long long where[BC / 32];
#pragma unroll
          for (int i = 0; i < BC / 32; ++i) {
            const int key = key0 + i * 32 + lane;
            where[i] = -1;
            if (used(key)) {
              const int pi = p.by_page.div(key), pg = table[pi];
              if (pg >= 0 && pg < p.num_pages)
                where[i] = pg * p.c_page + u.h * p.c_head + (key - pi * p.page_size) * p.c_row;
              else
                note_bad();
            }
          }
          constexpr int PIECES = D / 8, RP = 32 / PIECES;
          const int pc = lane % PIECES;
#pragma unroll
          for (int i = 0; i < BC / RP; ++i) {
            const int r = i * RP + lane / PIECES;
            const long long from = __shfl_sync(0xffffffffu, where[i * RP / 32], r & 31);
            cp_async16(dst + pc / 8 * C::KV_CH_BYTES + r * 128 + ((pc % 8 ^ (r & 7)) << 4), cache + (from < 0 ? 0 : from) + pc * 8,
                       from < 0 ? 0 : 16);
          }
          cp_async_commit();
          cp_async_wait<0>();
        };
        int page = page_of(u.jb);
        for (int j = u.jb; ok && j < u.je; ++j, ++n) {
          const int s = n % STAGES;
          const uint32_t ph = ((n / STAGES) & 1) ^ 1;
          const int key0 = key_tile(u, j) * BC;
          if (do_k) {
            ok = wait_all(bar_ke(s), ph, W_KE);
            if (!ok) break;
            const uint32_t dk = sbase + C::OFF_K + s * C::KV_BYTES;
            if constexpr (C::GATHER) {
              copy_rows(p.k, dk, key0);
              fence_proxy_async();
              __syncwarp();
              if (lane == 0) mbar_arrive(bar_kf(s));
            } else {
              copy_boxes(&tm_k, dk, bar_kf(s), key0, page);
              nk = n + 1;
            }
            if (j == u.jb) {  // the block's queries, once the last block's products have read theirs
              if (nq > 0) ok = wait_all(bar_qe, (nq - 1) & 1, W_QFREE);
              if (!ok) break;
              if (lane == 0) {
                const int tiles_q = u.ntok > p.tile_tokens ? 2 : 1;
                mbar_expect_tx(bar_q, tiles_q * C::NCH * p.G * p.tile_tokens * 128);
                for (int t = 0; t < tiles_q; ++t)
#pragma unroll
                  for (int c = 0; c < C::NCH; ++c)
                    tma_load_3d(sbase + C::OFF_Q + t * C::Q_BYTES + c * C::Q_CH_BYTES, &tm_q, bar_q, c * 64, u.h * p.G,
                                u.q0 + t * p.tile_tokens);
              }
              ++nq;
            }
          }
          if (do_v) {
            ok = wait_all(bar_ve(s), ph, W_VE);
            if (!ok) break;
            const uint32_t dv = sbase + C::OFF_V + s * C::KV_BYTES;
            const bool edge = has_edge(key0);
            if constexpr (C::GATHER) {
              copy_rows(p.v, dv, key0);
              __syncwarp();  // other lanes' copies
              if (edge) clean(dv, key0);
              fence_proxy_async();
              __syncwarp();
              if (lane == 0) mbar_arrive(bar_vf(s));
            } else if (!edge) {
              copy_boxes(&tm_v, dv, bar_vf(s), key0, page);
              nv = n + 1;
            } else {
              copy_boxes(&tm_v, dv, bar_tail, key0, page);
              ok = wait_all(bar_tail, n_tail & 1, W_TAIL);
              ++n_tail;
              if (!ok) break;
              clean(dv, key0);
              fence_proxy_async();
              __syncwarp();
              if (lane == 0) mbar_arrive(bar_vf(s));
              nv = n + 1;
            }
          }
          page = page_of(j + 1);
        }
      }
      if (!do_k && lane == 0) mbar_arrive(bar_ue(slot));
      // A range is a tile long at least: every CTA between the first and the last one has a part.
      if (!CLUSTER && do_k && (u.kind == UNIT_BEGUN || u.kind == UNIT_CONTINUED) && lane == 0) {
        const int from = range_of(total, ranges, cut_at), to = range_of(total, ranges, cut_at + cut_tiles - 1);
        p.shared[blockIdx.x] = Shared{from, to - from + 1, u.h, u.q0, u.ntok};
      }
    }
    if (!C::GATHER || do_k) {
      if (lane == 0) {  // every copy issued must land before the CTA exits
        for (int s = 0; !C::GATHER && s < STAGES; ++s) {
          const int nks = nk > s ? (nk - 1 - s) / STAGES + 1 : 0, nvs = nv > s ? (nv - 1 - s) / STAGES + 1 : 0;
          if (do_k && nks > 0) mbar_wait_drain(bar_kf(s), (nks - 1) & 1, p.err, W_DRAIN_K);
          if (do_v && nvs > 0) mbar_wait_drain(bar_vf(s), (nvs - 1) & 1, p.err, W_DRAIN_V);
        }
        if (do_v && n_tail > 0) mbar_wait_drain(bar_tail, (n_tail - 1) & 1, p.err, W_DRAIN_V);
        if (do_k && nq > 0) mbar_wait_drain(bar_q, (nq - 1) & 1, p.err, W_DRAIN_K);
      }
      __syncwarp();
    }
  } else if (warp == C::MMA_WARP) {
    // ------------------------------------------------------------ products (one elected lane issues)
    const auto wait_all = [&](uint32_t bar, uint32_t parity, int where) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, p.err, where));
    };
    constexpr uint32_t idesc_qk = make_idesc(1, C::BR, BC, 0, 0), idesc_pv = make_idesc(1, C::BR, D, 0, 1);
    const uint64_t dq0 = sdesc_sw128(sbase + C::OFF_Q, 16, 1024), dk0 = sdesc_sw128(sbase + C::OFF_K, 16, 1024);
    const uint64_t dv0 = sdesc_sw128(sbase + C::OFF_V, C::KV_CH_BYTES, 1024);
    const auto issue_qk = [&](int t, int s) {
      const uint64_t qa = dq0 + static_cast<uint64_t>((t * C::Q_BYTES) >> 4);
      const uint64_t kb = dk0 + static_cast<uint64_t>((s * C::KV_BYTES) >> 4);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const int e = kk * 16;
        mma_ss<0>(tmem + t * BC, qa + ((e / 64 * C::Q_CH_BYTES + e % 64 * 2) >> 4),
                  kb + ((e / 64 * C::KV_CH_BYTES + e % 64 * 2) >> 4), idesc_qk, kk > 0);
      }
    };
    const auto issue_pv = [&](int t, int s, bool acc, int kk0, int kk1) {
      const uint64_t vb = dv0 + static_cast<uint64_t>((s * C::KV_BYTES) >> 4);
#pragma unroll
      for (int kk = kk0; kk < kk1; ++kk)
        mma_ts<0>(tmem + C::O_COL0 + t * D, tmem + t * BC + kk * 8, vb + ((kk * 16 * 128) >> 4), idesc_pv,
                  (acc || kk > 0) ? 1u : 0u);
    };
    int n = 0, nq = 0, done[2] = {0, 0};
    bool ok = true;
    for (int iu = 0; ok; ++iu) {
      const int slot = iu % C::UNITS;
      ok = wait_all(bar_uf(slot), (iu / C::UNITS) & 1, W_DESC);
      if (!ok) break;
      const Unit u = units[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_ue(slot));
      if (u.kind == UNIT_NONE) break;
      const int T = u.je - u.jb;
      if (T == 0) continue;
      const int st[2] = {steps_of<BC>(u, 0, p.tile_tokens), steps_of<BC>(u, 1, p.tile_tokens)};
      ok = wait_all(bar_q, nq & 1, W_Q) && wait_all(bar_kf(n % STAGES), (n / STAGES) & 1, W_KF);
      ++nq;
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (st[t] > 0) {
            issue_qk(t, n % STAGES);
            mma_commit(bar_sf(t));
          }
        mma_commit(bar_ke(n % STAGES));
        if (T == 1) mma_commit(bar_qe);
      }
      __syncwarp();
      for (int j = 0; ok && j < T; ++j, ++n) {
        const int s = n % STAGES, n1 = n + 1, s1 = n1 % STAGES;
        ok = wait_all(bar_vf(s), (n / STAGES) & 1, W_VF);
        if (ok && j + 1 < T) ok = wait_all(bar_kf(s1), (n1 / STAGES) & 1, W_KF);
        if (!ok) break;
        const int last = st[1] > j ? 1 : 0;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (st[t] <= j) continue;
          if constexpr (C::PV2) {
            ok = ok && wait_all(bar_ph(t), done[t] & 1, W_PF);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) issue_pv(t, s, j > 0, 0, BC / 32);
            __syncwarp();
          }
          ok = ok && wait_all(bar_pf(t), done[t] & 1, W_PF);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            issue_pv(t, s, C::PV2 || j > 0, C::PV2 ? BC / 32 : 0, BC / 16);
            if (t == last) mma_commit(bar_ve(s));
            if (j + 1 < st[t]) {
              issue_qk(t, s1);
              mma_commit(bar_sf(t));
            } else {
              mma_commit(bar_od(t));
            }
            if (t == last && j + 1 < T) {
              mma_commit(bar_ke(s1));
              if (j + 2 == T) mma_commit(bar_qe);
            }
          }
          __syncwarp();
          ++done[t];
        }
      }
    }
    // every product issued above completes before tensor memory is freed
    if (elect_one()) mma_commit(bar_drain);
    __syncwarp();
    mbar_wait_drain(bar_drain, 0, p.err, W_DRAIN_MMA);
  } else {
    // ------------------------------------------------------------ softmax warpgroups, a thread a row
    const int t = warp >> 2, wq = warp & 3, row = wq * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem + lane_base + t * BC, tO = tmem + lane_base + C::O_COL0 + t * D;
    const int my_tok = p.by_g.div(row), g = row - my_tok * p.G;
    const float c = p.c;
    const uint64_t c2 = f2_pack(c, c);
    const uint32_t hidden = __float_as_uint(c >= 0.f ? -INFINITY : INFINITY);  // a score that is not seen, before scaling
    int done = 0, n_od = 0;
    bool ok = true;
    const auto rescale = [&](float alpha) {
      const uint64_t a2 = f2_pack(alpha, alpha);
#pragma unroll
      for (int cc = 0; cc < D / 32; ++cc) {
        uint32_t orr[32];
        tmem_ld32(tO + cc * 32, orr);
        tmem_wait_ld();
        reg_fence(orr);
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const uint64_t v = f2_mul(f2_pack(__uint_as_float(orr[e]), __uint_as_float(orr[e + 1])), a2);
          f2_unpack(v, orr[e], orr[e + 1]);
        }
        tmem_st32(tO + cc * 32, orr);
      }
    };
    const auto hand_over = [&](uint32_t bar) {
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    for (int iu = 0; ok; ++iu) {
      const int slot = iu % C::UNITS;
      ok = __all_sync(0xffffffffu, mbar_wait(bar_uf(slot), (iu / C::UNITS) & 1, abort_flag, p.err, W_DESC));
      if (!ok) break;
      const volatile Unit& uv = units[slot];
      if (uv.kind == UNIT_NONE) break;
      // What the steps below do not need is read again where it is used: they have no registers to spare.
      const int pos = uv.pos0 + min(t * p.tile_tokens + my_tok, uv.ntok - 1);
      const int steps = steps_of<BC>(uv, t, p.tile_tokens);
      // Rows that are not the unit's hold other sequences' queries, or whatever lies in unused places.  In a warp with rows of the
      // unit their reference maximum is infinity: their P are zeros or NaN, and they hold up none of the votes below, which NaN
      // passes.  (A warp without rows of the unit votes for itself; with infinity there too it takes the fast path on a unit's
      // first tile beside the others' general one: 256 single tokens behind 100 keys, d = 128, 65 us instead of 62.)
      const bool mine = my_tok < p.tile_tokens && t * p.tile_tokens + my_tok < uv.ntok;
      const bool any_mine = __any_sync(0xffffffffu, mine);
      float m_ref = mine || !any_mine ? -INFINITY : INFINITY, l = 0.f;
      for (int j = 0; j < steps; ++j, ++done) {
        const bool okw = __all_sync(0xffffffffu, mbar_wait(bar_sf(t), done & 1, abort_flag, p.err, W_SF));
        if (!okw) {
          ok = false;
          break;
        }
        const int jj = uv.jb + j, ns = uv.ns;
        const int key0 = (jj < ns ? jj : uv.w0 + jj - ns) * BC;
        // columns valid > e, and from `first` on or among the sinks
        const int valid = pos + 1 - key0;
        const int first = p.window > 0 ? pos - p.window + 1 - key0 : 0, sink = p.sinks - key0;
        const bool full = __all_sync(0xffffffffu, valid >= BC && (first <= 0 || sink >= BC));
        const bool started = __all_sync(0xffffffffu, m_ref != -INFINITY);
        tc_fence_after();
        // Once every row of the warp has a reference maximum and sees all columns, P is computed against it with no row maximum
        // in front of it; row sums of at most 2^tau (and at d = 128 the second half's maximum) show that no score moved past
        // m_ref + tau.  Otherwise nothing has been stored yet, and the general path reads S again (fa_fwd_kernel.cuh, `fast`, PV2).
        // (A row with NaN among its scores is NaN by either path.)
        // (A masked copy of it costs more in registers and code than it saves: 375 us on a prompt of 8191 tokens, d = 128, without
        // it 371; a mixed batch, d = 64, 89 and 86.)
        const auto fast = [&]() -> bool {
          const uint64_t negm2 = f2_pack(-m_ref, -m_ref);
          float r0, r1, r2, r3;
          if constexpr (C::PV2) {
            uint32_t sr[BC / 32][32];
#pragma unroll
            for (int i = 0; i < BC / 32; ++i) tmem_ld32(tS + i * 32, sr[i]);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < BC / 32; ++i) reg_fence(sr[i]);
            constexpr int HC = BC / 2, HP = BC / 128;  // columns and packed 32-column chunks of half of P
            auto& sr_a = reinterpret_cast<uint32_t(&)[HC / 32][32]>(sr[0]);
            auto& sr_b = reinterpret_cast<uint32_t(&)[HC / 32][32]>(sr[HC / 32]);
            uint32_t pk[HP][32];
            uint64_t rs[2] = {0ull, 0ull};
            softmax_p_bf16<HC, false>(sr_a, pk, c2, negm2, HC, rs);
            const float m_b = (c >= 0.f ? row_extreme<HC, true>(sr_b) : row_extreme<HC, false>(sr_b)) * c;
            f2_unpack_f(rs[0], r0, r1);
            f2_unpack_f(rs[1], r2, r3);
            const float l_a = (r0 + r1) + (r2 + r3);
            if (__any_sync(0xffffffffu, l_a > p.p_lim || m_b > m_ref + p.tau)) return false;
#pragma unroll
            for (int i = 0; i < HP; ++i) tmem_st32(tS + i * 32, pk[i]);
            hand_over(bar_ph(t));
            uint64_t rs_b[2] = {0ull, 0ull};
            softmax_p_bf16<HC, false>(sr_b, pk, c2, negm2, HC, rs_b);
#pragma unroll
            for (int i = 0; i < HP; ++i) tmem_st32(tS + (HP + i) * 32, pk[i]);
            hand_over(bar_pf(t));
            f2_unpack_f(rs_b[0], r0, r1);
            f2_unpack_f(rs_b[1], r2, r3);
            l += l_a + ((r0 + r1) + (r2 + r3));
          } else {  // the scores of 32 columns arrive while those before them are worked on
            uint32_t sc[2][32], pk[32];
            uint64_t rs[2] = {0ull, 0ull};
            tmem_ld32(tS, sc[0]);
            tmem_wait_ld();
            reg_fence(sc[0]);
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) {
              if (cc == 0) tmem_ld32(tS + 32, sc[1]);
#pragma unroll
              for (int qc = 0; qc < 16; ++qc) {
                const uint64_t x = f2_fma(f2_pack(__uint_as_float(sc[cc][2 * qc]), __uint_as_float(sc[cc][2 * qc + 1])), c2, negm2);
                float x0, x1;
                f2_unpack_f(x, x0, x1);
                const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                rs[qc & 1] = f2_add(rs[qc & 1], f2_pack(p0, p1));
                pk[cc * 16 + qc] = pack_bf16x2(p0, p1);
              }
              if (cc == 0) {
                tmem_wait_ld();
                reg_fence(sc[1]);
              }
            }
            f2_unpack_f(rs[0], r0, r1);
            f2_unpack_f(rs[1], r2, r3);
            const float l_tile = (r0 + r1) + (r2 + r3);
            if (__any_sync(0xffffffffu, l_tile > p.p_lim)) return false;
            tmem_st32(tS, pk);
            hand_over(bar_pf(t));
            l += l_tile;
          }
          return true;
        };
        if (started && full && fast()) continue;
        // The general path: the maximum of the columns that the row sees, then P.
        uint32_t sr[BC / 32][32];
#pragma unroll
        for (int cc = 0; cc < BC / 32; ++cc) tmem_ld32(tS + cc * 32, sr[cc]);
        tmem_wait_ld();
        float m_new = m_ref;
#pragma unroll
        for (int cc = 0; cc < BC / 32; ++cc) {
          reg_fence(sr[cc]);
          if (!full) {
            const uint32_t vis = low_bits(valid - 32 * cc) & (~low_bits(first - 32 * cc) | low_bits(sink - 32 * cc));
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(vis >> e & 1u)) sr[cc][e] = hidden;
          }
          auto& one = reinterpret_cast<uint32_t(&)[1][32]>(sr[cc]);
          m_new = fmaxf(m_new, (c >= 0.f ? row_extreme<32, true>(one) : row_extreme<32, false>(one)) * c);
        }
        const bool need = m_new > m_ref + p.tau;  // always true on the first tile that a row sees
        float alpha = 1.f;
        if (need) {
          alpha = ex2_approx(m_ref - m_new);  // 0 the first time
          m_ref = m_new;
        }
        const float m_use = m_ref == -INFINITY ? 0.f : m_ref;  // a row that has seen nothing: 2^(-inf - 0) = 0
        const uint64_t negm2 = f2_pack(-m_use, -m_use);
        uint64_t rs[2] = {0ull, 0ull};
#pragma unroll
        for (int cc = 0; cc < BC / 32; ++cc) {
          uint32_t pk[32];
#pragma unroll
          for (int qc = 0; qc < 16; ++qc) {
            const uint64_t x = f2_fma(f2_pack(__uint_as_float(sr[cc][2 * qc]), __uint_as_float(sr[cc][2 * qc + 1])), c2, negm2);
            float x0, x1;
            f2_unpack_f(x, x0, x1);
            const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
            rs[qc & 1] = f2_add(rs[qc & 1], f2_pack(p0, p1));
            pk[qc] = pack_bf16x2(p0, p1);
          }
          tmem_st16_lo(tS + cc * 16, pk);
          if (cc == BC / 64 - 1 || BC == 64) {
            // the correction of O, before the first product that adds to it
            if ((C::PV2 || cc == BC / 32 - 1) && j > 0 && __any_sync(0xffffffffu, need)) rescale(alpha);
            if (C::PV2) hand_over(bar_ph(t));
          }
        }
        hand_over(bar_pf(t));
        float r0, r1, r2, r3;
        f2_unpack_f(rs[0], r0, r1);
        f2_unpack_f(rs[1], r2, r3);
        l = l * alpha + ((r0 + r1) + (r2 + r3));
      }
      if (!ok) break;
      // ---------------------------------------------------------- epilogue
      if (steps > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar_od(t), n_od & 1, abort_flag, p.err, W_OD));
        ++n_od;
        if (!ok) break;
        tc_fence_after();
      }
      const int kind = uv.kind, ntok = uv.ntok, tok = t * p.tile_tokens + my_tok;
      const bool real = my_tok < p.tile_tokens && tok < ntok, aside = uv.set_aside != 0;
      if (uv.bad_page || kind == UNIT_BAD) l = __int_as_float(0x7fc00000);
      const bool any_rows = t * p.tile_tokens < ntok;
      if (!any_rows) {
        // a block of one tile
      } else if (CLUSTER ? p.cl == 1 : kind == UNIT_WHOLE || kind == UNIT_BAD) {
        // A thread holds a row: written straight from there, a warp's 16 bytes a lane would touch 32 half sectors.  So OUT_COLS
        // columns at a time go through shared memory (16-byte pieces swapped by the row) and out in whole sectors.
        constexpr int PCS = C::OUT_COLS / 8, RPI = 32 / PCS;  // pieces of a row, rows a store
        const float inv_l = 1.f / l;
        const size_t out = static_cast<size_t>(uv.q0 + tok) * p.H + uv.h * p.G + g;
        uint8_t* const stage = smem + C::OFF_STAGE + warp * C::STAGE_BYTES;
        const int piece = lane % PCS;
        const auto at16 = [&](int r, int pc) {
          return reinterpret_cast<uint4*>(stage + r * (PCS * 16) + ((pc ^ (r / (8 / PCS) % PCS)) << 4));
        };
        __nv_bfloat16* rows[PCS];  // that this lane writes pieces of
#pragma unroll
        for (int i = 0; i < PCS; ++i) {
          const int r = wq * 32 + i * RPI + lane / PCS, rt = p.by_g.div(r), tk = t * p.tile_tokens + rt;
          rows[i] = rt < p.tile_tokens && tk < ntok
                        ? p.o + (static_cast<size_t>(uv.q0 + tk) * p.H + uv.h * p.G + r - rt * p.G) * D + piece * 8
                        : nullptr;
        }
#pragma unroll
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t orr[32];
          tmem_ld32(tO + cc * 32, orr);
          tmem_wait_ld();
          reg_fence(orr);
#pragma unroll
          for (int half = 0; half < 32 / C::OUT_COLS; ++half) {
#pragma unroll
            for (int v4 = 0; v4 < PCS; ++v4) {
              const auto two = [&](int e) {
                const int at = half * C::OUT_COLS + 8 * v4 + e;
                return pack_bf16x2(__uint_as_float(orr[at]) * inv_l, __uint_as_float(orr[at + 1]) * inv_l);
              };
              *at16(lane, v4) = make_uint4(two(0), two(2), two(4), two(6));
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < PCS; ++i) {
              const uint4 w = *at16(i * RPI + lane / PCS, piece);
              if (rows[i] != nullptr) *reinterpret_cast<uint4*>(rows[i] + cc * 32 + half * C::OUT_COLS) = w;
            }
            __syncwarp();
          }
        }
        if (p.lse != nullptr && real) p.lse[out] = (m_ref + log2f(l)) * 0.6931471805599453f;
        if (aside && real) add_aside<C, false>(p, uv, pos, p.o + out * D, D, 0);
      } else {
        // Partial state: 16-byte pieces of the rows side by side, so that a warp's stores are whole lines; in a cluster rows side
        // by side in shared memory, their pieces swapped by the row.
        const size_t part = (static_cast<size_t>(blockIdx.x) * 2 + (kind == UNIT_BEGUN)) * p.part_tiles + t;
        float4* const po = CLUSTER ? reinterpret_cast<float4*>(smem + C::OFF_STATE) + row * (D / 4)
                                   : p.part_o + part * (D / 4) * p.part_rows + row;
#pragma unroll
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t orr[32];
          if (steps > 0) {
            tmem_ld32(tO + cc * 32, orr);
            tmem_wait_ld();
            reg_fence(orr);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) orr[e] = 0;
          }
          if (real) {
#pragma unroll
            for (int v4 = 0; v4 < 8; ++v4)
              po[CLUSTER ? (cc * 8 + v4) ^ (row & (D / 4 - 1)) : static_cast<size_t>(cc * 8 + v4) * p.part_rows] =
                  make_float4(__uint_as_float(orr[4 * v4]), __uint_as_float(orr[4 * v4 + 1]), __uint_as_float(orr[4 * v4 + 2]),
                              __uint_as_float(orr[4 * v4 + 3]));
          }
        }
        float2* const pml = CLUSTER ? reinterpret_cast<float2*>(smem + C::OFF_ML) + row : p.part_ml + part * p.part_rows + row;
        if (real) *pml = make_float2(m_ref, l);
        if (aside && real) add_aside<C, CLUSTER>(p, uv, pos, reinterpret_cast<float*>(po), 4, CLUSTER ? row : 4LL * p.part_rows);
      }
      tc_fence_before();  // O has been read: the next unit's first P V comes behind this warp's next hand_over
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_ue(slot));
    }
  }

  __syncwarp();
  tc_fence_before();
  const bool shared = CLUSTER && p.cl > 1;
  if (shared) cluster_sync();
  else __syncthreads();
  if (warp == C::LOAD_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
  if (shared) {
    join_cluster<C>(p, units[0], sbase);
    cluster_sync();  // a CTA's shared memory is there while others read it
  }
}

// Joins the states of shared units in the order of their keys: O = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.  A block has 32 rows
// (a lane each) of one row tile, each of its D / 8 warps 8 columns of a unit that two CTAs share.  A unit that n CTAs share has
// the blocks of the first n - 1 of them, or as many as a power of two and D / 8 allow: each has a share of the columns, and its
// warps split the parts, whose states they join in shared memory.
template <int D>
__global__ void __launch_bounds__(D * 4, D == 128 ? 3 : 6) fa_fwd_paged_join_kernel(const ChunkParams p) {
  constexpr int WARPS = D / 8;
  __shared__ float4 states[WARPS][2][32];
  __shared__ float2 states_ml[WARPS][32];
  griddep_wait();
  const int t = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.z * 32 + lane;
  const Shared u = p.shared[blockIdx.x];
  if (u.parts == 0) return;
  const int mine = blockIdx.x - u.first;  // which of the unit's blocks
  int blocks = 1;
  while (2 * blocks <= min(u.parts - 1, WARPS)) blocks *= 2;
  if (mine >= blocks || t * p.tile_tokens >= u.ntok) return;
  const int slice = warp % blocks, col8 = mine * (WARPS / blocks) + warp / blocks;
  const int my_tok = p.by_g.div(row), g = row - my_tok * p.G, tok = t * p.tile_tokens + my_tok;
  const bool real = my_tok < p.tile_tokens && tok < u.ntok;
  float m = -INFINITY, l = 0.f, o[8] = {};
  for (int i0 = slice; real && i0 < u.parts; i0 += 2 * blocks) {  // two parts at a time
    float2 ml[2];
    float4 x[2][2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = i0 + k * blocks;
      ml[k] = make_float2(-INFINITY, 0.f);
      x[k][0] = x[k][1] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < u.parts) {
        // the first CTA's state of a unit that it begins, or another one's of a unit that it continues
        const size_t part = static_cast<size_t>(u.first + i) * 2 * p.part_tiles + (i == 0 ? p.part_tiles : 0) + t;
        const float4* const po = p.part_o + (part * (D / 4) + col8 * 2) * p.part_rows + row;
        ml[k] = p.part_ml[part * p.part_rows + row];
        x[k][0] = po[0];
        x[k][1] = po[p.part_rows];
      }
    }
    const float m_new = fmaxf(m, fmaxf(ml[0].x, ml[1].x));
    const float m_use = m_new == -INFINITY ? 0.f : m_new;  // no part so far sees a key of this row: weights of 0
    const float old = ex2_approx(m - m_use);
    l *= old;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] *= old;
    m = m_new;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float w = ex2_approx(ml[k].x - m_use);
      l = fmaf(w, ml[k].y, l);
      o[0] = fmaf(w, x[k][0].x, o[0]);
      o[1] = fmaf(w, x[k][0].y, o[1]);
      o[2] = fmaf(w, x[k][0].z, o[2]);
      o[3] = fmaf(w, x[k][0].w, o[3]);
      o[4] = fmaf(w, x[k][1].x, o[4]);
      o[5] = fmaf(w, x[k][1].y, o[5]);
      o[6] = fmaf(w, x[k][1].z, o[6]);
      o[7] = fmaf(w, x[k][1].w, o[7]);
    }
  }
  if (blocks > 1) {
    states_ml[warp][lane] = make_float2(m, l);
    states[warp][0][lane] = make_float4(o[0], o[1], o[2], o[3]);
    states[warp][1][lane] = make_float4(o[4], o[5], o[6], o[7]);
    __syncthreads();
    if (slice > 0) return;
    for (int w = 1; w < blocks; ++w) m = fmaxf(m, states_ml[warp + w][lane].x);
    const float m_use = m == -INFINITY ? 0.f : m;
    l = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = 0.f;
    for (int w = 0; w < blocks; ++w) {
      const float2 ml = states_ml[warp + w][lane];
      const float4 a = states[warp + w][0][lane], b = states[warp + w][1][lane];
      const float f = ex2_approx(ml.x - m_use);
      l = fmaf(f, ml.y, l);
      o[0] = fmaf(f, a.x, o[0]);
      o[1] = fmaf(f, a.y, o[1]);
      o[2] = fmaf(f, a.z, o[2]);
      o[3] = fmaf(f, a.w, o[3]);
      o[4] = fmaf(f, b.x, o[4]);
      o[5] = fmaf(f, b.y, o[5]);
      o[6] = fmaf(f, b.z, o[6]);
      o[7] = fmaf(f, b.w, o[7]);
    }
  }
  if (!real) return;
  const float inv = 1.f / l;
  const size_t out = static_cast<size_t>(u.q0 + tok) * p.H + u.h * p.G + g;
  *reinterpret_cast<uint4*>(p.o + out * D + col8 * 8) =
      make_uint4(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv), pack_bf16x2(o[4] * inv, o[5] * inv),
                 pack_bf16x2(o[6] * inv, o[7] * inv));
  if (p.lse != nullptr && col8 == 0) p.lse[out] = (m + log2f(l)) * 0.6931471805599453f;
}

// The workspace: states of shared units, and who shares them.
struct Layout {
  int rows, tiles;
  size_t part_ml, shared, total;
};
Layout layout_of(int T, int H, int Hkv, int d, int sms) {
  const int G = H / Hkv, tokens = FWD_PAGED_MAX_G / G;
  Layout l;
  l.tiles = T > tokens ? 2 : 1;
  l.rows = T >= tokens ? 128 : (T * G + 31) / 32 * 32;
  const size_t ctas = static_cast<size_t>(sms) * (d == 128 ? Ranges<128, false>::MINB : Ranges<64, false>::MINB);
  const size_t states = ctas * 2 * l.tiles * l.rows;
  l.part_ml = states * d * 4;
  l.shared = l.part_ml + states * 8;
  l.total = l.shared + ctas * sizeof(Shared);
  return l;
}

// Rows of the largest copy that stays in one page and starts on a swizzle boundary: a power of two that divides the page
// size, at most the key tile.  Under 8 rows there is none.
int box_rows_of(int page_size, int bc) {
  const int r = page_size & -page_size;
  return r > bc ? bc : r;
}

// As many units as a call of its sizes can have.
template <class C>
long long units_of(const FwdPagedLaunch& a) {
  return (static_cast<long long>(a.T) / (C::BR / (a.H / a.Hkv)) + (a.B < a.T ? a.B : a.T)) * a.Hkv;
}

// Rows of a unit, if the sequences have as many tokens each.
template <class C>
int rows_of(const FwdPagedLaunch& a) {
  const int G = a.H / a.Hkv;
  return std::min<long long>(C::BR / G, (static_cast<long long>(a.T) + a.B - 1) / a.B) * G;
}

// CTAs of a unit where every unit has a cluster, or 0 for ranges.  `tiles`: of the longest one that its table, or the window,
// allows; n_cta: CTAs that may run at once.  As many as there is room for, less the places that clusters of this size leave free
// in each of the GPU's 8 processor clusters; one for two tiles, which take less than one and the join.
//
// A cluster saves the dealing, the states in memory and the join, 3 to 7 us, and two CTAs on an SM work on units of few rows at the
// same time, where one range has them one behind the other; but its CTAs work on no other unit.  So it is taken where its CTAs'
// tiles are at most `more` more than an even share: that of one longest sequence alone, or of sequences half as long, or of one's
// units, three quarters.  Ranges and clusters, device time, 32 heads on 8, us: 23 tokens behind 1000 keys d = 128 13.2 and 9.2,
// d = 64 12.5 and 8.4; behind 4000 15.8 and 13.7, 16.2 and 11.1; behind 16000 20.9 and 25.5, 20.5 and 21.1; 16 x 4 tokens behind
// 1000 21.1 and 15.8, 21.0 and 13.9; behind 1 to 2000 27.2 and 23.0, 21.9 and 19.8; behind 1 to 4000 39 and 46, 29 and 36; a
// prompt of 500 17.8 and 12.0, 17.8 and 12.5.  Clusters of more than 8: 23 tokens behind 8000, d = 64, 17.7 with 8 CTAs, 14.2
// with 16.  (A cluster of cl CTAs is taken only where there are 9 cl - 8 places for CTAs at least, and so at least cl in one of the
// 8 processor clusters: it can be placed.)
//
// The host has bounds of the tiles and units only: tables much wider than the sequences, or places for many more tokens, are
// taken for long sequences and many units, and their calls dealt (the first times of the pairs above instead of the second).
//
// More units than CTAs may run at once, if short, come in waves, of a CTA each, up to `halves` halves of what may run: 128 single
// tokens behind 300 (3.5 waves) 59.6 and 48.1, 37.2 and 38.4; 256 behind 100 (7) 70.7 and 60.9, 40.5 and 49.8; 60 x 18 tokens
// behind 200 (2.4) 31.7 and 21.1, 22.5 and 19.5; 64 x 100 behind 100 (7) 63 and 77, 45 and 67.
template <class C>
int cluster_size(const FwdPagedLaunch& a, long long tiles) {
  const long long units = units_of<C>(a), n_cta = a.sms * C::MINB;
  const bool few = rows_of<C>(a) <= 64;
  if (units > n_cta) {
    const int halves = !few ? 5 : C::D == 128 ? 16 : 7, most = few && C::D == 128 ? 16 : 8;
    return 2 * units <= halves * n_cta && tiles <= most ? 1 : 0;
  }
  int cl = 1;
  if (tiles > 2)
    while (cl < MAX_CLUSTER && cl < tiles && units * (cl + 1) <= n_cta - 8 * cl) ++cl;
  const long long share = std::max(tiles * a.Hkv, units * tiles * (a.B == 1 ? 3 : 2) / 4) / n_cta;
  const int more = few ? 12 : 8;
  return (tiles + cl - 1) / cl <= share + more ? cl : 0;
}

// p.cl by the keys' tiles of C, 0 for ranges, and about how long the call takes after its start, in tenths of a microsecond.
struct Form {
  int cl;
  long long cost;
};
template <class C>
Form form_of(const FwdPagedLaunch& a) {
  const int tokens = C::BR / (a.H / a.Hkv);
  long long tiles = (static_cast<long long>(a.max_pages) * a.page_size + C::BC - 1) / C::BC;
  if (a.window > 0) {
    const long long seen = (static_cast<long long>(a.window) + tokens) / C::BC + 2 + a.sinks / C::BC + 1;
    tiles = seen < tiles ? seen : tiles;
  }
  const int cl = cluster_size<C>(a, tiles);
  if (cl == 0) return {0, 0};
  // Two CTAs on an SM take their steps at the same time only while their tiles have few rows.
  const int step = C::BC == 128 || (rows_of<C>(a) > 64 && units_of<C>(a) * cl > a.sms) ? 19 : 15;
  return {cl, (tiles + cl - 1) / cl * step + (cl == 1 ? 0 : cl <= 8 ? 20 : 27)};
}

template <class C>
cudaError_t launch_cfg(const FwdPagedLaunch& a, int cl) {
  cudaError_t e = allow_shared_memory<fa_fwd_paged_kernel<C>>(C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  const Layout l = layout_of(a.T, a.H, a.Hkv, a.d, a.sms);
  ChunkParams p = {};
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.lse = a.lse;
  p.k = static_cast<const __nv_bfloat16*>(a.k_cache);
  p.v = static_cast<const __nv_bfloat16*>(a.v_cache);
  p.c_page = a.c_page;
  p.c_head = a.c_head;
  p.c_row = a.c_row;
  p.table = a.table;
  p.cu = a.cu;
  p.lens = a.lens;
  p.table_stride = a.table_stride;
  p.err = a.err;
  if (!C::CLUSTER) {
    p.part_o = reinterpret_cast<float4*>(a.ws);
    p.part_ml = reinterpret_cast<float2*>(a.ws + l.part_ml);
    p.shared = reinterpret_cast<Shared*>(a.ws + l.shared);
  }
  p.G = a.H / a.Hkv;
  p.tile_tokens = C::BR / p.G;
  p.by_g = FastDiv(static_cast<unsigned>(p.G));
  p.by_page = FastDiv(static_cast<unsigned>(a.page_size));
  p.by_block = FastDiv(static_cast<unsigned>(C::TILES * p.tile_tokens));
  p.T = a.T;
  p.B = a.B;
  p.H = a.H;
  p.Hkv = a.Hkv;
  p.cl = cl;
  p.part_rows = l.rows;
  p.part_tiles = l.tiles;
  p.num_pages = a.num_pages;
  p.page_size = a.page_size;
  p.max_pages = a.max_pages;
  p.box_rows = box_rows_of(a.page_size, C::BC);
  p.heads_inner = a.c_row > a.c_head;
  p.window = std::min(a.window, 1 << 30);  // no more keys than that: `pos - window + 1 - key` stays in 32 bits
  p.sinks = a.window > 0 ? a.sinks : 0;
  p.c = a.c == 0.f ? 1e-30f : a.c;  // a hidden score (an infinity) times zero would be NaN
  p.tau = kTau;
  p.p_lim = exp2f(kTau);
  CUtensorMap tq, tk = {}, tv = {};
  e = encode_heads_map(&tq, a.q, a.d, a.H, a.T, a.q_head, a.q_tok, p.G, p.tile_tokens);
  if (e == cudaSuccess && !C::GATHER)
    e = encode_paged_map(&tk, a.k_cache, a.d, a.page_size, a.Hkv, a.num_pages, a.c_row, a.c_head, a.c_page, p.box_rows,
                         p.heads_inner);
  if (e == cudaSuccess && !C::GATHER)
    e = encode_paged_map(&tv, a.v_cache, a.d, a.page_size, a.Hkv, a.num_pages, a.c_row, a.c_head, a.c_page, p.box_rows,
                         p.heads_inner);
  if (e != cudaSuccess) return e;
  if constexpr (C::CLUSTER) {
    if (cl > 8) e = cudaFuncSetAttribute(fa_fwd_paged_kernel<C>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    return launch_dependent_clusters(fa_fwd_paged_kernel<C>, dim3(cl, a.Hkv, static_cast<unsigned>(units_of<C>(a) / a.Hkv)), cl,
                                     C::NTHREADS, C::SMEM_BYTES, a.stream, tq, tk, tv, p);
  } else {
    const unsigned grid = static_cast<unsigned>(a.sms * C::MINB);
    e = launch_dependent(fa_fwd_paged_kernel<C>, dim3(grid), C::NTHREADS, C::SMEM_BYTES, a.stream, tq, tk, tv, p);
    if (e != cudaSuccess) return e;
    return launch_dependent(fa_fwd_paged_join_kernel<C::D>, dim3(grid, l.tiles, l.rows / 32), C::D * 4, 0, a.stream, p);
  }
}

// At d = 128 a cluster's CTAs have key tiles of 64, or, where units of many rows are few, one CTA an SM with tiles of 128 (a
// prompt of 500, 32 heads on 8: 12.0 us instead of 15.8, 23 tokens behind 1000 9.2 instead of 10.5; 4 x 4 tokens behind 1000 10.9
// instead of 10.1, 32 single tokens behind 200 18.1 instead of 10.5).  Copies of single rows change nothing here.
template <int D>
FwdPagedForm choose(const FwdPagedLaunch& a) {
  using C = Cluster<D, false>;
  const Form f = form_of<C>(a);
  if constexpr (D == 128) {
    const Form g = form_of<Cluster<D, false, 128>>(a);
    if (f.cl > 0 && g.cl > 0 && rows_of<C>(a) > 64 && units_of<C>(a) <= a.sms && g.cost <= f.cost) return {g.cl, 1};
  }
  return {f.cl, 0};
}

template <int D, bool GATHER>
cudaError_t launch_form(const FwdPagedLaunch& a, FwdPagedForm form) {
  if (form.cl == 0) return launch_cfg<Ranges<D, GATHER>>(a, 0);
  if constexpr (D == 128) {
    if (form.wide) return launch_cfg<Cluster<D, GATHER, 128>>(a, form.cl);
  }
  return launch_cfg<Cluster<D, GATHER>>(a, form.cl);
}

}  // namespace

FwdPagedForm fwd_paged_form(const FwdPagedLaunch& a) { return a.d == 64 ? choose<64>(a) : choose<128>(a); }

size_t fwd_paged_workspace(int T, int H, int Hkv, int d, int sms) { return layout_of(T, H, Hkv, d, sms).total; }

cudaError_t launch_fwd_paged(const FwdPagedLaunch& a, FwdPagedForm form) {
  const bool gather = a.page_size % 8 != 0;
  if (a.d == 64) return gather ? launch_form<64, true>(a, form) : launch_form<64, false>(a, form);
  return gather ? launch_form<128, true>(a, form) : launch_form<128, false>(a, form);
}

}  // namespace fa
