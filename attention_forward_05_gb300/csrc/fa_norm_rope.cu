// fa_norm_rope.cu -- root-mean-square norms of the query and key heads with the position rotation in the same pass:
// on dense q and k, on their gradients, and on new tokens as they are appended to a paged cache.
//
// Mathematics.  For a head x of d elements with weights w,
//   r = (mean(x^2) + eps)^(-1/2),  u = r x,  y = R(w u),
// R the rotation of fa_rope.cu.  R is orthogonal, so with the output's gradient dy and g = R^-1 dy,
//   dw = sum over tokens and heads of g u,   dx = r (w g - u mean(w g u)).
// The backward pass forms r again from x: reading a stored one would save nothing, x is needed anyway.
//
// Work split.  That of fa_rope_items.cuh: a lane holds 16 elements of a head, so a head's sums are d / 16 lanes' sums and
// two or three shuffles; everything between the ring and the store stays in registers, in fp32, rounded once.  Every block
// has its part of the query heads, then of the key heads, so a lane's registers hold one set of weights.  Forward, the
// weights are multiplied into a token's turn, once for all of its heads.  Backward, a lane adds up its elements' share of dw
// over all its items, a block joins its lanes' shares in a fixed order and leaves them in the workspace, and
// fa_norm_rope_join_kernel adds the blocks' (no atomics: the same bits every time).
//
// Bound by device memory: 336 MB forward (2 x 8192 tokens, 32 + 8 heads of 128, bf16) 57 us, 5.9 TB/s with the launch, where
// the rotation alone takes 53 on as many bytes; 503 MB backward 86 us, 5.9 TB/s.  With all heads of an item in registers at a
// time (they spill) 78 and 138 us; with query and key heads on blocks of their own 63.5 and 94; forward with 4 and 2 blocks a
// SM 62.5 and 64, with items of twice as many heads 65.  The same in fp32 118 us, 5.7 TB/s, and 172 backward, 5.8.  Appended, 8191
// tokens of 32 + 2 x 8 heads of 128 (201 MB): 40 us, 5.0 TB/s.  Small calls are bound by the launch (333 tokens of 20 heads of 64,
// fp32: 3.3 us in a graph; 3.9 with each lane reading its weights from device memory behind the wait for the rotation's table).
#include "fa_rope_items.cuh"

namespace fa {

using namespace rope;

namespace {

// A lane's 16 elements in fp32, as the rotation takes them: first and second elements of pairs 2j and 2j + 1.
struct Head16 {
  uint64_t x1[4], x2[4];
};

// Which of the unit's 16 elements is the first (second) one of its pair q.
template <bool INTER>
__device__ __forceinline__ constexpr int first_of(int q) {
  return INTER ? 2 * q : q;
}
template <bool INTER>
__device__ __forceinline__ constexpr int second_of(int q) {
  return INTER ? 2 * q + 1 : 8 + q;
}

template <bool INTER>
__device__ __forceinline__ Head16 unpack(const Unit<__nv_bfloat16>& u) {
  const uint32_t w[8] = {u.a.x, u.a.y, u.a.z, u.a.w, u.b.x, u.b.y, u.b.z, u.b.w};
  Head16 h;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t p = w[INTER ? 2 * j : j], q = w[INTER ? 2 * j + 1 : 4 + j];
    h.x1[j] = INTER ? f2_pack(bf16lo(p), bf16lo(q)) : f2_pack(bf16lo(p), bf16hi(p));
    h.x2[j] = INTER ? f2_pack(bf16hi(p), bf16hi(q)) : f2_pack(bf16lo(q), bf16hi(q));
  }
  return h;
}
template <bool INTER>
__device__ __forceinline__ Head16 unpack(const Unit<float>& u) {
  const uint32_t w[16] = {u.v[0].x, u.v[0].y, u.v[0].z, u.v[0].w, u.v[1].x, u.v[1].y, u.v[1].z, u.v[1].w,
                          u.v[2].x, u.v[2].y, u.v[2].z, u.v[2].w, u.v[3].x, u.v[3].y, u.v[3].z, u.v[3].w};
  Head16 h;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    h.x1[j] = f2_pack(__uint_as_float(w[first_of<INTER>(2 * j)]), __uint_as_float(w[first_of<INTER>(2 * j + 1)]));
    h.x2[j] = f2_pack(__uint_as_float(w[second_of<INTER>(2 * j)]), __uint_as_float(w[second_of<INTER>(2 * j + 1)]));
  }
  return h;
}

// The one rounding, to nearest even.
template <bool INTER>
__device__ __forceinline__ void pack(const Head16& h, Unit<__nv_bfloat16>* u) {
  uint32_t w[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float a0, a1, b0, b1;
    f2_unpack_f(h.x1[j], a0, a1);
    f2_unpack_f(h.x2[j], b0, b1);
    w[INTER ? 2 * j : j] = INTER ? pack_bf16x2(a0, b0) : pack_bf16x2(a0, a1);
    w[INTER ? 2 * j + 1 : 4 + j] = INTER ? pack_bf16x2(a1, b1) : pack_bf16x2(b0, b1);
  }
  u->a = make_uint4(w[0], w[1], w[2], w[3]);
  u->b = make_uint4(w[4], w[5], w[6], w[7]);
}
template <bool INTER>
__device__ __forceinline__ void pack(const Head16& h, Unit<float>* u) {
  uint32_t w[16];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f2_unpack(h.x1[j], w[first_of<INTER>(2 * j)], w[first_of<INTER>(2 * j + 1)]);
    f2_unpack(h.x2[j], w[second_of<INTER>(2 * j)], w[second_of<INTER>(2 * j + 1)]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) u->v[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}

// Both kinds' weights into shared memory, in fp32 (nullptr: no such heads).  Beside the rotation's table, so that both wait for
// memory once; the caller synchronises.
template <int D>
__device__ __forceinline__ void load_weights(const void* wq, const void* wk, int fp32, float (&w)[2][D]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const void* const p = k ? wk : wq;
    for (int i = threadIdx.x; i < D; i += ROPE_THREADS)
      w[k][i] = p == nullptr ? 0.f
                : fp32       ? static_cast<const float*>(p)[i]
                             : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  }
}

// Those of a lane's elements.
template <typename T, bool INTER>
__device__ __forceinline__ Head16 lane_weight(const float* w, int e0, int es) {
  constexpr int W = 16 / sizeof(T);
  const auto at = [&](int i) { return w[e0 + i / W * es + i % W]; };
  Head16 h;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    h.x1[j] = f2_pack(at(first_of<INTER>(2 * j)), at(first_of<INTER>(2 * j + 1)));
    h.x2[j] = f2_pack(at(second_of<INTER>(2 * j)), at(second_of<INTER>(2 * j + 1)));
  }
  return h;
}

// sum a b over the lane's elements
__device__ __forceinline__ float dot16(const Head16& a, const Head16& b) {
  uint64_t s = f2_mul(a.x1[0], b.x1[0]), t = f2_mul(a.x2[0], b.x2[0]);
#pragma unroll
  for (int j = 1; j < 4; ++j) {
    s = f2_fma(a.x1[j], b.x1[j], s);
    t = f2_fma(a.x2[j], b.x2[j], t);
  }
  float lo, hi;
  f2_unpack_f(f2_add(s, t), lo, hi);
  return lo + hi;
}

__device__ __forceinline__ Head16 mul16(const Head16& a, const Head16& b) {
  Head16 r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    r.x1[j] = f2_mul(a.x1[j], b.x1[j]);
    r.x2[j] = f2_mul(a.x2[j], b.x2[j]);
  }
  return r;
}

__device__ __forceinline__ void scale16(Head16& a, float f) {
  const uint64_t f2 = f2_pack(f, f);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    a.x1[j] = f2_mul(a.x1[j], f2);
    a.x2[j] = f2_mul(a.x2[j], f2);
  }
}

// The UNITS lanes of a head, which are neighbours (other heads' lanes may be elsewhere).
template <int UNITS>
__device__ __forceinline__ unsigned head_mask() {
  return ((1u << UNITS) - 1u) << ((threadIdx.x & 31) & ~(UNITS - 1));
}

__device__ __forceinline__ float inv_rms(float squares, int d, float eps) { return rsqrtf(squares * (1.f / d) + eps); }

// Sums over a head's lanes, side by side.
template <int UNITS, int N>
__device__ __forceinline__ void head_sums(float (&x)[N], unsigned mask) {
#pragma unroll
  for (int i = 1; i < UNITS; i *= 2)
#pragma unroll
    for (int k = 0; k < N; ++k) x[k] += __shfl_xor_sync(mask, x[k], i);
}

template <int UNITS>
__device__ __forceinline__ float head_sum(float x, unsigned mask) {
  float v[1] = {x};
  head_sums<UNITS>(v, mask);
  return v[0];
}

template <bool INTER, typename T>
__device__ __forceinline__ Head16 read16(const uint4* src) {
  Unit<T> x;
  x.load(src);
  return unpack<INTER>(x);
}

// The weights times a token's turn: y1 = x1 a - x2 b, y2 = x1 c + x2 d (b with its sign), the same for all of its heads.  Elements
// that are not rotated take their weight alone (a, d): with products of zero beside it an infinite element, NaN once it is normed,
// would reach another one.
struct Fold {
  uint64_t a[4], b[4], c[4], d[4];
  bool rotated;
  __device__ __forceinline__ Fold(const Head16& w, const Turn& t, bool rotated) : rotated(rotated) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a[j] = rotated ? f2_mul(w.x1[j], t.c[j]) : w.x1[j];
      b[j] = f2_mul(w.x2[j], t.n[j]);
      c[j] = f2_mul(w.x1[j], t.s[j]);
      d[j] = rotated ? f2_mul(w.x2[j], t.c[j]) : w.x2[j];
    }
  }
  __device__ __forceinline__ void apply(Head16& x) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (rotated) {
        const uint64_t y = f2_fma(x.x1[j], a[j], f2_mul(x.x2[j], b[j]));
        x.x2[j] = f2_fma(x.x1[j], c[j], f2_mul(x.x2[j], d[j]));
        x.x1[j] = y;
      } else {
        x.x1[j] = f2_mul(x.x1[j], a[j]);
        x.x2[j] = f2_mul(x.x2[j], d[j]);
      }
    }
  }
};

// The heads of one kind, of B * N tokens, and how they are cut.
struct Heads {
  const void* x;    // inputs
  const void* dy;   // backward: gradients of the outputs
  void* out;
  const void* w;
  RowStrides sx, sdy, so;
  int n;
  int first_block;  // that takes the first item
  int quad;         // up to three heads take the lanes without quads (fa_rope_items.cuh)
  Tiling g;
};
__device__ __forceinline__ int block_of(const Heads& hs) { return (blockIdx.x + gridDim.x - hs.first_block) % gridDim.x; }
__device__ __forceinline__ bool has_items(const Heads& hs) { return block_of(hs) * (ROPE_THREADS / 32) < hs.g.count; }

struct NormParams {
  Heads heads[2];   // query and key heads
  Rotary r;
  FastDiv by_n;
  float eps;
  int w_fp32, N, tokens;
  int* err;
  float* parts;     // backward
};

constexpr int FWD_SLOTS = 8, FWD_BLOCKS = 3;

// A block's items, forward.
template <typename T, int D, bool INTER, bool QUAD>
__device__ __forceinline__ void norm_items(const NormParams& p, const Heads& hs, const PairTurn* pairs, const float* weight) {
  constexpr int P = Unit<T>::PIECES, PER = FWD_SLOTS / P, STEP = Lane<D, QUAD>::STEP, UNITS = D / 16;
  int e0, es;
  const bool rotated = unit_pieces<T, D>(p.r.rot, Lane<D, QUAD>().u, &e0, &es);
  const Head16 w = lane_weight<T, INTER>(weight, e0, es);
  const unsigned mask = head_mask<UNITS>();
  run_items<T, D, INTER, QUAD, FWD_SLOTS>(
      hs.g, p.r, pairs, rotated, p.tokens, block_of(hs), gridDim.x,
      [&](int t, int h0, uint32_t dst, uint32_t) {
        const int b = p.by_n.div(t), n = t - b * p.N;
        const T* const x = static_cast<const T*>(hs.x) + b * hs.sx.b + n * hs.sx.n;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int h = h0 + STEP * i;
          if (i < hs.g.per && h < hs.n) Unit<T>::fetch(dst + i * P * 512, x + h * hs.sx.h, e0, es);
        }
        return p.r.pos + (p.r.batch_stride ? t : n);
      },
      [&](int t, int h0, const uint4* src, long long, const Turn& turn) {
        const int b = p.by_n.div(t), n = t - b * p.N;
        T* const out = static_cast<T*>(hs.out) + b * hs.so.b + n * hs.so.n;
        const Fold fold(w, turn, rotated);
#pragma unroll 1
        for (int i = 0; i < hs.g.per; ++i) {  // one head at a time: several in registers spill
          const int h = h0 + STEP * i;
          if (h >= hs.n) break;
          Head16 x = read16<INTER, T>(src + i * P * 32);
          scale16(x, inv_rms(head_sum<UNITS>(dot16(x, x), mask), D, p.eps));
          fold.apply(x);
          Unit<T> y;
          pack<INTER>(x, &y);
          y.store(out + h * hs.so.h, e0, es);
        }
      });
}

// The backward pass has as many heads an item as the forward one, from two tensors, and dw's sums in registers.  With half as
// many heads an item 97 us instead of 88; 2 blocks a SM 104, 4 (128 registers a thread, which spill) 105.
constexpr int BWD_SLOTS = 16, BWD_BLOCKS = 3;

// A block's items, backward; leaves the block's share of dw in `parts`.
template <typename T, int D, bool INTER, bool QUAD>
__device__ __forceinline__ void norm_items_bwd(const NormParams& p, const Heads& hs, const PairTurn* pairs, const float* weight,
                                               float (*share)[D], float* parts) {
  constexpr int P = Unit<T>::PIECES, PER = BWD_SLOTS / (2 * P), STEP = Lane<D, QUAD>::STEP, UNITS = D / 16;
  int e0, es;
  const bool rotated = unit_pieces<T, D>(p.r.rot, Lane<D, QUAD>().u, &e0, &es);
  const Head16 w = lane_weight<T, INTER>(weight, e0, es);
  const unsigned mask = head_mask<UNITS>();
  Head16 sum{};
  run_items<T, D, INTER, QUAD, BWD_SLOTS>(
      hs.g, p.r, pairs, rotated, p.tokens, block_of(hs), gridDim.x,
      [&](int t, int h0, uint32_t dst, uint32_t) {
        const int b = p.by_n.div(t), n = t - b * p.N;
        const T* const x = static_cast<const T*>(hs.x) + b * hs.sx.b + n * hs.sx.n;
        const T* const dy = static_cast<const T*>(hs.dy) + b * hs.sdy.b + n * hs.sdy.n;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int h = h0 + STEP * i;
          if (i < hs.g.per && h < hs.n) {
            Unit<T>::fetch(dst + 2 * i * P * 512, dy + h * hs.sdy.h, e0, es);
            Unit<T>::fetch(dst + (2 * i + 1) * P * 512, x + h * hs.sx.h, e0, es);
          }
        }
        return p.r.pos + (p.r.batch_stride ? t : n);
      },
      [&](int t, int h0, const uint4* src, long long, const Turn& turn) {
        const int b = p.by_n.div(t), n = t - b * p.N;
        T* const out = static_cast<T*>(hs.out) + b * hs.so.b + n * hs.so.n;
#pragma unroll 1
        for (int i = 0; i < hs.g.per; ++i) {
          const int h = h0 + STEP * i;
          if (h >= hs.n) break;
          Head16 gr = read16<INTER, T>(src + 2 * i * P * 32);
          if (rotated) {
#pragma unroll
            for (int j = 0; j < 4; ++j) turn.apply(j, gr.x1[j], gr.x2[j]);
          }
          Head16 u = read16<INTER, T>(src + (2 * i + 1) * P * 32);
          float s[2] = {dot16(u, u), dot16(mul16(gr, w), u)};  // sums of x^2 and of w g x
          head_sums<UNITS>(s, mask);
          const float f = inv_rms(s[0], D, p.eps), m = s[1] * (1.f / D) * f;  // mean(w g u)
          scale16(u, f);
          const uint64_t f2 = f2_pack(f, f), m2 = f2_pack(-m * f, -m * f);
          Head16 dx;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            dx.x1[j] = f2_fma(u.x1[j], m2, f2_mul(f2_mul(gr.x1[j], w.x1[j]), f2));
            dx.x2[j] = f2_fma(u.x2[j], m2, f2_mul(f2_mul(gr.x2[j], w.x2[j]), f2));
            sum.x1[j] = f2_fma(gr.x1[j], u.x1[j], sum.x1[j]);
            sum.x2[j] = f2_fma(gr.x2[j], u.x2[j], sum.x2[j]);
          }
          Unit<T> y;
          pack<INTER>(dx, &y);
          y.store(out + h * hs.so.h, e0, es);
        }
      });
  // The block's share: lanes of the same unit, then its warps, in order.
  __syncwarp();
  constexpr int W = 16 / sizeof(T);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float lo, hi, v = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if (first_of<INTER>(q) == i) f2_unpack_f(sum.x1[q / 2], lo, hi), v = q % 2 ? hi : lo;
      if (second_of<INTER>(q) == i) f2_unpack_f(sum.x2[q / 2], lo, hi), v = q % 2 ? hi : lo;
    }
#pragma unroll
    for (int step = UNITS; step < 32; step *= 2) v += __shfl_xor_sync(0xffffffffu, v, step);
    if ((threadIdx.x & 31) < UNITS) share[threadIdx.x / 32][e0 + i / W * es + i % W] = v;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < D; i += ROPE_THREADS) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < ROPE_THREADS / 32; ++k) v += share[k][i];
    parts[i] = v;
  }
  __syncthreads();  // `share` has been read
}

}  // namespace

template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(ROPE_THREADS, FWD_BLOCKS) fa_norm_rope_kernel(const __grid_constant__ NormParams p) {
  __shared__ PairTurn pairs[D / 2];
  __shared__ float weights[2][D];
  griddep_wait();
  load_rotation<D>(p.r, pairs, p.err);
  load_weights<D>(p.heads[0].w, p.heads[1].w, p.w_fp32, weights);
  __syncthreads();
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    const Heads& hs = p.heads[k];
    if (!has_items(hs)) continue;
    if (hs.quad)
      norm_items<T, D, INTER, true>(p, hs, pairs, weights[k]);
    else
      norm_items<T, D, INTER, false>(p, hs, pairs, weights[k]);
  }
}

// p.r turns by the negative angle.
template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(ROPE_THREADS, BWD_BLOCKS) fa_norm_rope_bwd_kernel(const __grid_constant__ NormParams p) {
  __shared__ PairTurn pairs[D / 2];
  __shared__ float weights[2][D];
  __shared__ float share[ROPE_THREADS / 32][D];
  griddep_launch_dependents();
  griddep_wait();
  load_rotation<D>(p.r, pairs, p.err);
  load_weights<D>(p.heads[0].w, p.heads[1].w, p.w_fp32, weights);
  __syncthreads();
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    const Heads& hs = p.heads[k];
    float* const parts = p.parts + (static_cast<long long>(blockIdx.x) * 2 + k) * D;
    if (!has_items(hs)) {
      for (int i = threadIdx.x; i < D; i += ROPE_THREADS) parts[i] = 0.f;
    } else if (hs.quad)
      norm_items_bwd<T, D, INTER, true>(p, hs, pairs, weights[k], share, parts);
    else
      norm_items_bwd<T, D, INTER, false>(p, hs, pairs, weights[k], share, parts);
  }
}

template <int D, bool INTER>
__global__ void __launch_bounds__(ROPE_THREADS, ROPE_BLOCKS) fa_norm_append_kernel(const AppendLaunch a, const HeadNorm nm,
                                                                                   const Tiling g, const FastDiv by_page) {
  using T = __nv_bfloat16;
  constexpr int P = Unit<T>::PIECES, PER = PIECE_SLOTS / P, STEP = Lane<D, true>::STEP, UNITS = D / 16;
  __shared__ PairTurn pairs[D / 2];
  __shared__ float weights[2][D];
  griddep_wait();
  load_rotation<D>(a.r, pairs, a.err);
  load_weights<D>(nm.wq, nm.wk, nm.fp32, weights);
  __syncthreads();
  const int hk = a.H, hv = a.H + a.Hkv, heads = a.H + 2 * a.Hkv;  // q, k and v heads in a row
  int e0, es;
  const bool rotated = unit_pieces<T, D>(a.r.rot, Lane<D, true>().u, &e0, &es);
  const Head16 wq = lane_weight<T, INTER>(weights[0], e0, es), wk = lane_weight<T, INTER>(weights[1], e0, es);
  const unsigned mask = head_mask<UNITS>();
  run_items<T, D, INTER, true>(
      g, a.r, pairs, rotated, a.T, blockIdx.x, gridDim.x,
      [&](int t, int h0, uint32_t dst, uint32_t slot_dst) {
        const T* const q = static_cast<const T*>(a.q) + t * a.q_tok;
        const T* const k = static_cast<const T*>(a.k) + t * a.k_tok;
        const T* const v = static_cast<const T*>(a.v) + t * a.v_tok;
        cp_async_small<8>(slot_dst, a.slots + t);
#pragma unroll
        for (int i = 0; i < PER; ++i) {  // unused places too: their slots are still on the way
          const int h = h0 + STEP * i;
          if (i < g.per && h < heads)
            Unit<T>::fetch(dst + i * P * 512,
                           h < hk ? q + h * a.q_head : h < hv ? k + (h - hk) * a.k_head : v + (h - hv) * a.v_head, e0, es);
        }
        return a.r.pos + t;
      },
      [&](int t, int h0, const uint4* src, long long slot, const Turn& turn) {
        if (slot >= a.n_slots) record_bad_index(a.err, W_SLOT);
        const bool store = slot >= 0 && slot < a.n_slots;
        const long long page = !store                     ? 0
                               : a.n_slots <= 0x7FFFFFFF ? by_page.div(static_cast<int>(slot))
                                                         : slot / a.page_size;
        const long long row = store ? page * a.c_page + (slot - page * a.page_size) * a.c_row : 0;
        T* const qo = static_cast<T*>(a.q_out) + static_cast<long long>(t) * a.H * D;
        T* const ko = static_cast<T*>(a.k_cache) + row;
        T* const vo = static_cast<T*>(a.v_cache) + row;
#pragma unroll 1
        for (int i = 0; i < g.per; ++i) {
          const int h = h0 + STEP * i;
          if (h >= heads || (h >= hk && !store)) break;
          Unit<T> x;
          x.load(src + i * P * 32);
          if (h < hv) {
            Head16 y = unpack<INTER>(x);
            scale16(y, inv_rms(head_sum<UNITS>(dot16(y, y), mask), D, nm.eps));
            y = mul16(y, h < hk ? wq : wk);
            if (rotated) {
#pragma unroll
              for (int j = 0; j < 4; ++j) turn.apply(j, y.x1[j], y.x2[j]);
            }
            pack<INTER>(y, &x);
          }
          x.store(h < hk ? qo + h * D : h < hv ? ko + (h - hk) * a.c_head : vo + (h - hv) * a.c_head, e0, es);
        }
      });
}

// dw = the blocks' shares, added in a fixed order: a block has 32 elements, each warp every 8th share.
__global__ void __launch_bounds__(256) fa_norm_rope_join_kernel(const float* parts, int n, int d, float* dwq,
                                                                float* dwk) {
  __shared__ float sum[8][32];
  griddep_wait();
  const int i = blockIdx.x * 32 + threadIdx.x % 32, w = threadIdx.x / 32;
  const bool k = blockIdx.y > 0;
  float v = 0.f;
#pragma unroll 8
  for (int p = w; p < n; p += 8) v += parts[(static_cast<long long>(p) * 2 + k) * d + i];
  sum[w][threadIdx.x % 32] = v;
  __syncthreads();
  if (w > 0) return;
#pragma unroll
  for (int j = 1; j < 8; ++j) v += sum[j][threadIdx.x];
  (k ? dwk : dwq)[i] = v;
}

namespace {

// The parameters of both directions, for items of up to `most` heads a lane and `blocks_sm` blocks a SM.
template <typename T, int D>
cudaError_t norm_params(const RopeLaunch& a, const HeadNorm& nm, int most, int blocks_sm, NormParams* p, unsigned* grid) {
  const long long tokens = static_cast<long long>(a.B) * a.N;
  const long long warps = static_cast<long long>(a.sms) * blocks_sm * (ROPE_THREADS / 32);
  long long items = 0;
  for (int k = 0; k < 2; ++k) {
    Heads& h = p->heads[k];
    h.x = k ? a.k : a.q;
    h.out = k ? a.k_out : a.q_out;
    h.w = k ? nm.wk : nm.wq;
    h.sx = k ? a.sk : a.sq;
    h.so = k ? a.sko : a.sqo;
    h.n = k ? a.Hkv : a.H;
    h.quad = h.n > 3;
    h.first_block = static_cast<int>(items);  // for now
    if (h.n == 0) continue;
    unsigned blocks = 0;
    const long long share = warps * h.n / (a.H + a.Hkv);
    const cudaError_t e = h.quad ? cut_items(tokens, h.n, most, share, Lane<D, true>::STEP, Lane<D, true>::TOKS, &h.g, &blocks)
                                 : cut_items(tokens, h.n, most, share, Lane<D, false>::STEP, Lane<D, false>::TOKS, &h.g, &blocks);
    if (e != cudaSuccess) return e;
    items += h.g.count;
  }
  const int per_block = ROPE_THREADS / 32;
  *grid = static_cast<unsigned>(((items < warps ? items : warps) + per_block - 1) / per_block);
  p->heads[1].first_block = static_cast<int>(p->heads[0].g.count / per_block % *grid);  // behind the query heads' last item
  p->r = a.r;
  p->by_n = FastDiv(static_cast<unsigned>(a.N));
  p->eps = nm.eps;
  p->w_fp32 = nm.fp32;
  p->N = a.N;
  p->tokens = static_cast<int>(tokens);
  p->err = a.err;
  return cudaSuccess;
}

template <typename T, int D>
cudaError_t launch_norm_d(const RopeLaunch& a, const HeadNorm& nm) {
  NormParams p = {};
  unsigned grid = 0;
  const cudaError_t e = norm_params<T, D>(a, nm, FWD_SLOTS / Unit<T>::PIECES, FWD_BLOCKS, &p, &grid);
  if (e != cudaSuccess) return e;
  return a.r.interleaved ? launch_items<fa_norm_rope_kernel<T, D, true>, FWD_SLOTS>(grid, a.stream, p)
                         : launch_items<fa_norm_rope_kernel<T, D, false>, FWD_SLOTS>(grid, a.stream, p);
}

template <typename T, int D>
cudaError_t launch_bwd_d(const RopeLaunch& a, const NormBwd& b, const HeadNorm& nm) {
  NormParams p = {};
  unsigned grid = 0;
  cudaError_t e = norm_params<T, D>(a, nm, BWD_SLOTS / (2 * Unit<T>::PIECES), BWD_BLOCKS, &p, &grid);
  if (e != cudaSuccess) return e;
  if (static_cast<int>(grid) > norm_bwd_parts(a.sms)) return cudaErrorInvalidValue;  // the workspace's room
  for (int k = 0; k < 2; ++k) {
    Heads& h = p.heads[k];
    h.dy = h.x;
    h.sdy = h.sx;
    h.x = k ? b.k : b.q;
    h.sx = k ? b.sk : b.sq;
  }
  p.parts = b.parts;
  e = a.r.interleaved ? launch_items<fa_norm_rope_bwd_kernel<T, D, true>, BWD_SLOTS>(grid, a.stream, p)
                      : launch_items<fa_norm_rope_bwd_kernel<T, D, false>, BWD_SLOTS>(grid, a.stream, p);
  if (e != cudaSuccess) return e;
  return launch_dependent(fa_norm_rope_join_kernel, dim3(D / 32, a.Hkv > 0 ? 2 : 1), 256, 0, a.stream,
                          static_cast<const float*>(b.parts), static_cast<int>(grid), D, b.dwq, b.dwk);
}

template <int D>
cudaError_t launch_norm_append_d(const AppendLaunch& a, const HeadNorm& nm) {
  Tiling g;
  unsigned grid = 0;
  const cudaError_t e = tile<__nv_bfloat16, D, true>(a.T, a.H + 2 * a.Hkv, a.sms, &g, &grid);
  if (e != cudaSuccess) return e;
  const FastDiv by_page(static_cast<unsigned>(a.page_size));
  return a.r.interleaved ? launch_items<fa_norm_append_kernel<D, true>>(grid, a.stream, a, nm, g, by_page)
                         : launch_items<fa_norm_append_kernel<D, false>>(grid, a.stream, a, nm, g, by_page);
}

}  // namespace

cudaError_t launch_norm_rope(const RopeLaunch& a, const HeadNorm& nm) {
  using bf = __nv_bfloat16;
  if (a.bf16) return a.d == 64 ? launch_norm_d<bf, 64>(a, nm) : launch_norm_d<bf, 128>(a, nm);
  return a.d == 64 ? launch_norm_d<float, 64>(a, nm) : launch_norm_d<float, 128>(a, nm);
}

cudaError_t launch_norm_append(const AppendLaunch& a, const HeadNorm& nm) {
  return a.d == 64 ? launch_norm_append_d<64>(a, nm) : launch_norm_append_d<128>(a, nm);
}

int norm_bwd_parts(int sms) { return sms * BWD_BLOCKS; }

cudaError_t launch_norm_rope_bwd(const RopeLaunch& a, const NormBwd& b, const HeadNorm& nm) {
  using bf = __nv_bfloat16;
  if (a.bf16) return a.d == 64 ? launch_bwd_d<bf, 64>(a, b, nm) : launch_bwd_d<bf, 128>(a, b, nm);
  return a.d == 64 ? launch_bwd_d<float, 64>(a, b, nm) : launch_bwd_d<float, 128>(a, b, nm);
}

}  // namespace fa
