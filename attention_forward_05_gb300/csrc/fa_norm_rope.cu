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
// two or three shuffles; everything between the load and the store stays in registers, in fp32, rounded once.  The
// weights of a lane's elements stay in its registers.  The backward pass copies dy and x of half as many heads an item;
// a lane adds up its elements' share of dw over all its items, a block joins its lanes' shares in a fixed order and
// leaves them in the workspace, and fa_norm_rope_join_kernel adds the blocks' (no atomics: the same bits every time).
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

// The weights of a lane's elements (nullptr: no such heads).
template <typename T, bool INTER>
__device__ __forceinline__ Head16 load_weight(const void* p, int fp32, int e0, int es) {
  constexpr int W = 16 / sizeof(T);
  const auto at = [&](int i) {
    const int e = e0 + i / W * es + i % W;
    if (p == nullptr) return 0.f;
    return fp32 ? static_cast<const float*>(p)[e] : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[e]);
  };
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

// Sum over the UNITS lanes of a head, which are neighbours; `mask` is theirs (other heads' lanes may be elsewhere).
template <int UNITS>
__device__ __forceinline__ float head_sum(float x, unsigned mask) {
#pragma unroll
  for (int i = 1; i < UNITS; i *= 2) x += __shfl_xor_sync(mask, x, i);
  return x;
}

template <int UNITS>
__device__ __forceinline__ unsigned head_mask() {
  return ((1u << UNITS) - 1u) << ((threadIdx.x & 31) & ~(UNITS - 1));
}

__device__ __forceinline__ float inv_rms(float squares, int d, float eps) { return rsqrtf(squares * (1.f / d) + eps); }

// Norms, rotates and rounds a head's 16 elements.
template <typename T, int D, bool INTER>
__device__ __forceinline__ void norm_turn(Unit<T>* x, const Head16& w, float eps, bool rotated, const Turn& turn,
                                          unsigned mask) {
  Head16 h = unpack<INTER>(*x);
  const float r = inv_rms(head_sum<D / 16>(dot16(h, h), mask), D, eps);
  scale16(h, r);
  h = mul16(h, w);
  if (rotated) {
#pragma unroll
    for (int j = 0; j < 4; ++j) turn.apply(j, h.x1[j], h.x2[j]);
  }
  pack<INTER>(h, x);
}

}  // namespace

template <typename T, int D, bool INTER, bool QUAD>
__global__ void __launch_bounds__(ROPE_THREADS, ROPE_BLOCKS) fa_norm_rope_kernel(const RopeLaunch a, const HeadNorm nm,
                                                                                 const Tiling g, const FastDiv by_n) {
  constexpr int PER = PIECE_SLOTS / Unit<T>::PIECES, STEP = Lane<D, QUAD>::STEP;
  __shared__ PairTurn pairs[D / 2];
  griddep_wait();
  load_rotation<D>(a.r, pairs, a.err);
  __syncthreads();
  const int tokens = a.B * a.N, heads = a.H + a.Hkv;
  int e0, es;
  const bool rotated = unit_pieces<T, D>(a.r.rot, Lane<D, QUAD>().u, &e0, &es);
  const Head16 wq = load_weight<T, INTER>(nm.wq, nm.fp32, e0, es), wk = load_weight<T, INTER>(nm.wk, nm.fp32, e0, es);
  const unsigned mask = head_mask<D / 16>();
  run_items<T, D, INTER, QUAD>(
      g, a.r, pairs, rotated, tokens,
      [&](int t, int h0, uint32_t dst, uint32_t) {
        const int b = by_n.div(t), n = t - b * a.N;
        const T* const q = static_cast<const T*>(a.q) + b * a.sq.b + n * a.sq.n;
        const T* const k = static_cast<const T*>(a.k) + b * a.sk.b + n * a.sk.n;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int h = h0 + STEP * i;
          if (i < g.per && h < heads)
            Unit<T>::fetch(dst + i * Unit<T>::PIECES * 512, h < a.H ? q + h * a.sq.h : k + (h - a.H) * a.sk.h, e0, es);
        }
        return a.r.pos + (a.r.batch_stride ? t : n);
      },
      [&](int t, int h0, const uint4* src, long long, const Turn& turn) {
        const int b = by_n.div(t), n = t - b * a.N;
        T* const qo = static_cast<T*>(a.q_out) + b * a.sqo.b + n * a.sqo.n;
        T* const ko = static_cast<T*>(a.k_out) + b * a.sko.b + n * a.sko.n;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int h = h0 + STEP * i;
          if (i < g.per && h < heads) {
            Unit<T> x;
            x.load(src + i * Unit<T>::PIECES * 32);
            norm_turn<T, D, INTER>(&x, h < a.H ? wq : wk, nm.eps, rotated, turn, mask);
            x.store(h < a.H ? qo + h * a.sqo.h : ko + (h - a.H) * a.sko.h, e0, es);
          }
        }
      });
}

template <int D, bool INTER>
__global__ void __launch_bounds__(ROPE_THREADS, ROPE_BLOCKS) fa_norm_append_kernel(const AppendLaunch a, const HeadNorm nm,
                                                                                   const Tiling g, const FastDiv by_page) {
  using T = __nv_bfloat16;
  constexpr int PER = PIECE_SLOTS / Unit<T>::PIECES, STEP = Lane<D, true>::STEP;
  __shared__ PairTurn pairs[D / 2];
  griddep_wait();
  load_rotation<D>(a.r, pairs, a.err);
  __syncthreads();
  const int hk = a.H, hv = a.H + a.Hkv, heads = a.H + 2 * a.Hkv;  // q, k and v heads in a row
  int e0, es;
  const bool rotated = unit_pieces<T, D>(a.r.rot, Lane<D, true>().u, &e0, &es);
  const Head16 wq = load_weight<T, INTER>(nm.wq, nm.fp32, e0, es), wk = load_weight<T, INTER>(nm.wk, nm.fp32, e0, es);
  const unsigned mask = head_mask<D / 16>();
  run_items<T, D, INTER, true>(
      g, a.r, pairs, rotated, a.T,
      [&](int t, int h0, uint32_t dst, uint32_t slot_dst) {
        const T* const q = static_cast<const T*>(a.q) + t * a.q_tok;
        const T* const k = static_cast<const T*>(a.k) + t * a.k_tok;
        const T* const v = static_cast<const T*>(a.v) + t * a.v_tok;
        cp_async_small<8>(slot_dst, a.slots + t);
#pragma unroll
        for (int i = 0; i < PER; ++i) {  // unused places too: their slots are still on the way
          const int h = h0 + STEP * i;
          if (i < g.per && h < heads)
            Unit<T>::fetch(dst + i * Unit<T>::PIECES * 512,
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
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int h = h0 + STEP * i;
          if (i < g.per && h < heads && (h < hk || store)) {
            Unit<T> x;
            x.load(src + i * Unit<T>::PIECES * 32);
            if (h < hv) norm_turn<T, D, INTER>(&x, h < hk ? wq : wk, nm.eps, rotated, turn, mask);
            x.store(h < hk ? qo + h * D : h < hv ? ko + (h - hk) * a.c_head : vo + (h - hv) * a.c_head, e0, es);
          }
        }
      });
}

// a.q, a.k: the outputs' gradients; b: the forward pass's inputs; a.r turns by the negative angle.
template <typename T, int D, bool INTER, bool QUAD>
__global__ void __launch_bounds__(ROPE_THREADS, ROPE_BLOCKS)
    fa_norm_rope_bwd_kernel(const RopeLaunch a, const NormBwd b, const HeadNorm nm, const Tiling g, const FastDiv by_n) {
  constexpr int P = Unit<T>::PIECES, PER = PIECE_SLOTS / (2 * P), STEP = Lane<D, QUAD>::STEP, UNITS = D / 16;
  __shared__ PairTurn pairs[D / 2];
  __shared__ float share[ROPE_THREADS / 32][2][D];
  griddep_launch_dependents();
  griddep_wait();
  load_rotation<D>(a.r, pairs, a.err);
  __syncthreads();
  const int tokens = a.B * a.N, heads = a.H + a.Hkv;
  int e0, es;
  const int u = Lane<D, QUAD>().u, lane = threadIdx.x & 31;
  const bool rotated = unit_pieces<T, D>(a.r.rot, u, &e0, &es);
  // Weights in shared memory, a unit's 16 bytes beside the next unit's: in registers, with dw's sums there, they spill.
  __shared__ ulonglong2 weights[2][4][UNITS];
  if (threadIdx.x < UNITS) {  // lane u of the first warp has unit u
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const Head16 w = load_weight<T, INTER>(which ? nm.wk : nm.wq, nm.fp32, e0, es);
#pragma unroll
      for (int j = 0; j < 4; ++j) weights[which][j][u] = make_ulonglong2(w.x1[j], w.x2[j]);
    }
  }
  __syncthreads();
  const unsigned mask = head_mask<UNITS>();
  Head16 sq{}, sk{};
  run_items<T, D, INTER, QUAD>(
      g, a.r, pairs, rotated, tokens,
      [&](int t, int h0, uint32_t dst, uint32_t) {
        const int bi = by_n.div(t), n = t - bi * a.N;
        const T* const dq = static_cast<const T*>(a.q) + bi * a.sq.b + n * a.sq.n;
        const T* const dk = static_cast<const T*>(a.k) + bi * a.sk.b + n * a.sk.n;
        const T* const q = static_cast<const T*>(b.q) + bi * b.sq.b + n * b.sq.n;
        const T* const k = static_cast<const T*>(b.k) + bi * b.sk.b + n * b.sk.n;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int h = h0 + STEP * i;
          if (i < g.per && h < heads) {
            Unit<T>::fetch(dst + 2 * i * P * 512, h < a.H ? dq + h * a.sq.h : dk + (h - a.H) * a.sk.h, e0, es);
            Unit<T>::fetch(dst + (2 * i + 1) * P * 512, h < a.H ? q + h * b.sq.h : k + (h - a.H) * b.sk.h, e0, es);
          }
        }
        return a.r.pos + (a.r.batch_stride ? t : n);
      },
      [&](int t, int h0, const uint4* src, long long, const Turn& turn) {
        const int bi = by_n.div(t), n = t - bi * a.N;
        T* const qo = static_cast<T*>(a.q_out) + bi * a.sqo.b + n * a.sqo.n;
        T* const ko = static_cast<T*>(a.k_out) + bi * a.sko.b + n * a.sko.n;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int h = h0 + STEP * i;
          if (i < g.per && h < heads) {
            Unit<T> y, x;
            y.load(src + 2 * i * P * 32);
            x.load(src + (2 * i + 1) * P * 32);
            Head16 dy = unpack<INTER>(y);
            const Head16 hx = unpack<INTER>(x);
            if (rotated) {
#pragma unroll
              for (int j = 0; j < 4; ++j) turn.apply(j, dy.x1[j], dy.x2[j]);
            }
            Head16 wg;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const ulonglong2 w = weights[h >= a.H][j][u];
              wg.x1[j] = f2_mul(dy.x1[j], w.x);
              wg.x2[j] = f2_mul(dy.x2[j], w.y);
            }
            const float r = inv_rms(head_sum<UNITS>(dot16(hx, hx), mask), D, nm.eps);
            const float m = head_sum<UNITS>(dot16(wg, hx), mask) * (1.f / D) * r * r;  // mean(w g u) r
            const uint64_t r2 = f2_pack(r, r), m2 = f2_pack(-m * r, -m * r);
            Head16 dx;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              dx.x1[j] = f2_fma(hx.x1[j], m2, f2_mul(wg.x1[j], r2));
              dx.x2[j] = f2_fma(hx.x2[j], m2, f2_mul(wg.x2[j], r2));
            }
            if (h < a.H) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                sq.x1[j] = f2_fma(dy.x1[j], f2_mul(hx.x1[j], r2), sq.x1[j]);
                sq.x2[j] = f2_fma(dy.x2[j], f2_mul(hx.x2[j], r2), sq.x2[j]);
              }
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                sk.x1[j] = f2_fma(dy.x1[j], f2_mul(hx.x1[j], r2), sk.x1[j]);
                sk.x2[j] = f2_fma(dy.x2[j], f2_mul(hx.x2[j], r2), sk.x2[j]);
              }
            }
            Unit<T> o;
            pack<INTER>(dx, &o);
            o.store(h < a.H ? qo + h * a.sqo.h : ko + (h - a.H) * a.sko.h, e0, es);
          }
        }
      });
  // The block's share: lanes of the same unit, then its warps, in order.
  __syncwarp();
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const Head16& s = which ? sk : sq;
    constexpr int W = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float lo, hi, v = 0.f;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (first_of<INTER>(q) == i) f2_unpack_f(s.x1[q / 2], lo, hi), v = q % 2 ? hi : lo;
        if (second_of<INTER>(q) == i) f2_unpack_f(s.x2[q / 2], lo, hi), v = q % 2 ? hi : lo;
      }
#pragma unroll
      for (int step = UNITS; step < 32; step *= 2) v += __shfl_xor_sync(0xffffffffu, v, step);
      if (lane < UNITS) share[threadIdx.x / 32][which][e0 + i / W * es + i % W] = v;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += ROPE_THREADS) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < ROPE_THREADS / 32; ++w) v += share[w][i / D][i % D];
    b.parts[static_cast<long long>(blockIdx.x) * 2 * D + i] = v;
  }
}

// dw = the blocks' shares, added in a fixed order: a block has 32 elements, each warp every 8th share.
__global__ void __launch_bounds__(256) fa_norm_rope_join_kernel(const float* parts, int n, int d, float* dwq, float* dwk) {
  __shared__ float sum[8][32];
  griddep_wait();
  const int i = blockIdx.x * 32 + threadIdx.x % 32, w = threadIdx.x / 32;
  float v = 0.f;
#pragma unroll 8
  for (int p = w; p < n; p += 8) v += parts[static_cast<long long>(p) * 2 * d + i];
  sum[w][threadIdx.x % 32] = v;
  __syncthreads();
  if (w > 0) return;
#pragma unroll
  for (int k = 1; k < 8; ++k) v += sum[k][threadIdx.x];
  float* const out = i < d ? dwq : dwk;
  if (out != nullptr) out[i < d ? i : i - d] = v;
}

template <typename T, int D, bool QUAD>
static cudaError_t launch_norm_q(const RopeLaunch& a, const HeadNorm& nm) {
  Tiling g;
  unsigned grid = 0;
  const long long tokens = static_cast<long long>(a.B) * a.N;
  const cudaError_t e = tile<T, D, QUAD>(tokens, a.H + a.Hkv, a.sms, &g, &grid);
  if (e != cudaSuccess) return e;
  const FastDiv by_n(static_cast<unsigned>(a.N));
  return a.r.interleaved ? launch_items<fa_norm_rope_kernel<T, D, true, QUAD>>(grid, a.stream, a, nm, g, by_n)
                         : launch_items<fa_norm_rope_kernel<T, D, false, QUAD>>(grid, a.stream, a, nm, g, by_n);
}

template <typename T>
static cudaError_t launch_norm_t(const RopeLaunch& a, const HeadNorm& nm) {
  if (a.H + a.Hkv > 3) return a.d == 64 ? launch_norm_q<T, 64, true>(a, nm) : launch_norm_q<T, 128, true>(a, nm);
  return a.d == 64 ? launch_norm_q<T, 64, false>(a, nm) : launch_norm_q<T, 128, false>(a, nm);
}

cudaError_t launch_norm_rope(const RopeLaunch& a, const HeadNorm& nm) {
  return a.bf16 ? launch_norm_t<__nv_bfloat16>(a, nm) : launch_norm_t<float>(a, nm);
}

template <int D>
static cudaError_t launch_norm_append_d(const AppendLaunch& a, const HeadNorm& nm) {
  Tiling g;
  unsigned grid = 0;
  const cudaError_t e = tile<__nv_bfloat16, D, true>(a.T, a.H + 2 * a.Hkv, a.sms, &g, &grid);
  if (e != cudaSuccess) return e;
  const FastDiv by_page(static_cast<unsigned>(a.page_size));
  return a.r.interleaved ? launch_items<fa_norm_append_kernel<D, true>>(grid, a.stream, a, nm, g, by_page)
                         : launch_items<fa_norm_append_kernel<D, false>>(grid, a.stream, a, nm, g, by_page);
}

cudaError_t launch_norm_append(const AppendLaunch& a, const HeadNorm& nm) {
  return a.d == 64 ? launch_norm_append_d<64>(a, nm) : launch_norm_append_d<128>(a, nm);
}

int norm_bwd_parts(int sms) { return sms * ROPE_BLOCKS; }

template <typename T, int D, bool QUAD>
static cudaError_t launch_bwd_q(const RopeLaunch& a, const NormBwd& b, const HeadNorm& nm) {
  Tiling g;
  unsigned grid = 0;
  const long long tokens = static_cast<long long>(a.B) * a.N;
  cudaError_t e = tile<T, D, QUAD, 2>(tokens, a.H + a.Hkv, a.sms, &g, &grid);
  if (e != cudaSuccess) return e;
  if (static_cast<int>(grid) > norm_bwd_parts(a.sms)) return cudaErrorInvalidValue;  // the workspace's room
  const FastDiv by_n(static_cast<unsigned>(a.N));
  e = a.r.interleaved ? launch_items<fa_norm_rope_bwd_kernel<T, D, true, QUAD>>(grid, a.stream, a, b, nm, g, by_n)
                      : launch_items<fa_norm_rope_bwd_kernel<T, D, false, QUAD>>(grid, a.stream, a, b, nm, g, by_n);
  if (e != cudaSuccess) return e;
  return launch_dependent(fa_norm_rope_join_kernel, dim3(2 * D / 32), 256, 0, a.stream, static_cast<const float*>(b.parts),
                          static_cast<int>(grid), D, b.dwq, b.dwk);
}

template <typename T>
static cudaError_t launch_bwd_t(const RopeLaunch& a, const NormBwd& b, const HeadNorm& nm) {
  if (a.H + a.Hkv > 3) return a.d == 64 ? launch_bwd_q<T, 64, true>(a, b, nm) : launch_bwd_q<T, 128, true>(a, b, nm);
  return a.d == 64 ? launch_bwd_q<T, 64, false>(a, b, nm) : launch_bwd_q<T, 128, false>(a, b, nm);
}

cudaError_t launch_norm_rope_bwd(const RopeLaunch& a, const NormBwd& b, const HeadNorm& nm) {
  return a.bf16 ? launch_bwd_t<__nv_bfloat16>(a, b, nm) : launch_bwd_t<float>(a, b, nm);
}

}  // namespace fa
