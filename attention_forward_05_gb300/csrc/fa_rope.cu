// fa_rope.cu -- rotary positions: on dense q and k (and on their gradients), and on the keys and queries
// of new tokens as they are appended to a paged key/value cache.
//
// Mathematics.  The first `rot` elements of a head form rot/2 pairs (x1, x2); pair i belongs to a position
// axis a(i) and turns by the angle phi = pos[a(i)] * f_i:
//   y1 = x1 cos phi - x2 sin phi,   y2 = x1 sin phi + x2 cos phi.
// The rotation is orthogonal, so its backward pass is the rotation by -phi.
//
// Angles, items and the cut into them: fa_rope_items.cuh.
//
// Both kernels are bound by device memory (each element is read once and written once) as long as the instructions
// are few: the products go in packed fp32 pairs.  Measured, bytes read and written over the time with the launch (about
// 3 us): q and k of 4 x 4096 tokens, 32 heads of 64, bf16: 23.8 us, 5.6 TB/s; 2 x 8192 tokens, 20 heads of 128, three
// axes, adjacent pairs: 29 us, 5.8 TB/s; appending 8191 tokens, 48 heads of 128: 34.7 us, 5.8 TB/s; 333 tokens, 20 heads
// of 64, fp32: 2.9 us.  With register loads of the current item, each block on one contiguous range: 26.3, 31.1, 36.3
// and 3.2 us; with adjacent pairs' 32 bytes a lane in two half-sector copies instead of pieces: 32.0 and 37.6 us for the
// second and third.  Two items ahead measured the same or up to 5 % more.
#include "fa_rope_items.cuh"

namespace fa {

using namespace rope;

template <typename T, int D, bool INTER, bool QUAD>
__global__ void __launch_bounds__(ROPE_THREADS, ROPE_BLOCKS) fa_rope_kernel(const RopeLaunch a, const Tiling g,
                                                                            const FastDiv by_n) {
  constexpr int PER = PIECE_SLOTS / Unit<T>::PIECES, STEP = Lane<D, QUAD>::STEP;
  __shared__ PairTurn pairs[D / 2];
  griddep_wait();
  load_rotation<D>(a.r, pairs, a.err);
  __syncthreads();
  const int tokens = a.B * a.N, heads = a.H + a.Hkv;
  int e0, es;
  const bool rotated = unit_pieces<T, D>(a.r.rot, Lane<D, QUAD>().u, &e0, &es);
  run_items<T, D, INTER, QUAD>(
      g, a.r, pairs, rotated, tokens, blockIdx.x, gridDim.x,
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
            if (rotated) x.template turn<INTER>(turn);
            x.store(h < a.H ? qo + h * a.sqo.h : ko + (h - a.H) * a.sko.h, e0, es);
          }
        }
      });
}

template <int D, bool INTER>
__global__ void __launch_bounds__(ROPE_THREADS, ROPE_BLOCKS) fa_paged_append_kernel(const AppendLaunch a, const Tiling g,
                                                                                    const FastDiv by_page) {
  using T = __nv_bfloat16;
  constexpr int PER = PIECE_SLOTS / Unit<T>::PIECES, STEP = Lane<D, true>::STEP;
  __shared__ PairTurn pairs[D / 2];
  griddep_wait();
  load_rotation<D>(a.r, pairs, a.err);
  __syncthreads();
  const int hk = a.H, hv = a.H + a.Hkv, heads = a.H + 2 * a.Hkv;  // q, k and v heads in a row
  int e0, es;
  const bool rotated = unit_pieces<T, D>(a.r.rot, Lane<D, true>().u, &e0, &es);
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
            if (rotated && h < hv) x.template turn<INTER>(turn);
            x.store(h < hk ? qo + h * D : h < hv ? ko + (h - hk) * a.c_head : vo + (h - hv) * a.c_head, e0, es);
          }
        }
      });
}

template <typename T, int D, bool QUAD>
static cudaError_t launch_rope_q(const RopeLaunch& a) {
  Tiling g;
  unsigned grid = 0;
  const long long tokens = static_cast<long long>(a.B) * a.N;
  const cudaError_t e = tile<T, D, QUAD>(tokens, a.H + a.Hkv, a.sms, &g, &grid);
  if (e != cudaSuccess) return e;
  const FastDiv by_n(static_cast<unsigned>(a.N));
  return a.r.interleaved ? launch_items<fa_rope_kernel<T, D, true, QUAD>>(grid, a.stream, a, g, by_n)
                         : launch_items<fa_rope_kernel<T, D, false, QUAD>>(grid, a.stream, a, g, by_n);
}

template <typename T>
static cudaError_t launch_rope_t(const RopeLaunch& a) {
  if (a.H + a.Hkv > 3) return a.d == 64 ? launch_rope_q<T, 64, true>(a) : launch_rope_q<T, 128, true>(a);
  return a.d == 64 ? launch_rope_q<T, 64, false>(a) : launch_rope_q<T, 128, false>(a);
}

cudaError_t launch_rope(const RopeLaunch& a) {
  return a.bf16 ? launch_rope_t<__nv_bfloat16>(a) : launch_rope_t<float>(a);
}

template <int D>
static cudaError_t launch_append_d(const AppendLaunch& a) {
  Tiling g;
  unsigned grid = 0;
  const cudaError_t e = tile<__nv_bfloat16, D, true>(a.T, a.H + 2 * a.Hkv, a.sms, &g, &grid);
  if (e != cudaSuccess) return e;
  const FastDiv by_page(static_cast<unsigned>(a.page_size));
  return a.r.interleaved ? launch_items<fa_paged_append_kernel<D, true>>(grid, a.stream, a, g, by_page)
                         : launch_items<fa_paged_append_kernel<D, false>>(grid, a.stream, a, g, by_page);
}

cudaError_t launch_append(const AppendLaunch& a) { return a.d == 64 ? launch_append_d<64>(a) : launch_append_d<128>(a); }

}  // namespace fa
