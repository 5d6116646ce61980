// fa_rope.cu -- rotary positions: on dense q and k (and on their gradients), and on the keys and queries
// of new tokens as they are appended to a paged key/value cache.
//
// Mathematics.  The first `rot` elements of a head form rot/2 pairs (x1, x2); pair i belongs to a position
// axis a(i) and turns by the angle phi = pos[a(i)] * f_i:
//   y1 = x1 cos phi - x2 sin phi,   y2 = x1 sin phi + x2 cos phi.
// The rotation is orthogonal, so its backward pass is the rotation by -phi.
//
// Angles.  pos * f_i in fp32 is off by pos * f_i * 2^-24 rad: 0.06 rad at position 10^6.  Only the angle's
// fraction of a turn matters, and that is exact in integers: f_i / (2 pi) modulo 1 is held as a 64-bit
// fraction F_i (units of 2^-64 turns), and pos * F_i modulo 2^64 is the phase of any 32-bit position, of
// either sign, with no range reduction.  F_i carries double precision's roundings of 1 / (2 pi) and of f_i / (2 pi)
// (2^-52 f_i rad together; a negative f_i's fraction is rounded once more, by 2^-54 turns), so the angle at position p is
// off by at most |p f_i| 2^-52 rad.  Its upper 32 bits split into the nearest quarter turn and a rest of at most an
// eighth, whose sine and cosine are Taylor polynomials (to x^9 and x^10: 2e-9 and 1e-10 off at pi/4); with the rest's
// and their own roundings in fp32 they are within 1.9e-7.  The F_i take four double-precision
// operations each and are formed once per block in shared memory (double precision runs at about two
// operations a clock and SM here).
//
// Work split.  A lane owns a unit of a head, eight pairs, in pieces of 16 bytes that lie next to its neighbours' pieces.  A
// warp's items are a few tokens with up to 16 heads each; their bytes arrive by asynchronous copies in a ring of the
// warp's own, an item ahead, with the positions (and slots) they need, so nothing waits for a load and no warp
// waits for another.  Four lanes hold the same unit of four heads and form two of its pairs' sines and cosines each.
// Consecutive items go to consecutive warps, so the whole GPU reads and writes in few places of device memory.
//
// Both kernels are bound by device memory (each element is read once and written once) as long as the instructions
// are few: the products go in packed fp32 pairs.  Measured, bytes read and written over the time with the launch (about
// 3 us): q and k of 4 x 4096 tokens, 32 heads of 64, bf16: 23.8 us, 5.6 TB/s; 2 x 8192 tokens, 20 heads of 128, three
// axes, adjacent pairs: 29 us, 5.8 TB/s; appending 8191 tokens, 48 heads of 128: 34.7 us, 5.8 TB/s; 333 tokens, 20 heads
// of 64, fp32: 2.9 us.  With register loads of the current item, each block on one contiguous range: 26.3, 31.1, 36.3
// and 3.2 us; with adjacent pairs' 32 bytes a lane in two half-sector copies instead of pieces: 32.0 and 37.6 us for the
// second and third.  Two items ahead measured the same or up to 5 % more.
#include <cuda_bf16.h>

#include "fa_internal.h"
#include "sm103_ptx.cuh"

namespace fa {

namespace {

constexpr int ROPE_THREADS = 128;
constexpr int ROPE_BLOCKS = 4;  // per SM, at most
enum : int { W_AXIS = 0x20, W_SLOT };  // sites recorded with DEV_BAD_INDEX

// F_i: radians per position as a 64-bit fraction of a turn.
__device__ __forceinline__ unsigned long long turn_fraction(double f) {
  double t = f * 0.15915494309189533577;  // 1 / (2 pi)
  t -= floor(t);
  return __double2ull_rn(t * 18446744073709551616.0);  // t in [0, 1]; 1 saturates, 2^-64 below a whole turn
}

// A pair's F_i and axis (255: out of range, the pair becomes NaN).
struct alignas(16) PairTurn {
  unsigned long long step;
  int axis, pad;
};

// Fills the block's table.  The caller synchronises.
template <int D>
__device__ __forceinline__ void load_rotation(const Rotary& r, PairTurn (&pairs)[D / 2], int* err) {
  for (int i = threadIdx.x; i < r.rot / 2; i += ROPE_THREADS) {
    int a = r.axes != nullptr ? r.axes[i] : 0;
    if (a < 0 || a >= r.n_axes) {
      record_bad_index(err, W_AXIS);
      a = 255;
    }
    pairs[i] = PairTurn{turn_fraction(r.freqs[i]), a, 0};
  }
}

// cos and sin of pos * step / 2^64 turns.
__device__ __forceinline__ void turn_sincos(int pos, unsigned long long step, float* cs, float* sn) {
  const unsigned lo = static_cast<unsigned>(step), up = static_cast<unsigned>(pos);
  unsigned ph = __umulhi(up, lo) + up * static_cast<unsigned>(step >> 32);
  if (pos < 0) ph -= lo;  // up is pos + 2^32
  const unsigned quarter = (ph + 0x20000000u) >> 30;
  const float x = static_cast<float>(static_cast<int>(ph - (quarter << 30))) * 1.4629180792671596e-9f;  // 2 pi / 2^32
  const float z = x * x;
  float s = fmaf(z, 2.7557319e-6f, -1.9841270e-4f);  // 1/9!, 1/7!, 1/5!, 1/3!
  s = fmaf(z, s, 8.3333333e-3f);
  s = fmaf(z, s, -1.6666667e-1f);
  s = fmaf(x * z, s, x);
  float c = fmaf(z, -2.7557319e-7f, 2.4801587e-5f);  // 1/10!, 1/8!, 1/6!, 1/4!, 1/2!
  c = fmaf(z, c, -1.3888889e-3f);
  c = fmaf(z, c, 4.1666667e-2f);
  c = fmaf(z, c, -0.5f);
  c = fmaf(z, c, 1.f);
  const bool odd = quarter & 1u;
  const float a = odd ? s : c, b = odd ? c : s;
  *cs = __uint_as_float(__float_as_uint(a) ^ ((quarter + 1) & 2u) << 30);  // cos: + - - + by quarter
  *sn = __uint_as_float(__float_as_uint(b) ^ (quarter & 2u) << 30);        // sin: + + - -
}

// Packed cosines and sines of pairs a and b at positions pa and pb.
__device__ __forceinline__ void two_turns(const PairTurn& a, const PairTurn& b, int pa, int pb, bool inverse, uint64_t* c,
                                          uint64_t* s) {
  float ca, sa, cb, sb;
  turn_sincos(pa, a.step, &ca, &sa);
  turn_sincos(pb, b.step, &cb, &sb);
  if (inverse) sa = -sa, sb = -sb;
  if (a.axis == 255) ca = sa = __int_as_float(0x7fc00000);
  if (b.axis == 255) cb = sb = __int_as_float(0x7fc00000);
  *c = f2_pack(ca, cb);
  *s = f2_pack(sa, sb);
}

// A thread's eight pairs as packed operands: cos, sin and -sin of pairs 2j and 2j + 1.
struct Turn {
  uint64_t c[4], s[4], n[4];

  // (cs, sn): packed cosines and sines of two pairs, those of pairs 2j and 2j + 1 in lane first + j * step
  __device__ __forceinline__ void gather(uint64_t cs, uint64_t sn, int first, int step) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      c[j] = __shfl_sync(0xffffffffu, cs, first + j * step);
      s[j] = __shfl_sync(0xffffffffu, sn, first + j * step);
      n[j] = s[j] ^ 0x8000000080000000ull;
    }
  }
  // x1, x2: the first and second elements of pairs 2j and 2j + 1
  __device__ __forceinline__ void apply(int j, uint64_t& x1, uint64_t& x2) const {
    const uint64_t y1 = f2_fma(x1, c[j], f2_mul(x2, n[j]));
    x2 = f2_fma(x1, s[j], f2_mul(x2, c[j]));
    x1 = y1;
  }
};

template <int BYTES>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}

// A 16-element unit of one head: two runs of eight elements at offsets e0 and e1.
template <typename T>
struct Unit;
template <>
struct Unit<__nv_bfloat16> {
  static constexpr int PIECES = 2;  // of 16 bytes
  uint4 a, b;
  // global -> this lane's places in shared memory, one every 512 bytes
  static __device__ __forceinline__ void fetch(uint32_t dst, const __nv_bfloat16* p, int e0, int es) {
    cp_async16(dst, p + e0);
    cp_async16(dst + 512, p + e0 + es);
  }
  __device__ __forceinline__ void load(const uint4* p) {
    a = p[0];
    b = p[32];
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p, int e0, int es) const {
    *reinterpret_cast<uint4*>(p + e0) = a;
    *reinterpret_cast<uint4*>(p + e0 + es) = b;
  }
  // in fp32, one rounding, to nearest even
  template <bool INTER>
  __device__ __forceinline__ void turn(const Turn& r) {
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // halves: pairs 2j, 2j + 1 are word j of the two runs; adjacent pairs: words 2j and 2j + 1
      uint32_t &p = w[INTER ? 2 * j : j], &q = w[INTER ? 2 * j + 1 : 4 + j];
      uint64_t x1 = INTER ? f2_pack(bf16lo(p), bf16lo(q)) : f2_pack(bf16lo(p), bf16hi(p));
      uint64_t x2 = INTER ? f2_pack(bf16hi(p), bf16hi(q)) : f2_pack(bf16lo(q), bf16hi(q));
      r.apply(j, x1, x2);
      float y1a, y1b, y2a, y2b;
      f2_unpack_f(x1, y1a, y1b);
      f2_unpack_f(x2, y2a, y2b);
      p = INTER ? pack_bf16x2(y1a, y2a) : pack_bf16x2(y1a, y1b);
      q = INTER ? pack_bf16x2(y1b, y2b) : pack_bf16x2(y2a, y2b);
    }
    a = make_uint4(w[0], w[1], w[2], w[3]);
    b = make_uint4(w[4], w[5], w[6], w[7]);
  }
};
template <>
struct Unit<float> {
  static constexpr int PIECES = 4;
  uint4 v[4];
  static __device__ __forceinline__ void fetch(uint32_t dst, const float* p, int e0, int es) {
#pragma unroll
    for (int i = 0; i < 4; ++i) cp_async16(dst + 512 * i, p + e0 + i * es);
  }
  __device__ __forceinline__ void load(const uint4* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = p[32 * i];
  }
  __device__ __forceinline__ void store(float* p, int e0, int es) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(p + e0 + i * es) = v[i];
  }
  template <bool INTER>
  __device__ __forceinline__ void turn(const Turn& r) {
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[4 * i] = v[i].x, w[4 * i + 1] = v[i].y, w[4 * i + 2] = v[i].z, w[4 * i + 3] = v[i].w;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // elements of pairs 2j and 2j + 1: first ones, then second ones
      const int f0 = INTER ? 4 * j : 2 * j, f1 = INTER ? 4 * j + 2 : 2 * j + 1;
      const int s0 = INTER ? 4 * j + 1 : 8 + 2 * j, s1 = INTER ? 4 * j + 3 : 9 + 2 * j;
      uint64_t x1 = f2_pack(__uint_as_float(w[f0]), __uint_as_float(w[f1]));
      uint64_t x2 = f2_pack(__uint_as_float(w[s0]), __uint_as_float(w[s1]));
      r.apply(j, x1, x2);
      f2_unpack(x1, w[f0], w[f1]);
      f2_unpack(x2, w[s0], w[s1]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
};

// Where unit u's pieces of 16 bytes begin: at e0, e0 + es, ... ; returns whether it is rotated.  Neighbouring units' pieces
// lie next to each other, so that the lanes' 16 bytes fill whole 32-byte sectors.
template <typename T, int D>
__device__ __forceinline__ bool unit_pieces(int rot, int u, int* e0, int* es) {
  constexpr int W = 16 / sizeof(T), NP = 16 / W;  // elements of a piece, pieces of a unit
  const bool rotated = u < rot / 16;
  *e0 = rotated ? W * u : rot + W * (u - rot / 16);
  *es = (rotated ? rot : D - rot) / NP;
  return rotated;
}
// The q-th of its eight pairs: runs of RUN pairs, RUN * 2 elements (adjacent pairs) or RUN elements of either half of `rot`.
template <typename T, bool INTER>
__device__ __forceinline__ int unit_pair(int rot, int u, int q) {
  constexpr int W = 16 / sizeof(T), RUN = INTER ? W / 2 : W;
  return q / RUN * (rot / 2 * RUN / 8) + RUN * u + q % RUN;
}

// A warp's item is a few tokens and one of `slices` parts of the heads.  QUAD: a lane is (token, head lane, unit) and takes
// heads part * 4 * per + head lane + 4 i, i < per; the four head lanes of a unit form two pairs' sines and cosines each.
// Without QUAD, for up to three heads, a lane is (token, unit), takes heads part * per + i and forms all eight (65536 tokens
// of one head of 64: 8.2 us, with QUAD 16.2; of four heads: 4.1 us on 8192 tokens with QUAD, 5.5 without).
// Warps take every (number of warps)-th item, so that they are near one another in memory.
struct Tiling {
  int count, slices, per;
};

template <int D, bool QUAD>
struct Lane {
  static constexpr int UNITS = D / 16, PER_TOKEN = QUAD ? 4 * UNITS : UNITS, TOKS = 32 / PER_TOKEN, STEP = QUAD ? 4 : 1;
  int lane, u, hl, tok;
  __device__ __forceinline__ Lane()
      : lane(threadIdx.x & 31), u(lane % UNITS), hl(QUAD ? lane / UNITS % 4 : 0), tok(lane / PER_TOKEN) {}
};

// A warp's stage of the ring: 8 pieces of data and a slot a lane, and the tokens' positions on up to 8 axes.
constexpr int STAGES = 2;
constexpr int PIECE_SLOTS = 8;
constexpr int OFF_POS = PIECE_SLOTS * 512, OFF_SLOT = OFF_POS + 256, STAGE_BYTES = OFF_SLOT + 256;
constexpr int ROPE_SMEM = ROPE_THREADS / 32 * STAGES * STAGE_BYTES;

struct Walk {
  int item, block, slice;
  __device__ __forceinline__ Walk(const Tiling& g) {
    item = blockIdx.x * (ROPE_THREADS / 32) + threadIdx.x / 32;
    block = item / g.slices;
    slice = item - block * g.slices;
  }
  __device__ __forceinline__ void next(const Tiling& g, int step, int step_block, int step_slice) {
    item += step;
    block += step_block;
    if (step_slice == 0) {  // all warps move on to the next part, so that none has the short one every time
      if (++slice == g.slices) slice = 0;
    } else {
      slice += step_slice;
      if (slice >= g.slices) slice -= g.slices, ++block;
    }
  }
};

// Runs a warp's items.  fetch(token, first head, address, address of the slot): starts a lane's copies and returns where the
// token's position on axis 0 is; finish(token, first head, pieces, slot, turn): rotates and stores them.
template <typename T, int D, bool INTER, bool QUAD, typename Fetch, typename Finish>
__device__ __forceinline__ void run_items(const Tiling& g, const Rotary& r, const PairTurn* pairs, bool rotated, int tokens,
                                          Fetch fetch, Finish finish) {
  extern __shared__ __align__(128) uint8_t ring[];
  using L = Lane<D, QUAD>;
  const L l;
  uint8_t* const mine = ring + threadIdx.x / 32 * STAGES * STAGE_BYTES;
  const int step = gridDim.x * (ROPE_THREADS / 32), step_block = step / g.slices, step_slice = step - step_block * g.slices;
  const auto pair = [&](int q) { return pairs[unit_pair<T, INTER>(r.rot, l.u, q)]; };
  PairTurn p0{0, 255, 0}, p1{0, 255, 0};
  if (QUAD && rotated) p0 = pair(2 * l.hl), p1 = pair(2 * l.hl + 1);
  Walk ld(g);
  int ld_stage = 0, stage = 0;
  auto load = [&]() {
    if (ld.item < g.count) {
      const int t = ld.block * L::TOKS + l.tok;
      if (t < tokens) {
        const uint32_t dst = smem_u32(mine) + ld_stage * STAGE_BYTES;
        const int* const pos = fetch(t, ld.slice * L::STEP * g.per + l.hl, dst + l.lane * 16, dst + OFF_SLOT + l.lane * 8);
        if (QUAD) {  // of its two pairs
          if (p0.axis != 255) cp_async_small<4>(dst + OFF_POS + l.lane * 8, pos + p0.axis * r.axis_stride);
          if (p1.axis != 255) cp_async_small<4>(dst + OFF_POS + l.lane * 8 + 4, pos + p1.axis * r.axis_stride);
        } else if (r.rot > 0) {  // the token's, on every axis
          for (int ax = l.u; ax < r.n_axes; ax += L::PER_TOKEN)
            cp_async_small<4>(dst + OFF_POS + l.tok * 32 + ax * 4, pos + ax * r.axis_stride);
        }
      }
    }
    cp_async_commit();
    ld.next(g, step, step_block, step_slice);
    ld_stage = ld_stage + 1 == STAGES ? 0 : ld_stage + 1;
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) load();
  for (Walk w(g); w.item < g.count; w.next(g, step, step_block, step_slice)) {
    __syncwarp();  // the stage of the item before this one has been read
    load();
    cp_async_wait<STAGES - 1>();
    if (!QUAD) __syncwarp();  // the positions that other lanes copied
    const uint8_t* const st = mine + stage * STAGE_BYTES;
    Turn turn;
    if constexpr (QUAD) {  // a lane past the last token turns by whatever its stage holds, and stores nothing
      const int2 pos = *reinterpret_cast<const int2*>(st + OFF_POS + l.lane * 8);
      uint64_t c, s;
      two_turns(p0, p1, pos.x, pos.y, r.inverse != 0, &c, &s);
      turn.gather(c, s, l.lane - l.hl * L::UNITS, L::UNITS);
    } else {
#pragma unroll
      for (int j = 0; rotated && j < 4; ++j) {
        const int* const pos = reinterpret_cast<const int*>(st + OFF_POS + l.tok * 32);
        const PairTurn a = pair(2 * j), b = pair(2 * j + 1);
        two_turns(a, b, pos[a.axis & 7], pos[b.axis & 7], r.inverse != 0, &turn.c[j], &turn.s[j]);
        turn.n[j] = turn.s[j] ^ 0x8000000080000000ull;
      }
    }
    const int t = w.block * L::TOKS + l.tok;
    if (t < tokens)
      finish(t, w.slice * L::STEP * g.per + l.hl, reinterpret_cast<const uint4*>(st) + l.lane,
             *reinterpret_cast<const long long*>(st + OFF_SLOT + l.lane * 8), turn);
    stage = stage + 1 == STAGES ? 0 : stage + 1;
  }
}

}  // namespace

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
            if (rotated && h < hv) x.template turn<INTER>(turn);
            x.store(h < hk ? qo + h * D : h < hv ? ko + (h - hk) * a.c_head : vo + (h - hv) * a.c_head, e0, es);
          }
        }
      });
}

// Cuts `tokens` x `heads`: as many heads a lane, up to what its stage holds, as leave an item for every warp.  Large inputs
// go faster with fewer blocks a SM, and so fewer places of device memory read and written at a time, as long as two full
// stages a warp are on their way for each of two blocks: heads that fill only part of the lanes' stages need more blocks.
// One launch behind another, times with 2 / 3 / 4 blocks at 290 MB read and written: bf16, 16 heads of 128 (stages full) 47.6 /
// 51.5 / 51.4 us; 20 heads (5/8) 53.7 / 47.2 / 50.3; 8 (half) 58.5 / 50.3 / 46.7; one of 64 (a quarter) 136 / 112 / 103; fp32, 8
// heads of 128 (full) 48.2 / 49.6 / 50.3; 5 (5/8) 51.7 / 46.2 / 50.3.  From 256 MB on that decides.  Smaller inputs depend on
// what the L2 cache holds: 200 MB of 32 heads of 64, 34.0 / 35.5 / 35.7 behind another launch, 39.6 / 41.6 / 41.6 with the
// cache full of unwritten lines, 35.5 / 31.4 / 31.4 with none; 48 heads of 128 appended, 34.7 / 34.5 / 35.4, 39.6 / 41.6 / 40.6 and
// 37.5 / 33.4 / 31.4.  So three at least there, and four below 165 MB, where they are as good or better in every state (140 MB
// of 20 heads of 128: 27.7 / 24.5 / 22.8 behind another launch).
template <typename T, int D, bool QUAD>
static cudaError_t tile(long long tokens, int heads, int sms, Tiling* g, unsigned* grid) {
  using L = Lane<D, QUAD>;
  const int warps = ROPE_THREADS / 32, most = PIECE_SLOTS / Unit<T>::PIECES;
  const long long bytes = tokens * heads * D * static_cast<long long>(2 * sizeof(T));
  const long long room = (heads + L::STEP * most - 1) / (L::STEP * most) * static_cast<long long>(L::STEP * most);  // heads the stages hold
  const int full = static_cast<int>((4 * room + heads) / (2 * heads));  // 2 * room / heads, to the nearest
  const int least = bytes < 165000000 ? ROPE_BLOCKS : bytes < 256000000 ? 3 : 2;
  const int blocks_sm = full > ROPE_BLOCKS ? ROPE_BLOCKS : full > least ? full : least;
  const long long resident = static_cast<long long>(sms) * blocks_sm * warps, blocks = (tokens + L::TOKS - 1) / L::TOKS;
  long long count = 0;
  for (int per = most;; per /= 2) {
    g->slices = (heads + L::STEP * per - 1) / (L::STEP * per);
    g->per = (heads + L::STEP * g->slices - 1) / (L::STEP * g->slices);  // parts alike
    count = blocks * g->slices;
    if (per == 1 || count >= resident) break;
  }
  if (count < 1 || count > 0x7FFFFFFF - STAGES * resident) return cudaErrorInvalidValue;
  g->count = static_cast<int>(count);
  *grid = static_cast<unsigned>(((count < resident ? count : resident) + warps - 1) / warps);
  return cudaSuccess;
}

template <auto kernel, typename... Args>
static cudaError_t launch_items(unsigned grid, cudaStream_t stream, Args... args) {
  const cudaError_t e = allow_shared_memory<kernel>(ROPE_SMEM);
  return e != cudaSuccess ? e : launch_dependent(kernel, grid, ROPE_THREADS, ROPE_SMEM, stream, args...);
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
