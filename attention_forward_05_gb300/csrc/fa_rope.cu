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
// either sign, with no range reduction.  F_i carries double precision's rounding of f_i / (2 pi)
// (2^-54 turns for f_i <= 1), so the phase at position p is off by at most p * 2^-54 turns.  Its upper
// 32 bits split into the nearest quarter turn and a rest of at most an eighth, whose sine and cosine are
// Taylor polynomials (to x^9 and x^10: 2e-9 and 1e-10 off at pi/4).  The F_i take four double-precision
// operations each and are formed once per block in shared memory (double precision runs at about two
// operations a clock and SM here).
//
// Work split.  A thread owns one 16-element unit (eight pairs) of one token; its eight sines and cosines serve
// all the heads it takes, and the loads of four heads are in flight together.  Copies are
// 16 bytes wide.  Items (a block of tokens, up to four heads) are dealt to the resident blocks in even,
// contiguous ranges, a token's heads next to each other: a block keeps the sines and cosines while the tokens
// stay the same, reads a projection's [heads, d] row at about one time, and no block has an item more than
// another one has.  Both kernels are bound by device memory (each element is read once and written once) as
// long as the instructions are few: the products go in packed fp32 pairs.  Measured in bf16, bytes read and
// written over the time with the launch (about 3 us): q and k of 4 x 4096 tokens, 32 heads of 64: 22 us, 6.0 TB/s
// (with eight heads an item, dealt in turn, and sincospif: 32 us); 2 x 8192 tokens, 20 heads of 128, three axes,
// adjacent pairs: 31 us, 5.4 TB/s (36); appending 8191 tokens, 48 heads of 128: 38 us, 5.4 TB/s (42).
#include <cuda_bf16.h>

#include "fa_internal.h"
#include "sm103_ptx.cuh"

namespace fa {

namespace {

constexpr int ROPE_THREADS = 128;
constexpr int ROPE_BLOCKS = 4;  // per SM
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

// A thread's eight pairs as packed operands: cos, sin and -sin of pairs 2j and 2j + 1.
struct Turn {
  uint64_t c[4], s[4], n[4];

  // pairs[0 .. 7] at the positions pos[axis * stride]
  __device__ __forceinline__ void set(const PairTurn* pairs, const int* pos, long long stride, bool inverse) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float cs[2], sn[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const PairTurn t = pairs[2 * j + i];
        const bool ok = t.axis != 255;
        turn_sincos(ok ? pos[t.axis * stride] : 0, t.step, &cs[i], &sn[i]);
        if (inverse) sn[i] = -sn[i];
        if (!ok) cs[i] = sn[i] = __int_as_float(0x7fc00000);
      }
      c[j] = f2_pack(cs[0], cs[1]);
      s[j] = f2_pack(sn[0], sn[1]);
      n[j] = f2_pack(-sn[0], -sn[1]);
    }
  }
  // x1, x2: the first and second elements of pairs 2j and 2j + 1
  __device__ __forceinline__ void apply(int j, uint64_t& x1, uint64_t& x2) const {
    const uint64_t y1 = f2_fma(x1, c[j], f2_mul(x2, n[j]));
    x2 = f2_fma(x1, s[j], f2_mul(x2, c[j]));
    x1 = y1;
  }
};

__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

// A 16-element unit of one head: two runs of eight elements at offsets e0 and e1.
template <typename T>
struct Unit;
template <>
struct Unit<__nv_bfloat16> {
  uint4 a, b;
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int e0, int e1) {
    a = load16(p + e0);
    b = load16(p + e1);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p, int e0, int e1) const {
    *reinterpret_cast<uint4*>(p + e0) = a;
    *reinterpret_cast<uint4*>(p + e1) = b;
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
  uint4 v[4];
  __device__ __forceinline__ void load(const float* p, int e0, int e1) {
    v[0] = load16(p + e0);
    v[1] = load16(p + e0 + 4);
    v[2] = load16(p + e1);
    v[3] = load16(p + e1 + 4);
  }
  __device__ __forceinline__ void store(float* p, int e0, int e1) const {
    *reinterpret_cast<uint4*>(p + e0) = v[0];
    *reinterpret_cast<uint4*>(p + e0 + 4) = v[1];
    *reinterpret_cast<uint4*>(p + e1) = v[2];
    *reinterpret_cast<uint4*>(p + e1 + 4) = v[3];
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

// Offsets of unit u's two runs, and whether it is rotated.
template <bool INTER>
__device__ __forceinline__ bool unit_offsets(int rot, int u, int* e0, int* e1) {
  if (u < rot / 16 && !INTER) {
    *e0 = 8 * u;
    *e1 = rot / 2 + 8 * u;
    return true;
  }
  *e0 = 16 * u;
  *e1 = 16 * u + 8;
  return u < rot / 16;
}

// Items of a kernel: item = token block * slices + slice; the slice is heads slice * per .. slice * per + per - 1,
// per <= HEADS.  Block i takes items i * count / gridDim.x to (i + 1) * count / gridDim.x - 1.
constexpr int HEADS = 4;
struct Items {
  long long count;
  int slices, per;
};

}  // namespace

template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(ROPE_THREADS, ROPE_BLOCKS) fa_rope_kernel(const RopeLaunch a, const Items items) {
  constexpr int UNITS = D / 16;
  constexpr int FLY = sizeof(T) == 2 ? HEADS : HEADS / 2;  // heads loaded together
  __shared__ PairTurn pairs[D / 2];
  griddep_wait();
  load_rotation<D>(a.r, pairs, a.err);
  __syncthreads();
  const int u = threadIdx.x % UNITS;
  int e0, e1;
  const bool rotated = unit_offsets<INTER>(a.r.rot, u, &e0, &e1);
  Turn r;
  bool known = false;  // r belongs to the item's tokens
  const long long last = items.count * (blockIdx.x + 1) / gridDim.x;
  long long item = items.count * blockIdx.x / gridDim.x, block = item / items.slices;
  int slice = static_cast<int>(item - block * items.slices);
  for (; item < last; ++item, ++slice) {
    if (slice == items.slices) {
      slice = 0;
      ++block;
      known = false;
    }
    const long long t = block * (ROPE_THREADS / UNITS) + threadIdx.x / UNITS;
    if (t >= static_cast<long long>(a.B) * a.N) continue;
    const long long b = t / a.N, n = t - b * a.N;
    const int h0 = slice * items.per, h1 = min(h0 + items.per, a.H + a.Hkv);
    const T* const q = static_cast<const T*>(a.q) + b * a.sq.b + n * a.sq.n;
    const T* const k = static_cast<const T*>(a.k) + b * a.sk.b + n * a.sk.n;
    T* const qo = static_cast<T*>(a.q_out) + b * a.sqo.b + n * a.sqo.n;
    T* const ko = static_cast<T*>(a.k_out) + b * a.sko.b + n * a.sko.n;
    for (int h = h0; h < h1; h += FLY) {
      Unit<T> x[FLY];
#pragma unroll
      for (int i = 0; i < FLY; ++i)
        if (h + i < h1) x[i].load(h + i < a.H ? q + (h + i) * a.sq.h : k + (h + i - a.H) * a.sk.h, e0, e1);
      if (!known && rotated)
        r.set(pairs + 8 * u, a.r.pos + b * a.r.batch_stride + n, a.r.axis_stride, a.r.inverse != 0);
      known = true;
#pragma unroll
      for (int i = 0; i < FLY; ++i)
        if (h + i < h1) {
          if (rotated) x[i].template turn<INTER>(r);
          x[i].store(h + i < a.H ? qo + (h + i) * a.sqo.h : ko + (h + i - a.H) * a.sko.h, e0, e1);
        }
    }
  }
}

template <int D, bool INTER>
__global__ void __launch_bounds__(ROPE_THREADS, ROPE_BLOCKS) fa_paged_append_kernel(const AppendLaunch a, const Items items) {
  using T = __nv_bfloat16;
  constexpr int UNITS = D / 16;
  constexpr int FLY = HEADS;
  __shared__ PairTurn pairs[D / 2];
  griddep_wait();
  load_rotation<D>(a.r, pairs, a.err);
  __syncthreads();
  const int u = threadIdx.x % UNITS;
  int e0, e1;
  const bool rotated = unit_offsets<INTER>(a.r.rot, u, &e0, &e1);
  const int hk = a.H, hv = a.H + a.Hkv;  // first key and first value head of the list of heads
  Turn r;
  bool known = false, store = false;  // r, store and row belong to the item's tokens
  long long row = 0;
  const long long last = items.count * (blockIdx.x + 1) / gridDim.x;
  long long item = items.count * blockIdx.x / gridDim.x, block = item / items.slices;
  int slice = static_cast<int>(item - block * items.slices);
  for (; item < last; ++item, ++slice) {
    if (slice == items.slices) {
      slice = 0;
      ++block;
      known = false;
    }
    const long long t = block * (ROPE_THREADS / UNITS) + threadIdx.x / UNITS;
    if (t >= a.T) continue;
    if (!known) {
      const long long slot = a.slots[t];
      if (slot >= a.n_slots) record_bad_index(a.err, W_SLOT);
      store = slot >= 0 && slot < a.n_slots;
      const long long page = store ? slot / a.page_size : 0;
      row = store ? page * a.c_page + (slot - page * a.page_size) * a.c_row : 0;
    }
    const int h0 = slice * items.per, h1 = min(h0 + items.per, a.H + 2 * a.Hkv);
    const T* const q = static_cast<const T*>(a.q) + t * a.q_tok;
    const T* const k = static_cast<const T*>(a.k) + t * a.k_tok;
    const T* const v = static_cast<const T*>(a.v) + t * a.v_tok;
    T* const qo = static_cast<T*>(a.q_out) + t * a.H * D;
    T* const ko = static_cast<T*>(a.k_cache) + row;
    T* const vo = static_cast<T*>(a.v_cache) + row;
    {
      const int h = h0;
      Unit<T> x[FLY];
#pragma unroll
      for (int i = 0; i < FLY; ++i) {
        const int hh = h + i;
        if (hh < h1 && (hh < hk || store))
          x[i].load(hh < hk ? q + hh * a.q_head : hh < hv ? k + (hh - hk) * a.k_head : v + (hh - hv) * a.v_head, e0, e1);
      }
      if (!known && rotated) r.set(pairs + 8 * u, a.r.pos + t, a.r.axis_stride, false);
      known = true;
#pragma unroll
      for (int i = 0; i < FLY; ++i) {
        const int hh = h + i;
        if (hh < h1 && (hh < hk || store)) {
          if (rotated && hh < hv) x[i].template turn<INTER>(r);
          x[i].store(hh < hk ? qo + hh * D : hh < hv ? ko + (hh - hk) * a.c_head : vo + (hh - hv) * a.c_head, e0, e1);
        }
      }
    }
  }
}

// Splits `tokens` x `heads` into items: one head a thread while that does not fill the GPU, up to HEADS beyond.
static cudaError_t plan_items(long long tokens, int d, int heads, int sms, Items* items, unsigned* grid) {
  const int units = d / 16;
  const long long resident = static_cast<long long>(sms) * ROPE_BLOCKS;
  const long long per = tokens * units * heads / (resident * ROPE_THREADS);
  items->per = per < 1 ? 1 : per > HEADS ? HEADS : static_cast<int>(per);
  items->slices = (heads + items->per - 1) / items->per;
  const long long block = ROPE_THREADS / units;
  items->count = (tokens + block - 1) / block * items->slices;
  if (items->count < 1) return cudaErrorInvalidValue;
  *grid = static_cast<unsigned>(items->count < resident ? items->count : resident);
  return cudaSuccess;
}

template <typename T, int D>
static cudaError_t launch_rope_d(const RopeLaunch& a) {
  Items items;
  unsigned grid = 0;
  const cudaError_t e = plan_items(static_cast<long long>(a.B) * a.N, D, a.H + a.Hkv, a.sms, &items, &grid);
  if (e != cudaSuccess) return e;
  if (a.r.interleaved)
    return launch_dependent(fa_rope_kernel<T, D, true>, grid, ROPE_THREADS, 0, a.stream, a, items);
  return launch_dependent(fa_rope_kernel<T, D, false>, grid, ROPE_THREADS, 0, a.stream, a, items);
}

cudaError_t launch_rope(const RopeLaunch& a) {
  if (a.bf16) return a.d == 64 ? launch_rope_d<__nv_bfloat16, 64>(a) : launch_rope_d<__nv_bfloat16, 128>(a);
  return a.d == 64 ? launch_rope_d<float, 64>(a) : launch_rope_d<float, 128>(a);
}

template <int D>
static cudaError_t launch_append_d(const AppendLaunch& a) {
  Items items;
  unsigned grid = 0;
  const cudaError_t e = plan_items(a.T, D, a.H + 2 * a.Hkv, a.sms, &items, &grid);
  if (e != cudaSuccess) return e;
  if (a.r.interleaved)
    return launch_dependent(fa_paged_append_kernel<D, true>, grid, ROPE_THREADS, 0, a.stream, a, items);
  return launch_dependent(fa_paged_append_kernel<D, false>, grid, ROPE_THREADS, 0, a.stream, a, items);
}

cudaError_t launch_append(const AppendLaunch& a) { return a.d == 64 ? launch_append_d<64>(a) : launch_append_d<128>(a); }

}  // namespace fa
