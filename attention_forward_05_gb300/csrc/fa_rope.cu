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
// (2^-54 turns for f_i <= 1), so the phase at position p is off by at most p * 2^-54 turns, and its upper
// 32 bits, as a signed fraction of half a turn, go to sincospif.  The F_i take four double-precision
// operations each and are formed once per block in shared memory (double precision runs at about two
// operations a clock and SM here).
//
// Work split.  A thread owns one 16-element unit (eight pairs) of one token and walks heads: the eight
// sines and cosines serve every head it visits.  Copies are 16 bytes wide.  Both kernels are bound by
// device memory: each element is read once and written once.
#include <cuda_bf16.h>

#include "fa_internal.h"
#include "sm103_ptx.cuh"

namespace fa {

namespace {

constexpr int ROPE_THREADS = 256;
enum : int { W_AXIS = 0x20, W_SLOT };  // sites recorded with DEV_BAD_INDEX

// F_i: radians per position as a 64-bit fraction of a turn.
__device__ __forceinline__ unsigned long long turn_fraction(double f) {
  double t = f * 0.15915494309189533577;  // 1 / (2 pi)
  t -= floor(t);
  return __double2ull_rn(t * 18446744073709551616.0);  // t in [0, 1]; 1 saturates, 2^-64 below a whole turn
}

// Fills the block's table of F_i and axes.  Ends with a barrier.
template <int D>
__device__ __forceinline__ void load_rotation(const Rotary& r, unsigned long long (&step)[D / 2],
                                              unsigned char (&axis)[D / 2], int* err) {
  for (int i = threadIdx.x; i < r.rot / 2; i += ROPE_THREADS) {
    step[i] = turn_fraction(r.freqs[i]);
    int a = r.axes != nullptr ? r.axes[i] : 0;
    if (a < 0 || a >= r.n_axes) {
      record_bad_index(err, W_AXIS);
      a = 255;  // the pair becomes NaN
    }
    axis[i] = static_cast<unsigned char>(a);
  }
  __syncthreads();
}

// cos and sin of the eight pairs from pair p0 on, at token (b, n).
template <int D>
__device__ __forceinline__ void unit_angles(const Rotary& r, const unsigned long long (&step)[D / 2],
                                            const unsigned char (&axis)[D / 2], int p0, const int* pos, float (&cs)[8],
                                            float (&sn)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int a = axis[p0 + i];
    const long long p = a == 255 ? 0 : pos[a * r.axis_stride];
    const unsigned long long ph = static_cast<unsigned long long>(p) * step[p0 + i];
    sincospif(static_cast<float>(static_cast<int>(ph >> 32)) * 4.656612873077393e-10f, &sn[i], &cs[i]);  // 2^-31
    if (r.inverse) sn[i] = -sn[i];
    if (a == 255) cs[i] = sn[i] = __int_as_float(0x7fc00000);
  }
}

// A 16-element unit of one head: two runs of eight elements at offsets e0 and e1.
template <typename T>
struct Unit;
template <>
struct Unit<__nv_bfloat16> {
  uint4 a, b;
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int e0, int e1) {
    a = *reinterpret_cast<const uint4*>(p + e0);
    b = *reinterpret_cast<const uint4*>(p + e1);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p, int e0, int e1) const {
    *reinterpret_cast<uint4*>(p + e0) = a;
    *reinterpret_cast<uint4*>(p + e1) = b;
  }
  __device__ __forceinline__ void get(float (&x)[16]) const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[2 * i] = bf16lo(w[i]);
      x[2 * i + 1] = bf16hi(w[i]);
    }
  }
  __device__ __forceinline__ void set(const float (&x)[16]) {  // one rounding, to nearest even
    a = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    b = make_uint4(pack_bf16x2(x[8], x[9]), pack_bf16x2(x[10], x[11]), pack_bf16x2(x[12], x[13]),
                   pack_bf16x2(x[14], x[15]));
  }
};
template <>
struct Unit<float> {
  float4 v[4];
  __device__ __forceinline__ void load(const float* p, int e0, int e1) {
    v[0] = *reinterpret_cast<const float4*>(p + e0);
    v[1] = *reinterpret_cast<const float4*>(p + e0 + 4);
    v[2] = *reinterpret_cast<const float4*>(p + e1);
    v[3] = *reinterpret_cast<const float4*>(p + e1 + 4);
  }
  __device__ __forceinline__ void store(float* p, int e0, int e1) const {
    *reinterpret_cast<float4*>(p + e0) = v[0];
    *reinterpret_cast<float4*>(p + e0 + 4) = v[1];
    *reinterpret_cast<float4*>(p + e1) = v[2];
    *reinterpret_cast<float4*>(p + e1 + 4) = v[3];
  }
  __device__ __forceinline__ void get(float (&x)[16]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[4 * i] = v[i].x;
      x[4 * i + 1] = v[i].y;
      x[4 * i + 2] = v[i].z;
      x[4 * i + 3] = v[i].w;
    }
  }
  __device__ __forceinline__ void set(const float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  }
};

template <typename T>
__device__ __forceinline__ void turn(Unit<T>& u, const float (&cs)[8], const float (&sn)[8], bool interleaved) {
  float x[16], y[16];
  u.get(x);
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[2 * i] = fmaf(x[2 * i], cs[i], -(x[2 * i + 1] * sn[i]));
      y[2 * i + 1] = fmaf(x[2 * i], sn[i], x[2 * i + 1] * cs[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = fmaf(x[i], cs[i], -(x[8 + i] * sn[i]));
      y[8 + i] = fmaf(x[i], sn[i], x[8 + i] * cs[i]);
    }
  }
  u.set(y);
}

// Offsets of unit u's two runs, and whether it is rotated.
__device__ __forceinline__ bool unit_offsets(const Rotary& r, int u, int* e0, int* e1) {
  if (u < r.rot / 16 && !r.interleaved) {
    *e0 = 8 * u;
    *e1 = r.rot / 2 + 8 * u;
    return true;
  }
  *e0 = 16 * u;
  *e1 = 16 * u + 8;
  return u < r.rot / 16;
}

}  // namespace

template <typename T, int D>
__global__ void __launch_bounds__(ROPE_THREADS) fa_rope_kernel(const RopeLaunch a, int slices) {
  constexpr int UNITS = D / 16;
  __shared__ unsigned long long step[D / 2];
  __shared__ unsigned char axis[D / 2];
  load_rotation<D>(a.r, step, axis, a.err);
  const long long tokens = static_cast<long long>(a.B) * a.N;
  const long long idx = static_cast<long long>(blockIdx.x) * ROPE_THREADS + threadIdx.x;
  const int u = static_cast<int>(idx % UNITS);
  const long long t = idx / UNITS % tokens;
  const int slice = static_cast<int>(idx / UNITS / tokens);
  if (slice >= slices) return;
  const long long b = t / a.N, n = t % a.N;
  int e0, e1;
  const bool rotated = unit_offsets(a.r, u, &e0, &e1);
  float cs[8], sn[8];
  if (rotated) unit_angles<D>(a.r, step, axis, 8 * u, a.r.pos + b * a.r.batch_stride + n, cs, sn);
  for (int h = slice; h < a.H + a.Hkv; h += slices) {
    const bool isq = h < a.H;
    const long long hh = isq ? h : h - a.H;
    const RowStrides& si = isq ? a.sq : a.sk;
    const RowStrides& so = isq ? a.sqo : a.sko;
    const T* src = static_cast<const T*>(isq ? a.q : a.k) + b * si.b + hh * si.h + n * si.n;
    T* dst = static_cast<T*>(isq ? a.q_out : a.k_out) + b * so.b + hh * so.h + n * so.n;
    Unit<T> x;
    x.load(src, e0, e1);
    if (rotated) turn(x, cs, sn, a.r.interleaved != 0);
    x.store(dst, e0, e1);
  }
}

template <int D>
__global__ void __launch_bounds__(ROPE_THREADS) fa_paged_append_kernel(const AppendLaunch a, int slices) {
  using T = __nv_bfloat16;
  constexpr int UNITS = D / 16;
  __shared__ unsigned long long step[D / 2];
  __shared__ unsigned char axis[D / 2];
  load_rotation<D>(a.r, step, axis, a.err);
  const long long idx = static_cast<long long>(blockIdx.x) * ROPE_THREADS + threadIdx.x;
  const int u = static_cast<int>(idx % UNITS);
  const int slice = static_cast<int>(idx / UNITS % slices);
  const long long t = idx / UNITS / slices;
  if (t >= a.T) return;
  const long long slot = a.slots[t];
  if (slot >= a.n_slots && slice == 0 && u == 0) record_bad_index(a.err, W_SLOT);
  const bool store = slot >= 0 && slot < a.n_slots;
  const long long row = store ? slot / a.page_size * a.c_page + slot % a.page_size * a.c_row : 0;
  int e0, e1;
  const bool rotated = unit_offsets(a.r, u, &e0, &e1);
  float cs[8], sn[8];
  if (rotated) unit_angles<D>(a.r, step, axis, 8 * u, a.r.pos + t, cs, sn);
  for (int h = slice; h < a.H + 2 * a.Hkv; h += slices) {
    const T* src;
    T* dst;
    bool turns = rotated;
    if (h < a.H) {
      src = static_cast<const T*>(a.q) + t * a.q_tok + h * a.q_head;
      dst = static_cast<T*>(a.q_out) + (t * a.H + h) * D;
    } else if (h < a.H + a.Hkv) {
      if (!store) continue;
      src = static_cast<const T*>(a.k) + t * a.k_tok + (h - a.H) * a.k_head;
      dst = static_cast<T*>(a.k_cache) + row + (h - a.H) * a.c_head;
    } else {
      if (!store) continue;
      src = static_cast<const T*>(a.v) + t * a.v_tok + (h - a.H - a.Hkv) * a.v_head;
      dst = static_cast<T*>(a.v_cache) + row + (h - a.H - a.Hkv) * a.c_head;
      turns = false;
    }
    Unit<T> x;
    x.load(src, e0, e1);
    if (turns) turn(x, cs, sn, a.r.interleaved != 0);
    x.store(dst, e0, e1);
  }
}

// Heads are dealt to `slices` threads per (token, unit): one head a thread while that does not fill the
// GPU, up to eight heads a thread beyond.
static int head_slices(long long tokens, int units, int heads, int sms) {
  const long long fill = static_cast<long long>(sms) * 2048;  // resident threads
  long long s = (fill + tokens * units - 1) / (tokens * units);
  const long long least = (heads + 7) / 8;
  if (s < least) s = least;
  return static_cast<int>(s < heads ? s : heads);
}

static cudaError_t grid_of(long long threads, unsigned* grid) {
  const long long g = (threads + ROPE_THREADS - 1) / ROPE_THREADS;
  if (g < 1 || g > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  *grid = static_cast<unsigned>(g);
  return cudaSuccess;
}

cudaError_t launch_rope(const RopeLaunch& a) {
  const int units = a.d / 16;
  const long long tokens = static_cast<long long>(a.B) * a.N;
  const int slices = head_slices(tokens, units, a.H + a.Hkv, a.sms);
  unsigned grid = 0;
  const cudaError_t e = grid_of(tokens * units * slices, &grid);
  if (e != cudaSuccess) return e;
  if (a.bf16 && a.d == 64) fa_rope_kernel<__nv_bfloat16, 64><<<grid, ROPE_THREADS, 0, a.stream>>>(a, slices);
  else if (a.bf16) fa_rope_kernel<__nv_bfloat16, 128><<<grid, ROPE_THREADS, 0, a.stream>>>(a, slices);
  else if (a.d == 64) fa_rope_kernel<float, 64><<<grid, ROPE_THREADS, 0, a.stream>>>(a, slices);
  else fa_rope_kernel<float, 128><<<grid, ROPE_THREADS, 0, a.stream>>>(a, slices);
  return cudaGetLastError();
}

cudaError_t launch_append(const AppendLaunch& a) {
  const int units = a.d / 16;
  const int slices = head_slices(a.T, units, a.H + 2 * a.Hkv, a.sms);
  unsigned grid = 0;
  const cudaError_t e = grid_of(static_cast<long long>(a.T) * units * slices, &grid);
  if (e != cudaSuccess) return e;
  if (a.d == 64) fa_paged_append_kernel<64><<<grid, ROPE_THREADS, 0, a.stream>>>(a, slices);
  else fa_paged_append_kernel<128><<<grid, ROPE_THREADS, 0, a.stream>>>(a, slices);
  return cudaGetLastError();
}

}  // namespace fa
