// mk_kvcache.cuh -- rows of keys and values into a paged cache and back.
//
// A cache of 16-bit values takes the rows as they are (rounded to nearest
// even where the types differ).  An e4m3 cache holds every row (one
// position of one head) with a power of two for scale:
//   s = the least 2^e with max|x| / s <= 448, e >= -64;  code = rne(x / s)
// A power of two makes x / s exact, so each value is rounded once, by at
// most 2^-4 of itself (half a step of e4m3's 3 mantissa bits); the floating
// code keeps its relative precision whatever the scale, and the exponent is
// found by bit operations.  Reading back, code * s is exact in bf16 and fp32.
//
// Both directions are bound by their bytes.  A group of HD / (2 * VEC) lanes
// takes one (token, head): each lane 2 * VEC consecutive values of the key
// and of the value row, all four loads in flight at once.
#pragma once
#include "mk_rows.cuh"

namespace mk {
namespace kv {

constexpr int THREADS = 128;

struct MoveArgs {
  PagedView c;
  const unsigned char *k, *v;  // write: the rows; read: unused
  unsigned char *k_out, *v_out;
  long long k_ts, k_hs, v_ts, v_hs;  // token and head strides of the rows, values
  const long long* slots;            // position in the pool, page * page_size + offset; < 0: skip
  int tokens;
};

// Exponent e of the scale of a row with largest magnitude m: the least e with
// m <= 448 * 2^e = 1.75 * 2^(e + 8), held at -64 and above.  An infinite m
// gives 2^120: its infinities read back as such (448 * 2^120), small values as 0.
__device__ __forceinline__ float e4m3_scale(float m) {
  const uint32_t b = __float_as_uint(m);
  int e = int(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = e < -64 ? -64 : e > 120 ? 120 : e;
  return __uint_as_float(uint32_t(e + 127) << 23);
}
// 1 / s of a power of two between 2^-64 and 2^120.
__device__ __forceinline__ float pow2_inverse(float s) {
  return __uint_as_float((254u << 23) - __float_as_uint(s));
}

template <class T>
struct Cached {
  static constexpr int SIZE = RowType<T>::SIZE;
};
template <>
struct Cached<E4m3> {
  static constexpr int SIZE = 1;
};

// N values to / from the cache's type at p (16-byte aligned for 16 values).
template <class C, int N>
__device__ __forceinline__ void store_values(unsigned char* p, const float (&f)[N]) {
  uint32_t w[N * Cached<C>::SIZE / 4];
  if constexpr (Cached<C>::SIZE == 1) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      w[i] = e4m3_pack2(f[4 * i], f[4 * i + 1]) | (e4m3_pack2(f[4 * i + 2], f[4 * i + 3]) << 16);
  } else if constexpr (Cached<C>::SIZE == 2) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w[i] = RowType<C>::pack2(f[2 * i], f[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = __float_as_uint(f[i]);
  }
  constexpr int W = sizeof(w) / 4;
  if constexpr (W == 2) {
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < W / 4; ++i)
      reinterpret_cast<uint4*>(p)[i] =
          make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
}
template <class C, int N>
__device__ __forceinline__ void load_values(const unsigned char* p, float (&f)[N]) {
  constexpr int W = N * Cached<C>::SIZE / 4;
  uint32_t w[W];
  if constexpr (W == 2) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    w[0] = u.x;
    w[1] = u.y;
  } else {
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const uint4 u = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = u.x;
      w[4 * i + 1] = u.y;
      w[4 * i + 2] = u.z;
      w[4 * i + 3] = u.w;
    }
  }
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if constexpr (Cached<C>::SIZE == 1) {
      const float2 a = e4m3_to_float2(w[i] & 0xFFFFu), b = e4m3_to_float2(w[i] >> 16);
      f[4 * i] = a.x;
      f[4 * i + 1] = a.y;
      f[4 * i + 2] = b.x;
      f[4 * i + 3] = b.y;
    } else if constexpr (Cached<C>::SIZE == 2) {
      const float2 a = RowType<C>::unpack2(w[i]);
      f[2 * i] = a.x;
      f[2 * i + 1] = a.y;
    } else {
      f[i] = __uint_as_float(w[i]);
    }
  }
}

// Address of the row of (slot, head) in the pool, in values; -1 where the slot
// names none.
__device__ __forceinline__ long long row_at(const PagedView& c, long long slot, int head) {
  if (slot < 0 || slot >= (long long)c.n_pages << c.page_shift) return -1;
  return (slot >> c.page_shift) * c.page_stride + (slot & (c.page_size - 1)) * c.pos_stride +
         head * c.head_stride;
}
__device__ __forceinline__ long long scale_at(const PagedView& c, long long slot, int head) {
  return (((slot >> c.page_shift) * c.kv_heads + head) << c.page_shift) +
         (slot & (c.page_size - 1));
}

template <class T, class C, int HD>
__global__ void __launch_bounds__(THREADS) kv_write_kernel(const __grid_constant__ MoveArgs a) {
  constexpr int N = 2 * RowType<T>::VEC, LANES = HD / N;
  const int s = threadIdx.x % LANES;
  const long long item = (long long)blockIdx.x * (THREADS / LANES) + threadIdx.x / LANES;
  const long long token = item / a.c.kv_heads;
  const int head = int(item % a.c.kv_heads);
  const long long slot = token < a.tokens ? a.slots[token] : -1;
  const long long at = row_at(a.c, slot, head);
  float k[N], v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) k[i] = v[i] = 0.f;
  if (at >= 0) {
    load_values<T>(a.k + (token * a.k_ts + head * a.k_hs + s * N) * RowType<T>::SIZE, k);
    load_values<T>(a.v + (token * a.v_ts + head * a.v_hs + s * N) * RowType<T>::SIZE, v);
  }
  if constexpr (Cached<C>::SIZE == 1) {
    float mk_ = 0.f, mv = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      mk_ = fmaxf(mk_, fabsf(k[i]));
      mv = fmaxf(mv, fabsf(v[i]));
    }
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
      mk_ = fmaxf(mk_, __shfl_xor_sync(0xffffffffu, mk_, o));
      mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, o));
    }
    const float sk = e4m3_scale(mk_), sv = e4m3_scale(mv);
    const float ik = pow2_inverse(sk), iv = pow2_inverse(sv);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      k[i] *= ik;
      v[i] *= iv;
    }
    if (at >= 0 && s == 0) {
      a.c.k_scale[scale_at(a.c, slot, head)] = sk;
      a.c.v_scale[scale_at(a.c, slot, head)] = sv;
    }
  }
  if (at >= 0) {
    store_values<C>(a.c.k + (at + s * N) * Cached<C>::SIZE, k);
    store_values<C>(a.c.v + (at + s * N) * Cached<C>::SIZE, v);
  }
}

template <class T, class C, int HD>
__global__ void __launch_bounds__(THREADS) kv_read_kernel(const __grid_constant__ MoveArgs a) {
  constexpr int N = 2 * RowType<T>::VEC, LANES = HD / N;
  const int s = threadIdx.x % LANES;
  const long long item = (long long)blockIdx.x * (THREADS / LANES) + threadIdx.x / LANES;
  const long long token = item / a.c.kv_heads;
  const int head = int(item % a.c.kv_heads);
  if (token >= a.tokens) return;
  const long long slot = a.slots[token];
  const long long at = row_at(a.c, slot, head);
  if (at < 0) return;  // the output row stays as it was
  float k[N], v[N];
  load_values<C>(a.c.k + (at + s * N) * Cached<C>::SIZE, k);
  load_values<C>(a.c.v + (at + s * N) * Cached<C>::SIZE, v);
  if constexpr (Cached<C>::SIZE == 1) {
    const float sk = a.c.k_scale[scale_at(a.c, slot, head)];
    const float sv = a.c.v_scale[scale_at(a.c, slot, head)];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      k[i] *= sk;
      v[i] *= sv;
    }
  }
  store_values<T>(a.k_out + (token * a.k_ts + head * a.k_hs + s * N) * RowType<T>::SIZE, k);
  store_values<T>(a.v_out + (token * a.v_ts + head * a.v_hs + s * N) * RowType<T>::SIZE, v);
}

}  // namespace kv
}  // namespace mk
