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
// takes one (token, head): each lane two 16-byte pieces of the key and of the
// value row, all four loads in flight at once, neighbouring lanes at neighbouring
// pieces so that every access of a warp covers whole sectors.
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

// N values to / from type C at p, in accesses of up to 16 bytes.
template <class C, int N>
__device__ __forceinline__ void store_values(unsigned char* p, const float (&f)[N]) {
  constexpr int W = N * Cached<C>::SIZE / 4;
  uint32_t w[W];
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if constexpr (Cached<C>::SIZE == 1)
      w[i] = e4m3_pack2(f[4 * i], f[4 * i + 1]) | (e4m3_pack2(f[4 * i + 2], f[4 * i + 3]) << 16);
    else if constexpr (Cached<C>::SIZE == 2)
      w[i] = RowType<C>::pack2(f[2 * i], f[2 * i + 1]);
    else
      w[i] = __float_as_uint(f[i]);
  }
  if constexpr (W == 1) {
    *reinterpret_cast<uint32_t*>(p) = w[0];
  } else if constexpr (W == 2) {
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
  if constexpr (W == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (W == 2) {
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
  if ((unsigned long long)slot >= (unsigned long long)c.n_pages << c.page_shift) return -1;
  return (slot >> c.page_shift) * c.page_stride + int(slot & (c.page_size - 1)) * c.pos_stride +
         head * c.head_stride;
}
__device__ __forceinline__ long long scale_at(const PagedView& c, long long slot, int head) {
  return (((slot >> c.page_shift) * c.kv_heads + head) << c.page_shift) +
         (slot & (c.page_size - 1));
}

// The largest magnitude of two raw pieces.
template <class T>
__device__ __forceinline__ float max_abs(const uint4& u0, const uint4& u1) {
  if constexpr (RowType<T>::SIZE == 2) {
    using R = RowType<T>;
    uint32_t m = R::max_abs2(u0.x & 0x7FFF7FFFu, u0.y), n = R::max_abs2(u1.x & 0x7FFF7FFFu, u1.y);
    m = R::max_abs2(R::max_abs2(m, u0.z), u0.w);
    n = R::max_abs2(R::max_abs2(n, u1.z), u1.w);
    const float2 f = R::unpack2(R::max_abs2(m, n));
    return fmaxf(f.x, f.y);  // of a NaN and a number the number; of two NaN, NaN
  } else {
    float a[4], b[4], m = 0.f;
    RowType<T>::unpack(u0, a);
    RowType<T>::unpack(u1, b);
#pragma unroll
    for (int e = 0; e < 4; ++e) m = fmaxf(m, fmaxf(fabsf(a[e]), fabsf(b[e])));
    return m;
  }
}

// Blocks are (tokens, key head).
template <class T, class C, int HD>
__global__ void __launch_bounds__(THREADS) kv_write_kernel(const __grid_constant__ MoveArgs a) {
  using R = RowType<T>;
  constexpr int VEC = R::VEC, LANES = HD / (2 * VEC);
  griddep_launch_dependents();
  griddep_wait();
  const int s = threadIdx.x % LANES, head = blockIdx.y;
  const unsigned token = blockIdx.x * (THREADS / LANES) + threadIdx.x / LANES;
  const bool live = token < unsigned(a.tokens);  // the others still take part in shuffles
  const long long row = live ? token : 0;
  const unsigned char* src[2] = {a.k + (row * a.k_ts + head * a.k_hs) * R::SIZE,
                                 a.v + (row * a.v_ts + head * a.v_hs) * R::SIZE};
  uint4 u[2][2];  // key and value, two pieces each
#pragma unroll
  for (int y = 0; y < 2; ++y)
#pragma unroll
    for (int i = 0; i < 2; ++i)
      u[y][i] = *reinterpret_cast<const uint4*>(src[y] + (s + i * LANES) * 16);
  const long long slot = live ? a.slots[row] : -1;  // (its load is in flight with the rows')
  const long long at = row_at(a.c, slot, head);
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    float x[2][VEC], inverse = 1.f;
    if constexpr (Cached<C>::SIZE == 1) {
      float top = max_abs<T>(u[y][0], u[y][1]);
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float scale = e4m3_scale(top);
      inverse = pow2_inverse(scale);
      if (at >= 0 && s == 0) (y == 0 ? a.c.k_scale : a.c.v_scale)[scale_at(a.c, slot, head)] = scale;
    }
    if (at < 0) continue;
    unsigned char* to = (y == 0 ? a.c.k : a.c.v) + at * Cached<C>::SIZE;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      R::unpack(u[y][i], x[i]);
      if constexpr (Cached<C>::SIZE == 1) {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) mul2(x[i][e], x[i][e + 1], inverse, inverse);
      }
      store_values<C>(to + (s + i * LANES) * VEC * Cached<C>::SIZE, x[i]);
    }
  }
}

template <class T, class C, int HD>
__global__ void __launch_bounds__(THREADS) kv_read_kernel(const __grid_constant__ MoveArgs a) {
  using R = RowType<T>;
  constexpr int VEC = R::VEC, LANES = HD / (2 * VEC);
  griddep_launch_dependents();
  griddep_wait();
  const int s = threadIdx.x % LANES, head = blockIdx.y;
  const unsigned token = blockIdx.x * (THREADS / LANES) + threadIdx.x / LANES;
  if (token >= unsigned(a.tokens)) return;
  const long long slot = a.slots[token];
  const long long at = row_at(a.c, slot, head);
  if (at < 0) return;  // the output row stays as it was
  float x[2][2][VEC], scale[2] = {1.f, 1.f};
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const unsigned char* row = (y == 0 ? a.c.k : a.c.v) + at * Cached<C>::SIZE;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      load_values<C>(row + (s + i * LANES) * VEC * Cached<C>::SIZE, x[y][i]);
    if constexpr (Cached<C>::SIZE == 1)
      scale[y] = (y == 0 ? a.c.k_scale : a.c.v_scale)[scale_at(a.c, slot, head)];
  }
  unsigned char* out[2] = {a.k_out + (token * a.k_ts + head * a.k_hs) * R::SIZE,
                           a.v_out + (token * a.v_ts + head * a.v_hs) * R::SIZE};
#pragma unroll
  for (int y = 0; y < 2; ++y)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (Cached<C>::SIZE == 1) {
#pragma unroll
        for (int e = 0; e < VEC; e += 2)
          mul2(x[y][i][e], x[y][i][e + 1], scale[y], scale[y]);
      }
      store_values<T>(out[y] + (s + i * LANES) * 16, x[y][i]);
    }
}

}  // namespace kv
}  // namespace mk
