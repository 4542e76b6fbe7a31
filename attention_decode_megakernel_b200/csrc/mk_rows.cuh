// mk_rows.cuh -- 16-byte pieces of a row of bf16, fp16 or fp32 values, as the
// row-wise operators load, convert and store them.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "mk_ptx.cuh"

namespace mk {

// {a, b} times {x, y}, two products in one instruction.
__device__ __forceinline__ void mul2(float& a, float& b, float x, float y) {
  asm("{\n\t.reg .b64 c, d;\n\t"
      "mov.b64 c, {%0, %1};\n\t"
      "mov.b64 d, {%2, %3};\n\t"
      "mul.rn.f32x2 c, c, d;\n\t"
      "mov.b64 {%0, %1}, c;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(x), "f"(y));
}

struct Bf16 {};
struct Fp16 {};
struct Fp32 {};
struct E4m3 {};

template <class T>
struct RowType;
template <>
struct RowType<Bf16> {
  static constexpr int SIZE = 2, VEC = 8;  // bytes of a value, values of a 16-byte piece
  __device__ static void unpack(const uint4& u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf_lo(w[i]);
      f[2 * i + 1] = bf_hi(w[i]);
    }
  }
  __device__ static float2 unpack2(uint32_t w) { return make_float2(bf_lo(w), bf_hi(w)); }
  __device__ static uint32_t pack2(float a, float b) {
    __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&p);
  }
  // the larger magnitudes of two pairs (a NaN gives way to a number)
  __device__ static uint32_t max_abs2(uint32_t m, uint32_t w) {
    w &= 0x7FFF7FFFu;
    __nv_bfloat162 p = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&m),
                               *reinterpret_cast<__nv_bfloat162*>(&w));
    return *reinterpret_cast<uint32_t*>(&p);
  }
  __device__ static uint4 pack(const float (&f)[8]) {
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
  }
};
template <>
struct RowType<Fp16> {
  static constexpr int SIZE = 2, VEC = 8;
  __device__ static void unpack(const uint4& u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = unpack2(w[i]);
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
  }
  __device__ static float2 unpack2(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  __device__ static uint32_t pack2(float a, float b) {
    __half2 p = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&p);
  }
  __device__ static uint32_t max_abs2(uint32_t m, uint32_t w) {
    w &= 0x7FFF7FFFu;
    __half2 p = __hmax2(*reinterpret_cast<__half2*>(&m), *reinterpret_cast<__half2*>(&w));
    return *reinterpret_cast<uint32_t*>(&p);
  }
  __device__ static uint4 pack(const float (&f)[8]) {
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
  }
};
template <>
struct RowType<Fp32> {
  static constexpr int SIZE = 4, VEC = 4;
  __device__ static void unpack(const uint4& u, float (&f)[4]) {
    f[0] = __uint_as_float(u.x);
    f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z);
    f[3] = __uint_as_float(u.w);
  }
  __device__ static uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};

// Two e4m3 codes of {a, b} (a in the low byte), nearest even; magnitudes above
// 448 are held at 448, NaN becomes the NaN code.
__device__ __forceinline__ uint32_t e4m3_pack2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
// The two values of a pair of codes, exact in fp16.
__device__ __forceinline__ uint32_t e4m3_to_half2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(uint16_t(codes)));
  return r;
}
__device__ __forceinline__ float2 e4m3_to_float2(uint32_t codes) {
  const uint32_t h = e4m3_to_half2(codes);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// A paged cache as the kernels see it: [page][head][position][dim].
struct PagedView {
  unsigned char *k, *v;
  float *k_scale, *v_scale;
  long long page_stride, head_stride, pos_stride;  // in values
  int n_pages, page_size, page_shift, kv_heads, head_dim;
};

}  // namespace mk
