// mk_rope.cuh -- RMSNorm of every query and key head and the rotation of its
// first rot_dim values by position, in one pass over the rows.
//
//   y = x * rsqrt(mean(x^2) + eps) * gain            (skipped without a gain)
//   (y_a, y_b) <- m (y_a cos t - y_b sin t, y_b cos t + y_a sin t)
//
// with t = 2 pi * position * turns[i] of pair i: (i, i + rot/2), or
// (2i, 2i + 1) when interleaved.  The bytes bound it: every row is read once
// and written once.
//
// A group of HD / (2 * VEC) lanes owns one token: each lane takes the two
// 16-byte pieces that hold both members of its pairs, so the rotation needs
// no exchange, and the same pairs of every head of the token.  Cosine and
// sine are therefore computed once for all of a lane's heads.  The
// angle is reduced in double, as a fraction of a turn: a position of 2^20
// times a frequency in fp32 would be off by 2^-24 * 2^20 radians.
// Measured (bf16, 8 + 2 heads of 256): see the table in the design notes.
#pragma once
#include "mk_rows.cuh"

namespace mk {
namespace rp {

constexpr int THREADS = 128;
constexpr int UNROLL = 4;  // rows in flight of a lane

struct RopeArgs {
  const unsigned char *q, *k;
  unsigned char *q_out, *k_out;
  const unsigned char *q_gain, *k_gain;  // [HD], or null: no norm
  const int* positions;
  long long q_ts, q_hs, k_ts, k_hs, qo_ts, qo_hs, ko_ts, ko_hs;  // token and head strides, values
  int tokens, q_heads, kv_heads;
  int per_group;  // heads one lane group takes
  int rot_dim, interleaved;
  float eps, magnitude;
  double turns[128];
};

template <class T, int HD>
__global__ void __launch_bounds__(THREADS) qk_norm_rope_kernel(const __grid_constant__ RopeArgs a) {
  using R = RowType<T>;
  constexpr int VEC = R::VEC, LANES = HD / (2 * VEC), GROUPS = THREADS / LANES;
  const int s = threadIdx.x % LANES;
  const int heads = a.q_heads + a.kv_heads;
  const int parts = (heads + a.per_group - 1) / a.per_group;
  const long long item = (long long)blockIdx.x * GROUPS + threadIdx.x / LANES;
  const bool live = item < (long long)a.tokens * parts;  // idle groups still take part in shuffles
  const long long token = live ? item / parts : 0;
  const int h_begin = live ? int(item % parts) * a.per_group : 0;
  const int h_end = !live ? 0 : h_begin + a.per_group < heads ? h_begin + a.per_group : heads;

  const int half = a.rot_dim / (2 * VEC);  // pieces of one half of the rotated part
  const bool rotates = s < half;
  int p0 = 2 * s, p1 = 2 * s + 1;
  if (!a.interleaved && rotates) {
    p0 = s;
    p1 = s + half;
  }
  float cs[VEC], sn[VEC];
  if (rotates && live) {
    const double pos = double(a.positions[token]);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const double t = pos * a.turns[s * VEC + i];
      sincospif(2.0f * float(t - rint(t)), &sn[i], &cs[i]);
      cs[i] *= a.magnitude;
      sn[i] *= a.magnitude;
    }
  }
  for (int h0 = h_begin; __any_sync(0xffffffffu, h0 < h_end); h0 += UNROLL) {
    uint4 u[UNROLL][2];
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) {
      const int h = h0 + j;
      u[j][0] = u[j][1] = make_uint4(0, 0, 0, 0);
      if (h < h_end) {
        const unsigned char* row =
            h < a.q_heads ? a.q + (token * a.q_ts + h * a.q_hs) * R::SIZE
                          : a.k + (token * a.k_ts + (h - a.q_heads) * a.k_hs) * R::SIZE;
        u[j][0] = *reinterpret_cast<const uint4*>(row + p0 * 16);
        u[j][1] = *reinterpret_cast<const uint4*>(row + p1 * 16);
      }
    }
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) {
      const int h = h0 + j;
      const bool is_q = h < a.q_heads;
      float x[VEC], y[VEC];
      R::unpack(u[j][0], x);
      R::unpack(u[j][1], y);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < VEC; ++i) sum += x[i] * x[i] + y[i] * y[i];
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (h >= h_end) continue;
      const unsigned char* gain = is_q ? a.q_gain : a.k_gain;
      if (gain) {
        const float r = 1.0f / sqrtf(sum * (1.0f / HD) + a.eps);
        float g[VEC];
        R::unpack(*reinterpret_cast<const uint4*>(gain + p0 * 16), g);
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[i] *= r * g[i];
        R::unpack(*reinterpret_cast<const uint4*>(gain + p1 * 16), g);
#pragma unroll
        for (int i = 0; i < VEC; ++i) y[i] *= r * g[i];
      }
      if (rotates) {
        if (a.interleaved) {
#pragma unroll
          for (int i = 0; i < VEC / 2; ++i) {
            const float x0 = x[2 * i], y0 = y[2 * i];
            x[2 * i] = x0 * cs[i] - x[2 * i + 1] * sn[i];
            x[2 * i + 1] = x[2 * i + 1] * cs[i] + x0 * sn[i];
            y[2 * i] = y0 * cs[VEC / 2 + i] - y[2 * i + 1] * sn[VEC / 2 + i];
            y[2 * i + 1] = y[2 * i + 1] * cs[VEC / 2 + i] + y0 * sn[VEC / 2 + i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            const float x0 = x[i];
            x[i] = x0 * cs[i] - y[i] * sn[i];
            y[i] = y[i] * cs[i] + x0 * sn[i];
          }
        }
      }
      unsigned char* out = is_q ? a.q_out + (token * a.qo_ts + h * a.qo_hs) * R::SIZE
                                : a.k_out + (token * a.ko_ts + (h - a.q_heads) * a.ko_hs) * R::SIZE;
      *reinterpret_cast<uint4*>(out + p0 * 16) = R::pack(x);
      *reinterpret_cast<uint4*>(out + p1 * 16) = R::pack(y);
    }
  }
}

}  // namespace rp
}  // namespace mk
