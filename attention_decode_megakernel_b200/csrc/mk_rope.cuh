// mk_rope.cuh -- RMSNorm of every query and key head and the rotation of its
// first rot_dim values by position, in one pass over the rows.
//
//   y = x * rsqrt(mean(x^2) + eps) * gain            (skipped without a gain)
//   (y_a, y_b) <- m (y_a cos t - y_b sin t, y_b cos t + y_a sin t)
//
// with t = 2 pi * position * (turns[i] / 2^64) of pair i: (i, i + rot/2), or
// (2i, 2i + 1) when interleaved.  The bytes bound it: every row is read once
// and written once.
//
// A group of HD / (2 * VEC) lanes owns one token: each lane takes the two
// 16-byte pieces that hold both members of its pairs, so the rotation needs
// no exchange, and the same pairs of every head of the token.  Cosine and
// sine are therefore computed once for all of a lane's heads.  The
// angle is a fraction of a turn in 64-bit fixed point: a position times
// turns[i] modulo 2^64 drops the whole turns by itself, so that only turns[i] is not
// exact: a frequency of 53 bits (power, scaling and division, within 64 * 2^-53 of itself;
// at most 1 / 2 pi turns), cut to a multiple of 2^-64.  The angle is off by
// |position| * 1.2e-15 turns, 1.3e-9 at a position of 2^20 where an angle in fp32 would be
// off by 2^-24 * 2^20 radians, and by 2^-32 more where it is cut to its upper 32 bits.
// Measured (32768 tokens, 8 + 2 heads of 256, bf16, 64 values rotated): 63.5 us,
// 5.3 TB/s; 0.45 instructions a scheduler and cycle, so bytes and issue share it.
#pragma once
#include "mk_rows.cuh"

namespace mk {
namespace rp {

constexpr int THREADS = 128;
// Rows of a lane in flight, and blocks a multiprocessor: 2 and 6 ran fastest of 1
// to 5 rows by 1 to 10 blocks (32768 tokens, 8 + 2 heads of 256, bf16: 63.5 us; 3
// rows 65.6, 8 blocks 69.6, as many registers as the compiler takes 71.7).
constexpr int UNROLL = 2, BLOCKS = 6;

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
  unsigned long long turns[128];
};

// The upper 32 bits of position * turns 2^-64 turns, whole turns dropped (unsigned, since
// the product is meant to wrap).
__host__ __device__ __forceinline__ unsigned turn_at(int position, unsigned long long turns) {
  return unsigned(((unsigned long long)(long long)position * turns) >> 32);
}

// m sin and m cos of t 2^-32 turns: the nearest quarter turn is taken off in
// integers, which leaves an angle of at most pi / 4 for the Taylor series to
// x^9 and x^8 (they leave off at most 2e-9 and 3e-8, below half a unit of the
// last place of 1).
__device__ __forceinline__ void sincos_turn(unsigned t, float m, float& sn, float& cs) {
  const unsigned quarter = (t + 0x20000000u) >> 30;
  const float x = float(int(t - (quarter << 30))) * (6.283185307179586f * 0x1p-32f);
  const float y = x * x;
  float s = fmaf(y, 2.7557319e-6f, -1.9841270e-4f);
  float c = fmaf(y, 2.4801587e-5f, -1.3888889e-3f);
  s = fmaf(y, s, 8.3333333e-3f);
  c = fmaf(y, c, 4.1666667e-2f);
  s = fmaf(y, s, -1.6666667e-1f);
  c = fmaf(y, c, -0.5f);
  s = fmaf(x * y, s, x) * m;
  c = fmaf(y, c, 1.0f) * m;
  const bool swap = quarter & 1;
  sn = swap ? c : s;
  cs = swap ? s : c;
  if (quarter & 2) sn = -sn;
  if ((quarter + 1) & 2) cs = -cs;
}

// Blocks are (tokens, parts of the heads); a lane group takes one token's heads
// [per_group * part, ...).  The block first computes the angles of its
// tokens side by side into shared memory; U rows of a lane are in flight.
template <class T, int HD>
__global__ void __launch_bounds__(THREADS, BLOCKS)
    qk_norm_rope_kernel(const __grid_constant__ RopeArgs a) {
  using R = RowType<T>;
  constexpr int U = UNROLL;
  constexpr int VEC = R::VEC, LANES = HD / (2 * VEC), GROUPS = THREADS / LANES;
  extern __shared__ float angles[];  // [GROUPS][cos: rot / 2, sin: rot / 2]
  const int s = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const long long token = (long long)blockIdx.x * GROUPS + group;
  const int heads = a.q_heads + a.kv_heads;
  int h = blockIdx.y * a.per_group;
  const int h_end = token >= a.tokens ? 0 : h + a.per_group < heads ? h + a.per_group : heads;

  // The lane's two pieces.  Interleaved pairs lie within a piece, so any two do;
  // otherwise piece s and its partner half the rotated part on, and beyond the
  // rotated part the pieces in order.  Neighbouring lanes hold neighbouring pieces.
  const int half = a.rot_dim / (2 * VEC);  // pieces of one half of the rotated part
  int p0 = s, p1 = s + LANES;
  if (!a.interleaved) {
    p0 = s < half ? s : s + half;
    p1 = s < half ? s + half : s + LANES;
  }
  const bool turn0 = a.interleaved ? p0 < 2 * half : s < half;
  const bool turn1 = a.interleaved ? p1 < 2 * half : s < half;

  // rows h, h + 1, .. from `in`; at the first key head the pointers move on
  const unsigned char *in, *gain;
  unsigned char* out;
  long long in_step, out_step;
  int side_end;
  uint4 g0, g1;
  auto side = [&] {
    const bool is_q = h < a.q_heads;
    const int i = is_q ? h : h - a.q_heads;
    in = is_q ? a.q + (token * a.q_ts + i * a.q_hs) * R::SIZE
              : a.k + (token * a.k_ts + i * a.k_hs) * R::SIZE;
    out = is_q ? a.q_out + (token * a.qo_ts + i * a.qo_hs) * R::SIZE
               : a.k_out + (token * a.ko_ts + i * a.ko_hs) * R::SIZE;
    in_step = (is_q ? a.q_hs : a.k_hs) * R::SIZE;
    out_step = (is_q ? a.qo_hs : a.ko_hs) * R::SIZE;
    gain = is_q ? a.q_gain : a.k_gain;
    side_end = is_q && a.q_heads < h_end ? a.q_heads : h_end;
    if (gain) {
      g0 = *reinterpret_cast<const uint4*>(gain + p0 * 16);
      g1 = *reinterpret_cast<const uint4*>(gain + p1 * 16);
    }
  };
  uint4 u[U][2];
  auto fetch = [&] {
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (h + j < side_end) {
        u[j][0] = *reinterpret_cast<const uint4*>(in + j * in_step + p0 * 16);
        u[j][1] = *reinterpret_cast<const uint4*>(in + j * in_step + p1 * 16);
      }
  };
  if (h < h_end) {
    side();
    fetch();
  }

  const int pairs = a.rot_dim / 2;
  for (int x = threadIdx.x; x < GROUPS * pairs; x += THREADS) {
    const int g = x / pairs, i = x - g * pairs;
    const long long tok = (long long)blockIdx.x * GROUPS + g;
    if (tok < a.tokens) {
      sincos_turn(turn_at(a.positions[tok], a.turns[i]), a.magnitude,
                  angles[g * a.rot_dim + pairs + i], angles[g * a.rot_dim + i]);
    }
  }
  __syncthreads();
  float cs[VEC], sn[VEC];
  if (turn0) {
    // interleaved: half of the angles for each piece; else one for each value of the first
    const float* from = angles + group * a.rot_dim;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int pair = !a.interleaved ? p0 * VEC + i
                       : i < VEC / 2  ? p0 * (VEC / 2) + i
                                      : p1 * (VEC / 2) + i - VEC / 2;
      if (a.interleaved && i >= VEC / 2 && !turn1) continue;
      cs[i] = from[pair];
      sn[i] = from[pairs + pair];
    }
  }
  // the lanes of a group take every branch together: shuffles name them alone
  const unsigned mask = LANES == 32 ? 0xffffffffu
                                    : ((1u << (LANES & 31)) - 1u) << (threadIdx.x & (32 - LANES));
  while (h < h_end) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (h + j >= side_end) break;
      float x[VEC], y[VEC];
      R::unpack(u[j][0], x);
      R::unpack(u[j][1], y);
      if (gain) {
        float s0 = 0.f, s1 = 0.f, w[VEC];
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
          ffma2(s0, s1, x[i], x[i + 1], x[i], x[i + 1]);
          ffma2(s0, s1, y[i], y[i + 1], y[i], y[i + 1]);
        }
        float sum = s0 + s1;
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(mask, sum, o);
        const float r = rsqrtf(fmaf(sum, 1.0f / HD, a.eps));
        R::unpack(g0, w);
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
          mul2(x[i], x[i + 1], w[i], w[i + 1]);
          mul2(x[i], x[i + 1], r, r);
        }
        R::unpack(g1, w);
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
          mul2(y[i], y[i + 1], w[i], w[i + 1]);
          mul2(y[i], y[i + 1], r, r);
        }
      }
      if (a.interleaved) {
        if (turn0) {
#pragma unroll
          for (int i = 0; i < VEC / 2; ++i) {
            const float x0 = x[2 * i];
            x[2 * i] = x0 * cs[i] - x[2 * i + 1] * sn[i];
            x[2 * i + 1] = x[2 * i + 1] * cs[i] + x0 * sn[i];
          }
        }
        if (turn1) {
#pragma unroll
          for (int i = 0; i < VEC / 2; ++i) {
            const float y0 = y[2 * i];
            y[2 * i] = y0 * cs[VEC / 2 + i] - y[2 * i + 1] * sn[VEC / 2 + i];
            y[2 * i + 1] = y[2 * i + 1] * cs[VEC / 2 + i] + y0 * sn[VEC / 2 + i];
          }
        }
      } else if (turn0) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float x0 = x[i];
          x[i] = x0 * cs[i] - y[i] * sn[i];
          y[i] = y[i] * cs[i] + x0 * sn[i];
        }
      }
      *reinterpret_cast<uint4*>(out + j * out_step + p0 * 16) = R::pack(x);
      *reinterpret_cast<uint4*>(out + j * out_step + p1 * 16) = R::pack(y);
    }
    h += U;
    in += U * in_step;
    out += U * out_step;
    if (h >= side_end) {
      h = side_end;
      if (h < h_end) side();
    }
    if (h < h_end) fetch();
  }
}

}  // namespace rp
}  // namespace mk
