// mk_attn.cuh -- causal attention of packed query rows over keys and values
// that lie packed beside them or in a paged cache.
//
//   o_t = sum_j p_tj v_j / sum_j p_tj,  p_tj = exp(scale q_t . k_j - m_t)
//
// over the keys j <= len - T + t of the row's own sequence (T new tokens, len
// keys).  One warp per (row, query head), an online softmax in fp32.
#pragma once
#include "mk_rows.cuh"

namespace mk {
namespace at {

struct AttnArgs {
  const unsigned char* q;
  unsigned char* out;
  float* lse;                          // [rows][q_heads], or null
  long long q_ts, q_hs, o_ts, o_hs;    // token and head strides, values
  const int* cu_q;                     // [batch + 1] first row of each sequence
  int rows, batch, q_heads, kv_heads, group;
  float scale_log2;                    // scale * log2(e)
  // packed keys and values
  const unsigned char *k, *v;
  long long k_ts, k_hs, v_ts, v_hs;
  // or a paged cache
  PagedView c;
  const int* table;                    // [batch][table_stride]
  int table_stride;
  const int* seq_lens;
};

template <class T, class C, int HD, bool PAGED>
__global__ void __launch_bounds__(128) attn_simple_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int N = HD / 32;  // values of a lane
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const long long row = w / a.q_heads;
  const int h = int(w % a.q_heads), kh = h / a.group;
  if (row >= a.rows || row >= a.cu_q[a.batch] || row < a.cu_q[0]) return;
  int lo = 0, hi = a.batch - 1;  // the last sequence that starts at or before the row
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (a.cu_q[mid] <= row) lo = mid;
    else hi = mid - 1;
  }
  const int first = a.cu_q[lo], n_new = a.cu_q[lo + 1] - first;
  int len = n_new;
  if constexpr (PAGED) {
    const long long room = (long long)a.table_stride << a.c.page_shift;
    len = a.seq_lens[lo];
    len = len < 0 ? 0 : len > room ? int(room) : len;
  }
  const int n = len - n_new + int(row - first) + 1;
  float q[N], o[N];
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 p = RowType<T>::unpack2(*reinterpret_cast<const uint32_t*>(
        a.q + (row * a.q_ts + h * a.q_hs + lane * N + i) * 2));
    q[i] = p.x * a.scale_log2;
    q[i + 1] = p.y * a.scale_log2;
    o[i] = o[i + 1] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < n; ++j) {
    float k[N], v[N], sk = 1.f, sv = 1.f;
#pragma unroll
    for (int i = 0; i < N; ++i) k[i] = v[i] = 0.f;
    const unsigned char *kp = nullptr, *vp = nullptr;
    if constexpr (PAGED) {
      const int page = a.table[(long long)lo * a.table_stride + (j >> a.c.page_shift)];
      if (page >= 0 && page < a.c.n_pages) {
        const int off = j & (a.c.page_size - 1);
        const long long p = page * a.c.page_stride + kh * a.c.head_stride + off * a.c.pos_stride;
        constexpr int S = __is_same(C, E4m3) ? 1 : 2;
        kp = a.c.k + (p + lane * N) * S;
        vp = a.c.v + (p + lane * N) * S;
        if constexpr (__is_same(C, E4m3)) {
          const long long s = ((((long long)page * a.c.kv_heads) + kh) << a.c.page_shift) + off;
          sk = a.c.k_scale[s];
          sv = a.c.v_scale[s];
        }
      }
    } else {
      kp = a.k + ((first + j) * a.k_ts + kh * a.k_hs + lane * N) * 2;
      vp = a.v + ((first + j) * a.v_ts + kh * a.v_hs + lane * N) * 2;
    }
    if (kp) {
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        float2 x, y;
        if constexpr (__is_same(C, E4m3)) {
          x = e4m3_to_float2(*reinterpret_cast<const uint16_t*>(kp + i));
          y = e4m3_to_float2(*reinterpret_cast<const uint16_t*>(vp + i));
        } else {
          x = RowType<T>::unpack2(*reinterpret_cast<const uint32_t*>(kp + 2 * i));
          y = RowType<T>::unpack2(*reinterpret_cast<const uint32_t*>(vp + 2 * i));
        }
        k[i] = x.x * sk;
        k[i + 1] = x.y * sk;
        v[i] = y.x * sv;
        v[i + 1] = y.y * sv;
      }
    }
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) x += q[i] * k[i];
    x = warp_sum(x);
    const float m1 = fmaxf(m, x), base = m1 == -INFINITY ? 0.f : m1;
    const float f = exp2f(m - base), p = exp2f(x - base);
    l = l * f + p;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = o[i] * f + p * v[i];
    m = m1;
  }
  const float inv = n > 0 ? 1.0f / l : 0.f;
#pragma unroll
  for (int i = 0; i < N; i += 2)
    *reinterpret_cast<uint32_t*>(a.out + (row * a.o_ts + h * a.o_hs + lane * N + i) * 2) =
        RowType<T>::pack2(o[i] * inv, o[i + 1] * inv);
  if (a.lse && lane == 0)
    a.lse[row * a.q_heads + h] = n > 0 ? m * 0.69314718055994531f + logf(l) : -INFINITY;
}

}  // namespace at
}  // namespace mk
