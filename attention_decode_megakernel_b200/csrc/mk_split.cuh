// mk_split.cuh -- how an attention call's work is divided over the CTAs, and
// how partial results are joined.
//
// A unit is one tile of query rows of one key head of one sequence: `tq`
// consecutive new tokens times the `group` query heads that share the head.
// It walks ceil(limit / KT) tiles of KT keys, where limit is what its last
// token sees (one tile at least, so that rows without keys are written too).
// All units, ordered by sequence, head and row tile, form one line, each as
// long as its key tiles and `extra` more for what a unit costs besides them
// (queries, first scores, epilogue), and CTA c takes the stretch [c * per,
// (c + 1) * per) of it: every CTA gets the same work whatever the lengths, for
// one long sequence as for a ragged batch.  (Without the extra length, CTAs
// among the short units at the front of a prompt took 1.7 times as long as the
// others.)  Key tile j of a unit lies at extra + j; a stretch that ends before the first
// one leaves the unit to the next CTA.  A unit that lies in one CTA's share is
// finished there.  A unit that crosses shares leaves a partial {sum of
// weighted values, maximum, sum of weights} in each CTA (a CTA has at most
// two: slot 2c for the unit it entered in the middle, 2c + 1 for the one it
// left), and join_kernel adds them in the order of the CTAs: no atomics, the
// same bits every time, no state kept between calls.
#pragma once
#include "mk_attn.cuh"

namespace mk {
namespace at {

// sum of floor((a i + b) / m) for i < n; a, b >= 0, m > 0 (the Euclid-like
// recursion on (a, m), a few steps for the sizes here).  U holds a n + b.
template <class U>
__device__ __forceinline__ long long floor_sum(U n, U m, U a, U b) {
  long long s = 0;
  while (n > 0) {
    s += (long long)(a / m) * ((long long)n * (n - 1) / 2) + (long long)(b / m) * n;
    a %= m;
    b %= m;
    const U y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const U t = a;
    a = m;
    m = t;
  }
  return s;
}

struct Seq {
  int first, n_new, len;  // first row, new tokens, keys
};

// Sequence b as the call's device arrays give it, held to the rows and the table.
__device__ __forceinline__ Seq seq_of(const AttnArgs& a, int b) {
  Seq s;
  int lo = a.cu_q[b], hi = a.cu_q[b + 1];
  lo = lo < 0 ? 0 : lo > a.rows ? a.rows : lo;
  hi = hi < lo ? lo : hi > a.rows ? a.rows : hi;
  s.first = lo;
  s.n_new = hi - lo;
  s.len = s.n_new;
  if (a.table) {
    long long room = (long long)a.table_stride << a.c.page_shift;
    if (room > 1 << 30) room = 1 << 30;  // positions stay clear of 32 bits' end
    const int len = a.seq_lens[b];
    s.len = len < 0 ? 0 : len > room ? int(room) : len;
  }
  return s;
}

template <int KT>
struct Line {
  const AttnArgs& a;
  int tq, extra;
  bool whole;  // units are not divided: a CTA finishes those that begin in its share

  __device__ int row_tiles(const Seq& s) const { return (s.n_new + tq - 1) / tq; }
  // keys that the last token of row tile i sees (may be negative)
  __device__ int limit(const Seq& s, int i) const {
    const int last = (i + 1) * tq;
    return s.len - s.n_new + (last < s.n_new ? last : s.n_new);
  }
  __device__ int tiles(const Seq& s, int i) const {
    const int l = limit(s, i);
    return l <= KT ? 1 : (l + KT - 1) / KT;
  }
  // key tiles of the first x row tiles, x < row_tiles: all of them full
  __device__ long long before(const Seq& s, int x) const {
    const int past = s.len - s.n_new;
    // row tiles whose limit is at most 0 count 1
    const int none = past < 0 ? (-past) / tq : 0;
    if (none >= x) return x;
    const long long b = (long long)(none + 1) * tq + past + KT - 1, n = x - none;
    if (b + n * tq < (1ll << 31)) {
      // the first step by the constant KT, a power of two; none or one follow as a rule
      const unsigned a0 = unsigned(tq) % KT, b0 = unsigned(b) % KT, y = a0 * unsigned(n) + b0;
      const long long s = (long long)(unsigned(tq) / KT) * (n * (n - 1) / 2) +
                          (long long)(unsigned(b) / KT) * n;
      return none + s + (y < KT ? 0 : floor_sum<unsigned>(y / KT, a0, KT, y % KT));
    }
    return none + floor_sum<unsigned long long>(n, KT, tq, b);
  }
  // the length of the first x row tiles, and of one head of the sequence
  __device__ long long length(const Seq& s, int x) const {
    return x ? before(s, x) + (long long)x * extra : 0;
  }
  __device__ long long all(const Seq& s) const {
    const int nq = row_tiles(s);
    return nq ? length(s, nq - 1) + tiles(s, nq - 1) + extra : 0;
  }
};

// A place on the line: key tile j of n of row tile i of nq of head h of sequence b.
template <int KT>
struct Cursor {
  Seq s;
  int b, h, i, j, n, nq;
  int at;    // place in the unit: 0 .. extra + n
  int left;  // length of this CTA's share from here on

  // tiles of the present unit that lie in this share
  __device__ int segment(const Line<KT>& line) const {
    const int end = at + left - line.extra;
    return (end < n && !line.whole ? end : n) - j;
  }
  // past `tiles` of them; at the unit's end, on to the next unit
  __device__ void skip(const Line<KT>& line, int tiles) {
    j += tiles;
    left -= line.extra + j - at;
    at = line.extra + j;
    if (j < n) {
      if (line.whole && left < 1) left = 1;  // past the share's end, to the unit's
      return;
    }
    if (left <= line.extra) {
      left = 0;  // the share ends before the next unit's first tile
      return;
    }
    at = j = 0;
    if (++i == nq) {
      i = 0;
      if (++h == line.a.kv_heads) {
        h = 0;
        do {  // a tile is left, so a sequence with rows follows
          s = seq_of(line.a, ++b);
        } while (s.n_new == 0 && b + 1 < line.a.batch);
        nq = line.row_tiles(s);
      }
    }
    n = line.tiles(s, i);
  }
};

// Brings what find_share and the page lookups read into L2: before the wait for the
// kernel in front, as a hint that takes no values.  Called by all threads of the call's
// CTAs (300 sequences of 300 keys: 44.2 to 43.2 us, one of 32768: 20.9 to 20.5).
__device__ __forceinline__ void warm_l2(const AttnArgs& a) {
  auto touch = [](const int* from, long long n, long long line) {
    if (line * 32 < n) asm volatile("prefetch.global.L2 [%0];" ::"l"(from + line * 32));
  };
  const long long x = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  touch(a.cu_q, a.batch + 1, x);
  if (a.table) {
    touch(a.seq_lens, a.batch, x);
    touch(a.table, a.batch * (long long)a.table_stride, x);
  }
}

// The place and share of CTA `cta` of `ctas`, shares of at least `least`;
// `per` receives a share's length.  Called by one whole warp with all
// lanes; the result is the same in every lane.
template <int KT>
__device__ __forceinline__ Cursor<KT> find_share(const Line<KT>& line, int cta, int ctas,
                                                 int least, long long& per) {
  const AttnArgs& a = line.a;
  const int lane = threadIdx.x & 31;
  long long total = 0, head = 0;  // length of a head of the lane's sequence
  Seq s = {};
  // Sequences in rounds of 32; lane x keeps the place where round x * stride starts.
  const int stride = (a.batch + 1023) / 1024;
  long long start_of = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    if (b0 / 32 == lane * stride) start_of = total;
    head = 0;
    if (b0 + lane < a.batch) {
      s = seq_of(a, b0 + lane);
      head = line.all(s);
    }
    long long w = head * a.kv_heads;
    for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
    total += w;
  }
  per = (total + ctas - 1) / ctas;
  if (per < least) per = least;
  Cursor<KT> c = {};
  const long long at = cta * per;
  if (at >= total) return c;
  c.left = int(total - at < per ? total - at : per);
  // the sequence that holds place `at`
  // (searched from the first round, 300 short sequences took 41.1 us instead of 39.6, 2300
  // 202 instead of 174)
  const int from = 31 - __clz(__ballot_sync(
                            0xffffffffu, lane * stride * 32 < a.batch && start_of <= at));
  long long before = __shfl_sync(0xffffffffu, start_of, from);
  for (int b0 = from * stride * 32; b0 < a.batch; b0 += 32) {
    if (a.batch > 32) {
      head = 0;
      if (b0 + lane < a.batch) {
        s = seq_of(a, b0 + lane);
        head = line.all(s);
      }
    }
    const long long mine = head * a.kv_heads;
    long long sum = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += up;
    }
    const unsigned past = __ballot_sync(0xffffffffu, before + sum > at);
    if (past) {
      const int found = __ffs(past) - 1;
      before += __shfl_sync(0xffffffffu, sum - mine, found);
      head = __shfl_sync(0xffffffffu, head, found);
      c.b = b0 + found;
      c.s.first = __shfl_sync(0xffffffffu, s.first, found);
      c.s.n_new = __shfl_sync(0xffffffffu, s.n_new, found);
      c.s.len = __shfl_sync(0xffffffffu, s.len, found);
      break;
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  c.nq = line.row_tiles(c.s);
  long long off = at - before;
  c.h = int(off / head);
  off -= c.h * head;
  // the last row tile that starts at or before `off`: 32 places at a time
  int lo = 0, span = c.nq;  // it is one of lo .. lo + span - 1
  long long start = 0;      // where it starts
  while (span > 1) {
    const int step = (span + 31) / 32, x = lo + lane * step;
    const long long here = lane * step < span ? line.length(c.s, x) : off + 1;
    const int last = 31 - __clz(__ballot_sync(0xffffffffu, here <= off));
    start = __shfl_sync(0xffffffffu, here, last);
    span = span - last * step < step ? span - last * step : step;
    lo += last * step;
  }
  c.i = lo;
  c.at = int(off - start);
  c.j = c.at > line.extra ? c.at - line.extra : 0;
  c.n = line.tiles(c.s, c.i);
  if (line.whole && c.j > 0) {
    // whole units only: the unit that the last CTA began is that one's
    c.skip(line, c.n - c.j);
    return c;
  }
  if (c.at + c.left <= line.extra) c.left = 0;
  return c;
}

// Partial results in the workspace: for slot s the rows' weighted sums, [R][HD]
// (few rows) or [HD / 4][R] float4 (tiles of rows), their {maximum, sum} [R], and
// for each CTA the unit that it left unfinished.
struct Left {
  int more;   // CTAs behind this one that hold the rest; 0: nothing was left
  int first;  // the unit's first row
  int h;
  int rows;   // its rows: tokens times the group
};
struct Partials {
  float* o;
  float2* ml;
  Left* left;
};
inline __host__ __device__ size_t partial_bytes(int ctas, int rows, int hd) {
  return size_t(ctas) * (2 * size_t(rows) * (hd + 2) * 4 + sizeof(Left));
}
inline __host__ Partials carve(void* ws, int ctas, int rows, int hd) {
  Partials p;
  p.o = static_cast<float*>(ws);
  p.ml = reinterpret_cast<float2*>(p.o + size_t(2) * ctas * rows * hd);
  p.left = reinterpret_cast<Left*>(p.ml + size_t(2) * ctas * rows);
  return p;
}

// The natural logarithm of a row's sum of weights 2^x = l * 2^m.
__device__ __forceinline__ float row_lse(float m, float l) {
  return l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : l == 0.f ? -INFINITY : l;
}

// Adds {m1, l1, o1} to {m, l, o}, both sums of weights 2^(x - m).
template <int N>
__device__ __forceinline__ void join_in(float& m, float& l, float (&o)[N], float m1, float l1,
                                        const float* o1, int step) {
  const float top = fmaxf(m, m1), base = top == -INFINITY ? 0.f : top;
  const float f0 = exp2f(m - base), f1 = exp2f(m1 - base);
  m = top;
  l = l * f0 + l1 * f1;
#pragma unroll
  for (int i = 0; i < N; ++i) o[i] = o[i] * f0 + o1[i * step] * f1;
}

// Joins the partials of the unit that CTA blockIdx.x left unfinished: block (c, r) takes
// row r of it; the lanes of a warp hold the row's values.  JOIN_SPLIT warps share the
// partials, a run of them each, read in the CTAs' order and several at once, and the first
// adds up the runs in their order: one token over 32768 keys leaves 74 partials a head
// (head_dim 256: 29.9 us with one warp, 21.6 with four, 21.0 with six, 20.5 with eight, which
// cost 64 sequences 0.3 us).  A few partials are one warp's.
constexpr int JOIN_SPLIT = 6;
template <class T, int HD>
__global__ void __launch_bounds__(JOIN_SPLIT * 32)
    join_kernel(const __grid_constant__ AttnArgs a, Partials p, int rows) {
  griddep_launch_dependents();
  griddep_wait();
  const Left u = p.left[blockIdx.x];
  const int r = blockIdx.y, lane = threadIdx.x & 31, split = threadIdx.x >> 5;
  if (u.more <= 0 || r >= u.rows) return;
  __shared__ float runs[JOIN_SPLIT - 1][HD / 32 + 2][32];
  constexpr int N = HD / 32;  // values of a lane, in pieces of 4 (2 for HD 64)
  constexpr int V = N < 4 ? N : 4;
  float m = -INFINITY, l = 0.f, o[N];
#pragma unroll
  for (int i = 0; i < N; ++i) o[i] = 0.f;
  constexpr int BATCH = N == 8 ? 4 : 8;
  const int n = u.more + 1, share = (n + JOIN_SPLIT - 1) / JOIN_SPLIT;
  const int run = n <= 2 * BATCH ? n : share;  // partials of a warp
  const int k1 = min(n, (split + 1) * run);
  for (int k0 = split * run; k0 < k1; k0 += BATCH) {  // so many partials on their way at once
    float2 ml[BATCH];
    float x[BATCH][N];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int i = 0; i < N; ++i) x[k][i] = 0.f;
      if (k0 + k < k1) {
        const size_t slot = k0 + k == 0 ? 2 * size_t(blockIdx.x) + 1
                                        : 2 * (size_t(blockIdx.x) + k0 + k);
        ml[k] = p.ml[slot * rows + r];
        const float* src = p.o + (slot * rows + r) * HD + lane * V;
#pragma unroll
        for (int i = 0; i < N; i += V) {
          if constexpr (V == 4) {
            const float4 y = *reinterpret_cast<const float4*>(src + i * 32);
            x[k][i] = y.x;
            x[k][i + 1] = y.y;
            x[k][i + 2] = y.z;
            x[k][i + 3] = y.w;
          } else {
            const float2 y = *reinterpret_cast<const float2*>(src);
            x[k][0] = y.x;
            x[k][1] = y.y;
          }
        }
      }
    }
    float top = m;
#pragma unroll
    for (int k = 0; k < BATCH; ++k) top = fmaxf(top, ml[k].x);
    const float base = top == -INFINITY ? 0.f : top, f0 = exp2f(m - base);
    m = top;
    l *= f0;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] *= f0;
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const float f = exp2f(ml[k].x - base);
      l += f * ml[k].y;
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] += f * x[k][i];
    }
  }
  if (run < n) {
    if (split > 0) {
      float(*to)[32] = runs[split - 1];
      to[N][lane] = m;
      to[N + 1][lane] = l;
#pragma unroll
      for (int i = 0; i < N; ++i) to[i][lane] = o[i];
    }
    __syncthreads();
    if (split == 0)
      for (int s = 0; s < JOIN_SPLIT - 1; ++s)
        join_in<N>(m, l, o, runs[s][N][lane], runs[s][N + 1][lane], &runs[s][0][lane], 32);
  }
  if (split > 0) return;
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  const long long row = u.first + r / a.group;
  const int head = u.h * a.group + r % a.group;
  unsigned char* out = a.out + (row * a.o_ts + head * a.o_hs + lane * V) * 2;
#pragma unroll
  for (int i = 0; i < N; i += V) {
    if constexpr (V == 4) {
      uint2 w;
      w.x = RowType<T>::pack2(o[i] * inv, o[i + 1] * inv);
      w.y = RowType<T>::pack2(o[i + 2] * inv, o[i + 3] * inv);
      *reinterpret_cast<uint2*>(out + i * 64) = w;
    } else {
      *reinterpret_cast<uint32_t*>(out) = RowType<T>::pack2(o[0] * inv, o[1] * inv);
    }
  }
  if (a.lse && lane == 0) a.lse[row * a.q_heads + head] = row_lse(m, l);
}

// The same for partials [HD / 4][rows]: block (c, y) takes 32 rows, a lane for each,
// and 64 columns, 16 to a warp.
template <class T, int HD>
__global__ void __launch_bounds__(128)
    join_tiles_kernel(const __grid_constant__ AttnArgs a, Partials p, int rows) {
  griddep_launch_dependents();
  griddep_wait();
  const Left u = p.left[blockIdx.x];
  if (u.more <= 0) return;
  const int lane = threadIdx.x & 31, r = blockIdx.y / (HD / 64) * 32 + lane;
  const int d = blockIdx.y % (HD / 64) * 64 + (threadIdx.x >> 5) * 16;
  if (r >= u.rows) return;
  const long long row = u.first + r / a.group;
  auto slot_of = [&](int k) {
    return k == 0 ? 2 * size_t(blockIdx.x) + 1 : 2 * (size_t(blockIdx.x) + k);
  };
  float m = -INFINITY, l = 0.f, o[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i] = 0.f;
  for (int k0 = 0; k0 <= u.more; k0 += 4) {  // four partials on their way at once
    float2 ml[4];
    float4 x[4][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[k][i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k0 + k <= u.more) {
        const size_t slot = slot_of(k0 + k);
        ml[k] = p.ml[slot * rows + r];
        const float4* src =
            reinterpret_cast<const float4*>(p.o) + (slot * (HD / 4) + d / 4) * rows + r;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[k][i] = src[i * rows];
      }
    }
    float top = m;
#pragma unroll
    for (int k = 0; k < 4; ++k) top = fmaxf(top, ml[k].x);
    const float base = top == -INFINITY ? 0.f : top, f0 = exp2f(m - base);
    m = top;
    l *= f0;
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] *= f0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float f = exp2f(ml[k].x - base);
      l += f * ml[k].y;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[4 * i] += f * x[k][i].x;
        o[4 * i + 1] += f * x[k][i].y;
        o[4 * i + 2] += f * x[k][i].z;
        o[4 * i + 3] += f * x[k][i].w;
      }
    }
  }
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  const int head = u.h * a.group + r % a.group;
  uint4* out = reinterpret_cast<uint4*>(a.out + (row * a.o_ts + head * a.o_hs + d) * 2);
#pragma unroll
  for (int i = 0; i < 16; i += 8)
    out[i / 8] = make_uint4(RowType<T>::pack2(o[i] * inv, o[i + 1] * inv),
                            RowType<T>::pack2(o[i + 2] * inv, o[i + 3] * inv),
                            RowType<T>::pack2(o[i + 4] * inv, o[i + 5] * inv),
                            RowType<T>::pack2(o[i + 6] * inv, o[i + 7] * inv));
  if (a.lse && d == 0) a.lse[row * a.q_heads + head] = row_lse(m, l);
}

}  // namespace at
}  // namespace mk
