// mk_paged.cuh -- attention of few query rows over a paged cache: decoding and
// short drafts, where a unit's rows (new tokens times the heads of the group)
// are at most 16.
//
// The cache's bytes bound it: every K and V row of a (sequence, key head) is
// read once, for 2 * 8 * NT multiply-adds a value.  So the layout serves the
// loads.  Each of four or eight warps walks its own subtiles of 16 keys through a
// private ring of stages in shared memory: one lane asks TMA for the 16 rows
// of K and of V, a box of (128 bytes, 16 positions, columns of 128 bytes) in the
// 128-byte swizzle, and looks the next page up a step ahead.  (16-byte cp.async copies
// by all lanes were a quarter of the instructions.)  Rows of up to 256 bytes, whose
// stages leave room, have eight warps (64 sequences over an e4m3 cache at head_dim 256:
// 36.8 us, 49 with four and 38.6 with twelve); rows of 512 bytes have four.  Between the
// first load and the last the copies run at the memory's rate (the same 64 sequences at
// head_dim 128 and 256 in bf16: 162 MB more in 24.5 us); more chains of products, fewer
// conversions or loads change nothing.  What is left is around them: finding the shares,
// first loads, joining warps and partials, 10 us.  No barrier joins the warps
// until the unit ends, and the ring runs ahead into the next unit.
//
// The products run on mma.m16n8k16 with the keys as M: S^T = K Q^T and
// O^T = V^T P^T, so that 8 rows (N) cost 8 columns, not a tile of 128 rows.
// At 8 rows the math of a 16-key subtile is 32 instructions against 16 KB of
// bytes (head_dim 256): a tcgen05 tile of 128 rows would only add latency.
// A lane reads 16 bytes of a key row for two k-steps (four of 8-bit values);
// the order of the head's dims inside a step is free as long as Q has the
// same.  Score columns turn into weight rows by movmatrix.
//
// Softmax: weights are 2^(x - m), and m is raised only when a score passes it
// by RAISE, so most subtiles need one vote and no rescaling.  bf16 weights
// start at 1 and stay below 2^8, their rounding relative throughout; fp16
// ones start at 2^7 and stay below 2^15 (LIFT), so that weights down to 2^-21
// of the largest are normal numbers.  (16 bits, since the matrix units multiply those: the
// outputs' root mean square error in bf16 is 1.9e-3 of them, 1.7e-3 with exact weights.)
// 8-bit caches: codes go to fp16, exactly,
// as do queries after a power of two for each row; the key row's scale
// multiplies its scores and log2 of the value row's scale is added to them,
// so that weights stay in fp16's range; their sum is taken without it.
#pragma once
#include <type_traits>

#include "mk_split.cuh"
#include "mk_tc.cuh"

namespace mk {
namespace at {

constexpr long long FEW_WAIT_NS = 2000000000LL;

// The weight of the score that sets m is 2^LIFT, the largest one 2^RAISE.
template <class M>
struct Weights {
  static constexpr float LIFT = __is_same(M, Fp16) ? 7.f : 0.f, RAISE = LIFT + 8.f;
};

template <int WARPS>
struct FewBars {
  uint64_t full[WARPS][8];  // of each warp's stages
  Cursor<16 * WARPS> start;
  int per, gave_up;
};

template <class C, int HD, int NT>
struct FewCfg {
  static constexpr bool E8 = __is_same(C, E4m3);
  static constexpr int ROW = HD * (E8 ? 1 : 2);  // bytes of a cache row
  static constexpr int WARPS = ROW <= 256 ? 8 : 4, THREADS = 32 * WARPS;
  static constexpr int KEYS = 16 * WARPS;        // of a tile: 16 a warp
  static constexpr int STAGE = 32 * ROW, SCALES = E8 ? 128 : 0;  // 16 keys, 16 values; their scales
  static constexpr int ROWS = 8 * NT;
  // The join: all warps' values of 8 rows and so many columns, then {maximum, sum} of each
  // warp's rows and of the rows themselves.
  static constexpr int COLS = WARPS == 8 && ROW * NT >= 256 ? 64 : HD < 128 ? HD : 128;
  static constexpr int JOIN = WARPS * 8 * (COLS + 4) * 4 + (WARPS + 1) * ROWS * 8;
  static constexpr int FIT = (227 * 1024 - int(sizeof(FewBars<WARPS>)) - JOIN) /
                             (WARPS * (STAGE + SCALES));
  static constexpr int STAGES = FIT < 8 ? FIT : 8;
  static constexpr int RING = WARPS * STAGES * STAGE;
  static constexpr size_t SMEM =
      size_t(RING) + WARPS * STAGES * SCALES + JOIN + sizeof(FewBars<WARPS>);
  static_assert(STAGES >= 2, "the ring needs two stages");
};

struct FewArgs {
  AttnArgs a;
  CUtensorMap k, v;  // (dim within 128 bytes, position, column of 128 bytes, head, page)
  int tq, extra, least, whole;
};

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, int c1, int c3,
                                            int c4, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %2, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(c1), "r"(c3), "r"(c4),
      "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 u;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
               : "r"(at));
  return u;
}
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t u;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(u) : "r"(at));
  return u;
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
template <class M>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (__is_same(M, Bf16)) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  } else {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// (relative errors of 2^-22 and less; exact for powers of two)
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Byte offset of 16-byte piece `ch` of row r of 16 rows as TMA lays them down:
// columns of 128 bytes, the rows of one after another, the piece turned by the
// row (64-byte rows: by the pair of rows).  Reads of two rows by four pieces then meet
// twice in a bank, four rows by two pieces and eight rows by one do not.
template <int ROW>
__device__ __forceinline__ uint32_t piece(int r, int ch) {
  if constexpr (ROW == 64) return uint32_t(r) * 64 + ((ch ^ ((r >> 1) & 3)) << 4);
  return uint32_t(ch >> 3) * 2048 + uint32_t(r) * 128 + (((ch & 7) ^ (r & 7)) << 4);
}

template <class T, class C, int HD, int NT>
__global__ void __launch_bounds__(FewCfg<C, HD, NT>::THREADS, 1)
    attn_few_kernel(const __grid_constant__ FewArgs fa, Partials part) {
  using F = FewCfg<C, HD, NT>;
  constexpr bool E8 = F::E8;
  using M = typename std::conditional<E8, Fp16, T>::type;  // what the products multiply
  constexpr int ROW = F::ROW, STAGES = F::STAGES, ROWS = F::ROWS, WARPS = F::WARPS;
  constexpr int KEYS = F::KEYS;
  constexpr int STEPS = HD / 16;               // k-steps of a score, m-tiles of the output
  constexpr int PIECES = HD / (E8 ? 64 : 32);  // 16-byte pieces of a key row a lane reads
  const AttnArgs& a = fa.a;
  const int tq = fa.tq;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* join = smem + F::RING + WARPS * STAGES * F::SCALES;
  FewBars<WARPS>& f = *reinterpret_cast<FewBars<WARPS>*>(join + F::JOIN);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const Line<KEYS> line{a, tq, fa.extra, fa.whole != 0};
  griddep_launch_dependents();
  warm_l2(a);
  if (warp == 0) {
    griddep_wait();
    long long per;
    const Cursor<KEYS> c = find_share<KEYS>(line, blockIdx.x, gridDim.x, fa.least, per);
    if (lane == 0) {
      f.per = int(per);
      f.start = c;
      f.gave_up = 0;
      Left none = {0, 0, 0, 0};
      part.left[blockIdx.x] = none;
    }
  } else if (warp == 1 && lane == 0) {
    for (int i = 0; i < WARPS * 8; ++i) mbar_init(&f.full[0][0] + i, 1);
    fence_barrier_init();
  } else if (warp == 2 && lane == 0) {
    prefetch_map(&fa.k);
    prefetch_map(&fa.v);
  }
  __syncthreads();
  griddep_wait();
  Cursor<KEYS> at = f.start, ahead = at;  // where the math is, where the copies are
  if (at.left <= 0) return;
  const int per = f.per;
  const uint32_t ring = smem_addr(smem) + warp * (STAGES * F::STAGE);
  const uint32_t scales = smem_addr(smem) + F::RING + warp * (STAGES * F::SCALES);
  constexpr int COLS = F::COLS;
  float* join_o = reinterpret_cast<float*>(join);  // [warp][8][COLS + 4]
  float2* join_ml = reinterpret_cast<float2*>(join + WARPS * 8 * (COLS + 4) * 4);
  float2* join_row = join_ml + WARPS * ROWS;

  // The page of this warp's keys at `ahead`; n_pages, which lies outside the maps and
  // arrives as zeros, for one outside the cache.
  auto page_at = [&] {
    int page = a.c.n_pages;
    const int key = ahead.j * KEYS + warp * 16;
    if (ahead.left > 0 && key < line.limit(ahead.s, ahead.i))
      page = a.table[(long long)ahead.b * a.table_stride + (key >> a.c.page_shift)];
    return page;
  };
  uint32_t strange = 0;  // stages whose page lies outside the cache
  int page = page_at();
  // copies of this warp's 16 keys of the tile at `ahead` into stage st
  auto fetch = [&](int st) {
    if (ahead.left <= 0) return;
    const int key = ahead.j * KEYS + warp * 16;
    if (key < line.limit(ahead.s, ahead.i)) {
      const bool known = page >= 0 && page < a.c.n_pages;
      strange = (strange & ~(1u << st)) | (known ? 0u : 1u << st);
      if (elect_one()) {
        const int off = key & (a.c.page_size - 1), p = known ? page : a.c.n_pages;
        const uint32_t dst = ring + st * F::STAGE;
        uint64_t* bar = &f.full[warp][st];
        mbar_arrive_expect_tx(bar, 32 * ROW + (E8 && known ? 128 : 0));
        tma_load_5d(dst, &fa.k, off, ahead.h, p, bar);
        tma_load_5d(dst + 16 * ROW, &fa.v, off, ahead.h, p, bar);
        if (E8 && known) {
          const long long sc =
              (((long long)page * a.c.kv_heads + ahead.h) << a.c.page_shift) + off;
          bulk_load(scales + st * 128, a.c.k_scale + sc, 64, bar);
          bulk_load(scales + st * 128 + 64, a.c.v_scale + sc, 64, bar);
        }
      }
      __syncwarp();
    }
    ahead.skip(line, 1);
    page = page_at();  // used by the next fetch
  };
#pragma unroll 1
  for (int s = 0; s < STAGES - 1; ++s) fetch(s);
  uint32_t phases = 0;  // parity of each stage's next load
  // this stage's load has landed (a wait that runs out: NaN from here on)
  auto landed = [&](int st) {
    uint64_t start = 0;
    while (!mbar_try_wait(&f.full[warp][st], phases >> st & 1)) {
      const uint64_t now = global_ns();
      if (start == 0) start = now;
      if (now - start > uint64_t(FEW_WAIT_NS) || *(volatile int*)&f.gave_up) {
        *(volatile int*)&f.gave_up = 1;
        break;
      }
    }
    __syncwarp();
    phases ^= 1u << st;
  };

  int stage = 0;
  while (at.left > 0) {
    // ---- one segment: the tiles of one unit that lie in this share
    const Cursor<KEYS> u = at;
    const int seg = u.segment(line);
    // queries: row r is token r / group of the tile, head r % group
    uint32_t q[NT][STEPS][2];
    float qs[NT][2];
    int limit[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = nt * 8 + g, token = u.i * tq + r / a.group;
      const bool live = r < tq * a.group && token < u.s.n_new;
      const unsigned char* src =
          a.q + ((u.s.first + (live ? token : 0)) * a.q_ts +
                 (long long)(u.h * a.group + (live ? r % a.group : 0)) * a.q_hs) * 2;
      float size = 0.f;
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
#pragma unroll
        for (int half = 0; half < (E8 ? 2 : 1); ++half) {
          uint4 w = make_uint4(0, 0, 0, 0);
          if (live)
            w = *reinterpret_cast<const uint4*>(src + ((4 * i + t) * (E8 ? 2 : 1) + half) * 16);
          const int st = E8 ? 4 * i + 2 * half : 2 * i;
          q[nt][st][0] = w.x;
          q[nt][st][1] = w.y;
          q[nt][st + 1][0] = w.z;
          q[nt][st + 1][1] = w.w;
        }
      }
      if constexpr (E8 && __is_same(T, Bf16)) {
        // bf16 to fp16: a power of two brings the row's largest value to [1, 2)
#pragma unroll
        for (int i = 0; i < STEPS; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            size = fmaxf(size, fmaxf(fabsf(bf_lo(q[nt][i][j])), fabsf(bf_hi(q[nt][i][j]))));
        size = fmaxf(size, __shfl_xor_sync(0xffffffffu, size, 1));
        size = fmaxf(size, __shfl_xor_sync(0xffffffffu, size, 2));
        uint32_t e = __float_as_uint(size) >> 23;
        e = e < 1 ? 1 : e > 253 ? 253 : e;
        const float down = __uint_as_float((254 - e) << 23);
        size = __uint_as_float(e << 23);
#pragma unroll
        for (int i = 0; i < STEPS; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            q[nt][i][j] = RowType<Fp16>::pack2(bf_lo(q[nt][i][j]) * down,
                                               bf_hi(q[nt][i][j]) * down);
      } else {
        size = 1.f;
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {  // the rows 2t, 2t + 1 whose scores this lane holds
        const int r2 = nt * 8 + 2 * t + x, tok = u.i * tq + r2 / a.group;
        const bool on = r2 < tq * a.group && tok < u.s.n_new;
        limit[nt][x] = on ? u.s.len - u.s.n_new + tok + 1 : 0;
        qs[nt][x] = a.scale_log2 * __shfl_sync(0xffffffffu, size, (2 * t + x) * 4);
      }
    }
    const int sure = u.s.len - u.s.n_new + u.i * tq + 1;  // keys that every row sees

    float o[NT][STEPS][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < STEPS; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.f;
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }

    for (int step = 0; step < seg; ++step) {
      __syncwarp();
      // the stage of the step before this one, which every lane has left
      fetch(stage == 0 ? STAGES - 1 : stage - 1);
      const int key = (u.j + step) * KEYS + warp * 16;
      if (key < line.limit(u.s, u.i)) {
        landed(stage);
        if (key + 16 > u.s.len) {
          // what the page holds behind the sequence: weights of 0 would keep its NaN
          const int keep = u.s.len - key;
          for (int x = lane; x < (16 - keep) * (ROW / 16); x += 32) {
            const uint32_t to = ring + stage * F::STAGE + 16 * ROW +
                                piece<ROW>(keep + x / (ROW / 16), x % (ROW / 16));
            asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(to), "r"(0) : "memory");
          }
          fence_async_smem();
          __syncwarp();
        }
        const uint32_t ks = ring + stage * F::STAGE, vs = ks + 16 * ROW;
        float s[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
          const uint4 lo = lds128(ks + piece<ROW>(g, 4 * i + t));
          const uint4 hi = lds128(ks + piece<ROW>(g + 8, 4 * i + t));
          if constexpr (E8) {
            const uint32_t w0[4] = {lo.x, lo.y, lo.z, lo.w}, w1[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint32_t a0 = e4m3_to_half2(w0[x]), a2 = e4m3_to_half2(w0[x] >> 16);
              const uint32_t a1 = e4m3_to_half2(w1[x]), a3 = e4m3_to_half2(w1[x] >> 16);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma16816<M>(s[nt], a0, a1, a2, a3, q[nt][4 * i + x][0], q[nt][4 * i + x][1]);
            }
          } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma16816<M>(s[nt], lo.x, hi.x, lo.y, hi.y, q[nt][2 * i][0], q[nt][2 * i][1]);
              mma16816<M>(s[nt], lo.z, hi.z, lo.w, hi.w, q[nt][2 * i + 1][0],
                          q[nt][2 * i + 1][1]);
            }
          }
        }
        // scores of the keys g, g + 8 (index / 2) and the rows 2t, 2t + 1 (index % 2), in
        // powers of two
        float kc[2] = {1.f, 1.f}, vl[2] = {0.f, 0.f}, vi[2] = {1.f, 1.f};
        if constexpr (E8) {
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            kc[y] = __uint_as_float(lds32(scales + stage * 128 + (g + 8 * y) * 4));
            float sv = __uint_as_float(lds32(scales + stage * 128 + 64 + (g + 8 * y) * 4));
            // zeros, whose scales were not read, and what the page holds behind the
            // sequence: any bits, by the key's place and not by their value (the reciprocal
            // of a subnormal is infinite, and a weight of 0 times that NaN)
            if ((strange >> stage & 1) || key + g + 8 * y >= u.s.len) kc[y] = sv = 1.f;
            sv = sv > 0.f ? sv : 1.f;  // (no row's scale may be otherwise)
            vl[y] = lg2(sv);
            vi[y] = rcp(sv);
          }
        }
        bool rise = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float x = s[nt][e] * qs[nt][e & 1];
            if constexpr (E8) x = fmaf(x, kc[e >> 1], vl[e >> 1]);
            if (key + 16 > sure && key + g + 8 * (e >> 1) >= limit[nt][e & 1]) x = -INFINITY;
            s[nt][e] = x;
            rise |= x > m[nt][e & 1] + Weights<M>::RAISE;
          }
        if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float top = fmaxf(s[nt][x], s[nt][2 + x]);
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
              top = fmaxf(top - Weights<M>::LIFT, m[nt][x]);
              const float f = top == -INFINITY ? 1.f : ex2(m[nt][x] - top);
              m[nt][x] = top;
              l[nt][x] *= f;
#pragma unroll
              for (int i = 0; i < STEPS; ++i) {
                o[nt][i][x] *= f;
                o[nt][i][2 + x] *= f;
              }
            }
        }
        uint32_t p[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float base = m[nt][e & 1];
            w[e] = ex2(s[nt][e] - (base == -INFINITY ? 0.f : base));
            l[nt][e & 1] = E8 ? fmaf(w[e], vi[e >> 1], l[nt][e & 1]) : l[nt][e & 1] + w[e];
          }
          p[nt][0] = transpose8x8(RowType<M>::pack2(w[0], w[1]));
          p[nt][1] = transpose8x8(RowType<M>::pack2(w[2], w[3]));
        }
        if constexpr (E8) {
#pragma unroll
          for (int i = 0; i < STEPS / 2; ++i) {  // 32 dims: dim 32 i + 4 g + x of tile x / 2
            uint32_t w[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const int r = 2 * t + (y & 1) + 8 * (y >> 1);
              w[y] = lds32(vs + piece<ROW>(r, 2 * i + (g >> 2)) + (g & 3) * 4);
            }
            const uint32_t lo01 = __byte_perm(w[0], w[1], 0x5140),
                           lo23 = __byte_perm(w[0], w[1], 0x7362),
                           hi01 = __byte_perm(w[2], w[3], 0x5140),
                           hi23 = __byte_perm(w[2], w[3], 0x7362);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma16816<M>(o[nt][2 * i], e4m3_to_half2(lo01), e4m3_to_half2(lo01 >> 16),
                          e4m3_to_half2(hi01), e4m3_to_half2(hi01 >> 16), p[nt][0], p[nt][1]);
              mma16816<M>(o[nt][2 * i + 1], e4m3_to_half2(lo23), e4m3_to_half2(lo23 >> 16),
                          e4m3_to_half2(hi23), e4m3_to_half2(hi23 >> 16), p[nt][0], p[nt][1]);
            }
          }
        } else {
          // matrix y = lane / 8: keys 8 (y / 2) .., dims 16 i + 8 (y % 2) ..
          const int r = (lane & 7) + 8 * (lane >> 4), ch = (lane >> 3) & 1;
#pragma unroll
          for (int i = 0; i < STEPS; ++i) {
            uint32_t v[4];
            ldmatrix_x4_trans(vs + piece<ROW>(r, 2 * i + ch), v);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma16816<M>(o[nt][i], v[0], v[1], v[2], v[3], p[nt][0], p[nt][1]);
          }
        }
      }
      stage = stage + 1 == STAGES ? 0 : stage + 1;
      at.skip(line, 1);
    }

    // ---- join the warps and write the segment: the rows' maxima first, then the sums of
    // all warps' values, 8 rows by COLS columns at a time, in the warps' order (half of the
    // warps left theirs to the other half in turn before: one token over 520 keys took 7.5
    // us instead of 7.0, 300 sequences of up to 300 43.4 instead of 41.1)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        l[nt][x] += __shfl_xor_sync(0xffffffffu, l[nt][x], 4);
        l[nt][x] += __shfl_xor_sync(0xffffffffu, l[nt][x], 8);
        l[nt][x] += __shfl_xor_sync(0xffffffffu, l[nt][x], 16);
        if (*(volatile int*)&f.gave_up) l[nt][x] = m[nt][x] = __int_as_float(0x7FC00000);
        if (g == 0) join_ml[warp * ROWS + nt * 8 + 2 * t + x] = make_float2(m[nt][x], l[nt][x]);
      }
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < WARPS; ++w)
          top = fmaxf(top, join_ml[w * ROWS + nt * 8 + 2 * t + x].x);
        const float f0 = ex2(m[nt][x] - (top == -INFINITY ? 0.f : top));
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
          o[nt][i][x] *= f0;
          o[nt][i][2 + x] *= f0;
        }
      }
    if (threadIdx.x < ROWS) {
      const int r = threadIdx.x;
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) top = fmaxf(top, join_ml[w * ROWS + r].x);
      const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float2 ml = join_ml[w * ROWS + r];
        sum += ex2(ml.x - base) * ml.y;
      }
      join_row[r] = make_float2(top, sum);
    }
    const bool whole = u.j == 0 && seg == u.n;
    const int tokens = u.s.n_new - u.i * tq, live = (tokens < tq ? tokens : tq) * a.group;
    const size_t slot = 2 * size_t(blockIdx.x) + (u.j == 0 ? 1 : 0);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int d0 = 0; d0 < HD; d0 += COLS) {
        if (nt + d0 > 0) __syncthreads();  // the last columns have been read
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (nt * 8 + 2 * t + x >= live) continue;
          float* to = join_o + (warp * 8 + 2 * t + x) * (COLS + 4) - d0;
#pragma unroll
          for (int i = d0 / 16; i < (d0 + COLS) / 16; ++i) {
            if constexpr (E8) {
              *reinterpret_cast<float2*>(to + 32 * (i >> 1) + 4 * g + 2 * (i & 1)) =
                  make_float2(o[nt][i][x], o[nt][i][2 + x]);
            } else {
              to[16 * i + g] = o[nt][i][x];
              to[16 * i + 8 + g] = o[nt][i][2 + x];
            }
          }
        }
        __syncthreads();
        for (int x = threadIdx.x; x < 8 * (COLS / 4); x += F::THREADS) {
          const int at8 = x / (COLS / 4), r = nt * 8 + at8, col = x % (COLS / 4) * 4;
          const int d = d0 + col;
          if (r >= live) break;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < WARPS; ++w) {
            const float4 y =
                *reinterpret_cast<const float4*>(join_o + (w * 8 + at8) * (COLS + 4) + col);
            acc.x += y.x;
            acc.y += y.y;
            acc.z += y.z;
            acc.w += y.w;
          }
          const float2 ml = join_row[r];
          if (whole) {
            const float inv = ml.y == 0.f ? 0.f : 1.0f / ml.y;
            const int head = u.h * a.group + r % a.group, token = u.i * tq + r / a.group;
            uint2 w;
            w.x = RowType<T>::pack2(acc.x * inv, acc.y * inv);
            w.y = RowType<T>::pack2(acc.z * inv, acc.w * inv);
            *reinterpret_cast<uint2*>(a.out + ((long long)(u.s.first + token) * a.o_ts +
                                               head * a.o_hs + d) * 2) = w;
            if (a.lse && d == 0)
              a.lse[(long long)(u.s.first + token) * a.q_heads + head] = row_lse(ml.x, ml.y);
          } else {
            *reinterpret_cast<float4*>(part.o + (slot * ROWS + r) * HD + d) = acc;
            if (d == 0) part.ml[slot * ROWS + r] = ml;
          }
        }
      }
    if (u.j == 0 && !whole && threadIdx.x == 0) {
      Left left = {(u.n - seg + per - 1) / per, u.s.first + u.i * tq, u.h, live};
      part.left[blockIdx.x] = left;
    }
    __syncthreads();  // the join buffer is free again
  }
  if (*(volatile int*)&f.gave_up)  // copies still on their way land before the CTA ends
    for (int st = 0; st < STAGES; ++st) {
      const uint64_t start = global_ns();
      while (!mbar_try_wait(&f.full[warp][st], (phases >> st & 1) ^ 1))
        if (global_ns() - start > uint64_t(FEW_WAIT_NS)) break;
    }
}

}  // namespace at
}  // namespace mk
