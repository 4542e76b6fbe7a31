// mk_flash.cuh -- attention of many query rows on the tensor cores: whole
// packed prompts, and chunks of new tokens over a paged cache.
//
// A unit's rows (tokens times the heads of the group) are tiles of 128, the M
// of tcgen05.mma; keys come in tiles of 128. For head_dim 64 and 128 two row
// tiles share every key tile (two streams, 256 rows); at 256 the output alone
// takes half of tensor memory and one row tile has two score buffers.
//
//   S = Q K^T   both from shared memory, 128 x 128 fp32 into TMEM
//   P = 2^(S c - m)  by two warpgroups, one or two threads for each row: scores from
//                    TMEM, weights back as 16-bit pairs over the scores' columns
//   O += P V    P from TMEM, V as it lies in memory (MN-major)
//
// Warps: one TMA producer, two MMA issuers, two softmax warpgroups.  While these work
// on one tile, the tensor cores run the other stream's products (or the next tile's
// scores and the last one's output).  The maximum of a row is raised only when a score
// passes it by far (mk_paged.cuh, Weights), and only then is O rescaled in TMEM;
// the sum of weights is kept in fp32 from the unrounded weights.  The weights' rounding to
// 16 bits is what the tensor cores' rate costs (operands in 32 bits would halve it and double
// V): in bf16 the root mean square error of the outputs is 2.3e-3 of them, 1.7e-3 with
// exact weights, which is the outputs' own rounding.
//
// K and V tiles: one TMA box of 64 dims by min(page, 128) positions each, the
// page looked up by the producer's lanes; boxes behind the last key and of
// pages outside the cache lie outside the tensor and arrive as zeros.  What the
// last page holds behind the sequence is zeroed in V before it is used (its
// scores are masked, but 0 * NaN is NaN).  An e4m3 cache has a warpgroup
// of converters in the producer's place: codes through registers to fp16
// tiles, exactly, the rows' scales beside them; queries become fp16 after a
// power of two for each row.  The converters set the pace there: each piece is a page
// lookup and a load behind it, one stage ahead (1024 tokens at 32768 keys, e4m3 / bf16: 219 /
// 105 us at head_dim 64, 1240 / 267 at 128, 2010 / 255 at 256).
//
// Every wait is bounded; one that runs out makes the CTA write NaN.
#pragma once
#include "mk_paged.cuh"
#include "mk_tc.cuh"

namespace mk {
namespace at {

constexpr int KEYS = 128;  // keys of a tile
constexpr long long FLASH_WAIT_NS = 2000000000LL;

template <int NQ>
struct FlashBars {
  uint64_t q_full, q_ready, q_empty;
  uint64_t full[2][8], empty[8];  // full: of keys, of values
  uint64_t s_full[2], p_full[2], o_full[2], o_empty[2];
  uint64_t sc_full[8];
  uint32_t tmem;
  int gave_up;
  int per;
  Cursor<KEYS> start;
  float trade[2][2][NQ == 1 ? 128 : 1];  // one stream: maxima and sums of a row's two halves
};

template <class C, int HD>
struct FlashCfg {
  static constexpr bool E8 = __is_same(C, E4m3);
  static constexpr int NQ = HD == 256 ? 1 : 2;  // row tiles (streams)
  static constexpr int CHUNKS = HD / 64;        // 64-value columns of an operand
  static constexpr int PARTS = HD == 256 ? 2 : 1;  // ring stages of a K or V tile
  static constexpr int VK = KEYS / PARTS;          // keys of a V stage
  static constexpr int KC = CHUNKS / PARTS;        // 64-value columns of a K stage
  static constexpr int STAGE = KEYS * KC * 128;    // bytes
  static constexpr int Q_TILE = 128 * HD * 2;
  static constexpr int STAGES = HD == 64 ? 8 : E8 ? 4 : 5;
  static constexpr int SCALES = E8 ? 8 : 0;  // tiles whose scales are kept
  // Two softmax warpgroups: one for each of two streams, or half of every tile's keys
  // each for one.
  static constexpr int HALVES = 2 / NQ, COLS = KEYS / HALVES, SOFT_WARPS = 8;
  static constexpr int THREADS = 128 + SOFT_WARPS * 32 + (E8 ? 128 : 0);
  static constexpr size_t SMEM = size_t(NQ) * Q_TILE + size_t(STAGES) * STAGE +
                                 size_t(SCALES) * 3 * KEYS * 4 + (E8 ? 4 * NQ * 128 * 4 : 0) +
                                 sizeof(FlashBars<NQ>);
  static_assert(SMEM <= 227 * 1024, "more shared memory than a block can have");
  // registers of a thread at launch, of softmax and of the others
  static constexpr int REGS = 65536 / THREADS / 8 * 8;
  static constexpr int REGS_REST = THREADS == 384 ? 72 : 56;
  static constexpr int REGS_SOFT =
      (REGS * THREADS - REGS_REST * (THREADS - SOFT_WARPS * 32)) / (SOFT_WARPS * 32) / 8 * 8;
  static_assert(REGS_SOFT * SOFT_WARPS * 32 + REGS_REST * (THREADS - SOFT_WARPS * 32) <=
                    REGS * THREADS,
                "the shares exceed what the block is launched with");
};
// A place in the ring of stages.  Keys and values share the ring but not the
// barriers that say a stage is full: an issuer that takes only keys (or only
// values) may be laps away from the others, where the parity of a shared barrier
// would mean nothing.  `phase` has a bit for each stage, [0] of its next load
// of keys and [1] of values.
template <int STAGES>
struct Ring {
  int stage = 0;
  uint32_t lap = 0, phase[2] = {0, 0};
  __device__ void next() {
    if (++stage == STAGES) {
      stage = 0;
      lap ^= 1;
    }
  }
  __device__ uint32_t flip(int v) {  // the parity of this load, and on to the next
    const uint32_t p = phase[v] >> stage & 1;
    phase[v] ^= 1u << stage;
    return p;
  }
};

template <int N>
__device__ __forceinline__ void more_registers() {
  if constexpr (N > 0) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  if constexpr (N > 0) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

struct FlashArgs {
  AttnArgs a;
  CUtensorMap q, k, v;  // q: (dim, head of the group, row, key head); k, v: (dim, position, head, page)
  int tq1;              // tokens of a row tile
  int box_shift;        // log2 of the positions of a K box
  int extra, least, whole;  // of the line (mk_split.cuh)
  int k_head, v_head;       // packed: a key head's place in k, v is `head & this`
};

// Called by whole warps; the answer is the same in every lane.
__device__ __forceinline__ bool flash_wait(uint64_t* bar, uint32_t parity, int* gave_up) {
  bool ok = true;
  uint64_t start = 0;
  while (!mbar_try_wait(bar, parity)) {
    const uint64_t now = global_ns();
    if (start == 0) start = now;
    if (now - start > uint64_t(FLASH_WAIT_NS) || *(volatile int*)gave_up) {
      *(volatile int*)gave_up = 1;
      ok = false;
      break;
    }
  }
  return __all_sync(0xffffffffu, ok);
}
// The cursor in a form that the compiler knows to be the same in every lane, so
// that what is computed from it stays in the warp's uniform registers.
__device__ __forceinline__ void make_uniform(Cursor<KEYS>& c) {
  c.s.first = uniform(c.s.first);
  c.s.n_new = uniform(c.s.n_new);
  c.s.len = uniform(c.s.len);
  c.b = uniform(c.b);
  c.h = uniform(c.h);
  c.i = uniform(c.i);
  c.j = uniform(c.j);
  c.n = uniform(c.n);
  c.nq = uniform(c.nq);
  c.at = uniform(c.at);
  c.left = uniform(c.left);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 32 bytes of a row: one access where the address allows it (rows start on 16).
__device__ __forceinline__ void store32(unsigned char* p, const uint32_t* w) {
  if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// {x0, x1} * {y, y} + {c, c}
__device__ __forceinline__ void fma2(float& x0, float& x1, float y, float c) {
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%0, %1};\n\t"
      "mov.b64 b, {%2, %2};\n\t"
      "mov.b64 d, {%3, %3};\n\t"
      "fma.rn.f32x2 a, a, b, d;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "f"(y), "f"(c));
}
__device__ __forceinline__ void add2(float& a, float& b, float x0, float x1) {
  asm("{\n\t.reg .b64 c, x;\n\t"
      "mov.b64 c, {%0, %1};\n\t"
      "mov.b64 x, {%2, %3};\n\t"
      "add.rn.f32x2 c, c, x;\n\t"
      "mov.b64 {%0, %1}, c;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(x0), "f"(x1));
}

template <class T, class C, int HD, bool PAGED>
__global__ void __launch_bounds__(FlashCfg<C, HD>::THREADS, 1)
    flash_kernel(const __grid_constant__ FlashArgs fa, Partials part) {
  using F = FlashCfg<C, HD>;
  constexpr bool E8 = F::E8, BF = !E8 && __is_same(T, Bf16);
  constexpr bool RESCALE_Q = E8 && __is_same(T, Bf16);
  constexpr int HALVES = F::HALVES, COLS = F::COLS;
  constexpr int NQ = F::NQ, STAGES = F::STAGES, PARTS = F::PARTS, CHUNKS = F::CHUNKS;
  using M = typename std::conditional<E8, Fp16, T>::type;
  const AttnArgs& a = fa.a;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t base = smem_addr(smem);
  unsigned char* base_ptr = smem;
  const uint32_t sq = base, ring = base + NQ * F::Q_TILE;
  float* scales = reinterpret_cast<float*>(base_ptr + NQ * F::Q_TILE + STAGES * F::STAGE);
  // sizes of the queries' rows, [4][NQ * 128]: with one stream the scores of two more
  // segments may come before the softmax of one reads them
  float* q_size = scales + F::SCALES * 3 * KEYS;
  FlashBars<NQ>& f =
      *reinterpret_cast<FlashBars<NQ>*>(q_size + (E8 ? 4 * NQ * 128 : 0));
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const Line<KEYS> line{a, NQ * fa.tq1, fa.extra, fa.whole != 0};
  const int tq1 = fa.tq1, tile_rows = tq1 * a.group;

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
  } else if (warp == 1) {
    tmem_alloc(&f.tmem, 512);
  } else if (warp == 2 && lane == 0) {
    mbar_init(&f.q_full, 1);
    mbar_init(&f.q_ready, 4);
    mbar_init(&f.q_empty, NQ);
    for (int i = 0; i < 8; ++i) {
      mbar_init(&f.full[0][i], E8 ? 4 : 1);
      mbar_init(&f.full[1][i], E8 ? 4 : 1);
      mbar_init(&f.empty[i], NQ);
      mbar_init(&f.sc_full[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&f.s_full[i], 1);
      mbar_init(&f.p_full[i], F::SOFT_WARPS / NQ);
      mbar_init(&f.o_full[i], 1);
      mbar_init(&f.o_empty[i], F::SOFT_WARPS / NQ);
    }
    fence_barrier_init();
  } else if (warp == 3 && lane == 0) {
    prefetch_map(&fa.q);
    if (!E8) {
      prefetch_map(&fa.k);
      prefetch_map(&fa.v);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();
  const uint32_t tmem = 0;  // all 512 columns: the allocation starts at the first
  Cursor<KEYS> at = f.start;
  make_uniform(at);

  // streams of a unit: the second row tile may have no tokens
  auto streams = [&](const Cursor<KEYS>& u) {
    return NQ == 2 && u.s.n_new - u.i * NQ * tq1 > tq1 ? 2 : 1;
  };
  // end of stream s's key tiles within a segment that ends at tile `end`
  auto stream_end = [&](const Cursor<KEYS>& u, int s, int end) {
    if (NQ == 1 || s == 1) return end;
    const int last = u.i * NQ * tq1 + tq1;
    const int limit = u.s.len - u.s.n_new + (last < u.s.n_new ? last : u.s.n_new);
    const int n = limit <= KEYS ? 1 : (limit + KEYS - 1) / KEYS;
    return n < end ? n : end;
  };

  // Each warpgroup changes its registers inside its own branch: code after a
  // common point would be held to the smallest share.
  if (warp < 4) {
    fewer_registers<F::REGS_REST>();
    if (warp == 0) {
      // ---- TMA producer: queries, and keys and values unless they are converted
      Ring<STAGES> to;
      int seg_no = 0;
      while (at.left > 0) {
        const int seg = at.segment(line), ns = streams(at);
        bool ok = seg_no == 0 || flash_wait(&f.q_empty, (seg_no - 1) & 1, &f.gave_up);
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&f.q_full, ns * CHUNKS * tile_rows * 128);
          for (int s = 0; s < ns; ++s)
            for (int c = 0; c < CHUNKS; ++c)
              tma_load_4d(sq + s * F::Q_TILE + c * (128 * 128), &fa.q, c * 64, 0,
                          at.s.first + at.i * NQ * tq1 + s * tq1, at.h, &f.q_full);
        }
        __syncwarp();
        if constexpr (!E8) {
          const int limit = line.limit(at.s, at.i), end = at.j + seg;
          const int shift = PAGED ? fa.box_shift : 7;
          // lane b: the page of box b of the tile, looked up a tile ahead
          auto pages_of = [&](int j) {
            int page = a.c.n_pages;
            if constexpr (PAGED) {
              const int key = j * KEYS + (lane << shift);
              if ((lane << shift) < KEYS && key < limit) {
                page = a.table[(long long)at.b * a.table_stride + (key >> a.c.page_shift)];
                if (page < 0 || page >= a.c.n_pages) page = a.c.n_pages;
              }
            }
            return page;
          };
          auto load = [&](bool v, int j, int pages) {
            for (int p = 0; p < PARTS; ++p, to.next()) {
              const int st = to.stage;
              // (a fresh barrier's phase before the first counts as complete)
              if (!flash_wait(&f.empty[st], to.lap ^ 1, &f.gave_up)) return false;
              to.flip(v);
              uint64_t* full = &f.full[v][st];
              const int rows = v && F::VK < (1 << shift) ? F::VK : 1 << shift;  // of a box
              const int n_rows = v ? F::VK : KEYS, cols = v ? CHUNKS : F::KC;
              if (elect_one()) mbar_arrive_expect_tx(full, F::STAGE);
              for (int row = 0; row < n_rows; row += rows) {
                const int key = row + (v ? p * F::VK : 0);  // in the tile
                const int page = __shfl_sync(0xffffffffu, pages, key >> shift);
                const int head = PAGED ? at.h : at.h & (v ? fa.v_head : fa.k_head);
                const int pos = PAGED ? (j * KEYS + key) & (a.c.page_size - 1)
                                      : at.s.first + j * KEYS + key;
                if (elect_one()) {
                  const uint32_t dst = ring + st * F::STAGE + row * 128;
                  for (int c = 0; c < cols; ++c)
                    tma_load_4d(dst + c * (n_rows * 128), v ? &fa.v : &fa.k,
                                (c + (v ? 0 : p * F::KC)) * 64, pos, head, PAGED ? page : 0, full);
                }
                __syncwarp();
              }
            }
            return true;
          };
          int now = pages_of(at.j), next = pages_of(at.j + 1 < end ? at.j + 1 : at.j);
          ok = load(false, at.j, now);
          for (int j = at.j; ok && j < end; ++j) {
            if (NQ == 1) {  // scores run a tile ahead of the output
              if (j + 1 < end) ok = load(false, j + 1, next);
              ok = ok && load(true, j, now);
            } else {
              ok = load(true, j, now);
              if (j + 1 < end) ok = ok && load(false, j + 1, next);
            }
            now = next;
            next = pages_of(j + 2 < end ? j + 2 : at.j);
          }
          if (!ok) break;
        }
        at.skip(line, seg);
        make_uniform(at);
        ++seg_no;
      }
      // copies in flight must land before the CTA can end
      if (seg_no > 0) flash_wait(&f.q_full, (seg_no - 1) & 1, &f.gave_up);
      if (!E8)
        for (int i = 0; i < STAGES; ++i)
          for (int v = 0; v < 2; ++v) {  // the last load of each kind (of none: complete at once)
            const uint64_t start = global_ns();
            while (!mbar_try_wait(&f.full[v][i], (to.phase[v] >> i & 1) ^ 1))
              if (global_ns() - start > uint64_t(FLASH_WAIT_NS)) break;
          }
    } else if (warp <= 2) {
      // ---- MMA issuers.  Two streams: warp 1 + s issues the scores and outputs of
      // stream s.  One stream: warp 1 issues the scores, warp 2 the outputs.
      constexpr uint32_t id_s = idesc_f16(BF, 128, KEYS, false), id_o = idesc_f16(BF, 128, HD, true);
      const int me = warp - 1;
      Ring<STAGES> ring_at;
      int seg_no = 0, cnt = 0, segs = 0;  // segments, own key tiles, own segments so far
      auto on = [](int stage) { return stage + 1 == STAGES ? 0 : stage + 1; };
      auto issue_s = [&](int slot, int q, int st) {
        uint64_t qd = desc_k_major(sq + q * F::Q_TILE);
#pragma unroll
        for (int p = 0; p < PARTS; ++p, st = on(st)) {
          uint64_t kd = desc_k_major(ring + st * F::STAGE);
#pragma unroll
          for (int c = 0; c < F::KC; ++c, qd += 128 * 128 / 16, kd += KEYS * 128 / 16)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc_mma(tmem + slot * KEYS, qd + k * 2, kd + k * 2, id_s, p + c + k > 0);
        }
      };
      // the weights lie over the scores, those of a half over its own
      auto weights_at = [](int key) { return key / 2 + (HALVES == 2 && key >= 64 ? 32 : 0); };
      auto issue_o = [&](int slot, int s, int st, bool more) {
#pragma unroll
        for (int p = 0; p < PARTS; ++p, st = on(st)) {
          const uint64_t vd = desc_mn_major(ring + st * F::STAGE, F::VK * 128);
#pragma unroll
          for (int k = 0; k < F::VK / 16; ++k)
            tc_mma_ts(tmem + 256 + s * HD, tmem + slot * KEYS + weights_at(p * F::VK + k * 16),
                      vd + k * (2048 / 16), id_o, more || p + k > 0);
        }
      };
      // Waits for the operand in the ring's next stages and moves past it; its first stage.
      auto take = [&](int v, int& first) {
        first = ring_at.stage;
        bool ok = true;
#pragma unroll
        for (int p = 0; p < PARTS; ++p, ring_at.next())
          ok = ok && flash_wait(&f.full[v][ring_at.stage], ring_at.flip(v), &f.gave_up);
        return ok;
      };
      auto pass = [&] {
#pragma unroll
        for (int p = 0; p < PARTS; ++p) ring_at.next();
      };
      auto release = [&](int st) {
#pragma unroll
        for (int p = 0; p < PARTS; ++p, st = on(st)) tc_commit(&f.empty[st]);
      };
      // Zero what lies behind the sequence in a V tile (both streams' issuers do: zeros
      // over zeros).
      auto clear_tail = [&](int st, int j) {
        if constexpr (!E8) {
          const int keep = at.s.len - j * KEYS;
          if (keep >= KEYS) return;
          for (int p = 0; p < PARTS; ++p, st = on(st))
            for (int x = lane; x < F::VK * 8; x += 32) {
              if (x / 8 + p * F::VK < keep) continue;
              const uint32_t to = ring + st * F::STAGE + x * 16;
              for (int c = 0; c < CHUNKS; ++c)
                asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(to + c * F::VK * 128),
                             "r"(0)
                             : "memory");
            }
          fence_async_smem();
          __syncwarp();
        }
      };
      bool ok = true;
      while (at.left > 0 && ok) {
        const int seg = at.segment(line), end = at.j + seg, ns = streams(at);
        // (whoever issues scores; the outputs' issuer of one stream may be two segments
        // behind, where the barrier's parity says nothing)
        if (NQ == 2 || me == 0)
          ok = flash_wait(RESCALE_Q ? &f.q_ready : &f.q_full, seg_no & 1, &f.gave_up);
        int k_at, v_at;
        if constexpr (NQ == 2) {
          const bool active = me < ns;
          const int e = !active ? at.j : me == 0 ? stream_end(at, 0, end) : end;
          ok = ok && take(0, k_at);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            if (at.j < e) {
              issue_s(me, me, k_at);
              tc_commit(&f.s_full[me]);
            }
            release(k_at);
            if (seg == 1) tc_commit(&f.q_empty);
          }
          for (int j = at.j; j < end && ok; ++j) {
            const bool more = j + 1 < end;
            ok = take(1, v_at);
            if (!ok) break;
            if (j < e) {
              clear_tail(v_at, j);
              // O is free once the epilogue of the stream's last segment has read it
              if (j == at.j && segs > 0) ok = flash_wait(&f.o_empty[me], (segs - 1) & 1, &f.gave_up);
              ok = ok && flash_wait(&f.p_full[me], cnt & 1, &f.gave_up);
              if (!ok) break;
              tc_fence_after();
              if (elect_one()) {
                issue_o(me, me, v_at, j > at.j);
                tc_commit(&f.o_full[me]);
                release(v_at);
              }
              ++cnt;
            } else if (elect_one()) {
              release(v_at);
            }
            if (more) {
              ok = take(0, k_at);
              if (!ok) break;
              tc_fence_after();
              if (elect_one()) {
                if (j + 1 < e) {
                  issue_s(me, me, k_at);
                  tc_commit(&f.s_full[me]);
                }
                release(k_at);
                if (j + 2 == end) tc_commit(&f.q_empty);
              }
            }
          }
          if (active) {
            // a stream without tiles here keeps step with its epilogues all the same
            if (ok && e <= at.j && segs > 0) ok = flash_wait(&f.o_empty[me], (segs - 1) & 1, &f.gave_up);
            ++segs;
          }
        } else if (me == 0) {
          for (int x = 0; x < seg && ok; ++x, ++cnt) {
            ok = take(0, k_at);
            // the scores' columns are free once the output has used the weights in them
            if (ok && cnt > 1) ok = flash_wait(&f.o_full[cnt & 1], ((cnt >> 1) - 1) & 1, &f.gave_up);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              issue_s(cnt & 1, 0, k_at);
              tc_commit(&f.s_full[cnt & 1]);
              release(k_at);
              if (x + 1 == seg) tc_commit(&f.q_empty);
            }
            if (x > 0) pass();         // the V tile behind it
            if (x + 1 == seg) pass();  // the last one
          }
        } else {
          pass();  // the first K tile
          for (int j = at.j; j < end && ok; ++j, ++cnt) {
            if (j + 1 < end) pass();
            ok = take(1, v_at);
            if (!ok) break;
            clear_tail(v_at, j);
            if (j == at.j && segs > 0) ok = flash_wait(&f.o_empty[0], (segs - 1) & 1, &f.gave_up);
            ok = ok && flash_wait(&f.p_full[cnt & 1], (cnt >> 1) & 1, &f.gave_up);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              issue_o(cnt & 1, 0, v_at, j > at.j);
              tc_commit(&f.o_full[cnt & 1]);
              release(v_at);
            }
          }
          ++segs;
        }
        at.skip(line, seg);
        make_uniform(at);
        ++seg_no;
      }
      __syncwarp();
    }
  } else if (warp < 4 + F::SOFT_WARPS) {
    // ---- softmax and epilogue.  Two streams: a thread for each row of its warpgroup's
    // stream.  (Two threads a row, 64 keys each, made the streams run in step, both at
    // the exponential unit and then both at the tensor cores: 4450 cycles a key
    // tile at head_dim 128 where this takes 3140.)  One stream: two threads a row, which halves
    // the time from scores to weights and the epilogue (2300 cycles a key tile, 2560 with
    // one).
    more_registers<F::REGS_SOFT>();
    const int group = (warp - 4) >> 2, quarter = warp & 3;
    const int s = NQ == 2 ? group : 0, half = NQ == 2 ? 0 : group;
    const int r = quarter * 32 + lane;
    const uint32_t lanes = tmem + (uint32_t(quarter * 32) << 16);
    int cnt = 0, seg_no = 0, tiles = 0;  // own key tiles, segments, all key tiles so far
    uint32_t turn = 0;                   // buffer of the next trade
    // The other half's number for this row; the two warps meet at their own barrier.
    // Every warp makes every trade, also after a wait that ran out: they meet as often.
    // (The buffers alternate: a trade's number is read before the next but one, which
    // follows another meeting.)
    auto trade = [&](float x) {
      f.trade[turn][half][r] = x;
      named_sync(1 + quarter, 64);
      const float y = f.trade[turn][half ^ 1][r];
      turn ^= 1;
      return y;
    };
    // The output through key tile x.  Its barrier goes by the score buffer: with one
    // stream the scores of tile x + 1 come before the output of tile x, so that two
    // outputs may be due at once, and one barrier's parity could not tell them apart.
    auto wait_output = [&](int x) {
      return flash_wait(&f.o_full[NQ == 1 ? x & 1 : s], (NQ == 1 ? x >> 1 : x) & 1, &f.gave_up);
    };
    while (at.left > 0) {
      const Cursor<KEYS> u = at;
      const int seg = u.segment(line), end = u.j + seg;
      at.skip(line, seg);
      make_uniform(at);
      const int seg_at = seg_no++, tile0 = tiles - u.j;
      tiles += seg;
      if (s >= streams(u)) continue;
      const int e = stream_end(u, s, end);
      const int token = (u.i * NQ + s) * tq1 + r / a.group;
      const bool live = r < tile_rows && token < u.s.n_new;
      const int limit = live ? u.s.len - u.s.n_new + token + 1 : 0;
      const int sure = u.s.len - u.s.n_new + (u.i * NQ + s) * tq1 + 1;  // every row sees so many
      const bool any_live = __any_sync(0xffffffffu, live);
      float m = -INFINITY, l0 = 0.f, l1 = 0.f;  // m in powers of two
      float c = a.scale_log2;
      bool ok = true;
      for (int j = u.j; j < e; ++j, ++cnt) {
        const int slot = NQ == 1 ? cnt & 1 : s;
        const uint32_t scores = lanes + slot * KEYS + half * COLS;
        const float* sc = scales + ((tile0 + j) & 7) * 3 * KEYS + half * COLS;
        ok = ok && flash_wait(&f.s_full[slot], (NQ == 1 ? cnt >> 1 : cnt) & 1, &f.gave_up);
        if constexpr (E8)
          ok = ok && flash_wait(&f.sc_full[(tile0 + j) & 7], (tile0 + j) >> 3 & 1, &f.gave_up);
        // (the converters wrote it before the first tile's scales)
        if (RESCALE_Q && j == u.j)
          c = a.scale_log2 * q_size[(seg_at & 3) * NQ * 128 + s * 128 + r];
        if (any_live) {
          // 16-bit caches keep the scores in registers; with an e4m3 cache's scales in the
          // way they are fetched from TMEM again, 32 at a time, for the weights.
          constexpr int HELD = E8 ? 32 : COLS;
          float x[HELD];
          const int keep = limit - j * KEYS - half * COLS;
          const bool masked = j * KEYS + KEYS > sure;
          auto fetch = [&](int from) {
            if (ok) {
              tc_fence_after();
#pragma unroll
              for (int i = 0; i < HELD; i += 32) tmem_ld32(scores + from + i, x + i);
              tmem_wait_ld();
            }
#pragma unroll
            for (int i = 0; i < HELD; ++i) pin(x[i]);
            if constexpr (E8) {
#pragma unroll
              for (int i = 0; i < HELD; i += 4) {
                const float4 kc = *reinterpret_cast<const float4*>(sc + from + i);
                const float4 vl = *reinterpret_cast<const float4*>(sc + KEYS + from + i);
                x[i] = fmaf(x[i] * c, kc.x, vl.x);
                x[i + 1] = fmaf(x[i + 1] * c, kc.y, vl.y);
                x[i + 2] = fmaf(x[i + 2] * c, kc.z, vl.z);
                x[i + 3] = fmaf(x[i + 3] * c, kc.w, vl.w);
              }
            }
            if (masked) {
#pragma unroll
              for (int i = 0; i < HELD; ++i) x[i] = from + i < keep ? x[i] : -INFINITY;
            }
          };
          auto largest = [&](float t0) {
            float t1 = x[0];
#pragma unroll
            for (int i = 1; i + 3 < HELD; i += 4) {
              t0 = max3(t0, x[i], x[i + 1]);
              t1 = max3(t1, x[i + 2], x[i + 3]);
            }
            t0 = max3(t0, x[HELD - 3], x[HELD - 2]);
            return max3(t0, t1, x[HELD - 1]);
          };
          float t0 = -INFINITY;
#pragma unroll
          for (int from = 0; from < COLS; from += HELD) {
            fetch(from);
            t0 = largest(t0);
          }
          const float unit = E8 ? 1.f : c;
          float top = t0 * unit;
          if (HALVES == 2) top = fmaxf(top, trade(top));
          const bool rise = top > m + Weights<M>::RAISE;
          if (__any_sync(0xffffffffu, rise)) {
            const float up = rise ? top - Weights<M>::LIFT : m;
            const float fac = rise ? ex2(m - up) : 1.f;
            l0 *= fac;
            l1 *= fac;
            m = up;
            if (j > u.j) {
              // the last tile's output is complete; scale this half of its columns
              ok = ok && wait_output(cnt - 1);
              tc_fence_after();
#pragma unroll 1
              for (int d = half * (HD / HALVES); ok && d < (half + 1) * (HD / HALVES); d += 32) {
                float o[32];
                tmem_ld32(lanes + 256 + s * HD + d, o);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                  pin(o[i]);
                  o[i] *= fac;
                }
                tmem_st32(lanes + 256 + s * HD + d, o);
              }
            }
          }
          const float off = m == -INFINITY ? 0.f : -m;
          const float* vi = sc + 2 * KEYS;
          uint32_t held[E8 ? COLS / 2 : 1];
#pragma unroll
          for (int i = 0; i < COLS; i += 32) {
            uint32_t p[16];
            if (HELD == 32) fetch(i);
#pragma unroll
            for (int y = 0; y < 32; y += 2) {
              float &p0 = x[i % HELD + y], &p1 = x[i % HELD + y + 1];
              fma2(p0, p1, unit, off);
              p0 = ex2(p0);
              p1 = ex2(p1);
              if constexpr (E8) {
                const float2 w = *reinterpret_cast<const float2*>(vi + i + y);
                l0 = fmaf(p0, w.x, l0);
                l1 = fmaf(p1, w.y, l1);
              } else {
                add2(l0, l1, p0, p1);
              }
              p[y / 2] = RowType<M>::pack2(p0, p1);
            }
            if (HELD == 32) {
              // (they go over scores that are still to be fetched)
#pragma unroll
              for (int y = 0; y < 16; ++y) held[i / 2 + y] = p[y];
            } else if (ok) {
              tmem_st16(scores + i / 2, p);
            }
          }
          if (HELD == 32 && ok) {
#pragma unroll
            for (int i = 0; i < COLS / 2; i += 16) tmem_st16(scores + i, held + i);
          }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&f.p_full[slot]);
      }
      // ---- epilogue
      if (ok && e > u.j) ok = wait_output(cnt - 1);
      tc_fence_after();
      const bool whole = u.j == 0 && seg == u.n;
      float l = l0 + l1;
      if (HALVES == 2) l += trade(l);
      if (!ok || *(volatile int*)&f.gave_up) {
        ok = false;
        l = m = __int_as_float(0x7FC00000);  // a wait ran out: NaN
      }
      const float inv = l == 0.f ? 0.f : 1.0f / l;
      const int head = u.h * a.group + r % a.group;
      const long long row = u.s.first + (live ? token : 0);
      const size_t slot = 2 * size_t(blockIdx.x) + (u.j == 0 ? 1 : 0);
      const int part_row = s * tile_rows + r;
      if (any_live) {
        // A thread has its row (or half of it), 32 columns at a time.  A finished row leaves in
        // whole 32-byte sectors; partial rows lie side by side, [column / 4][row] float4, so
        // that a warp's store is 512 bytes in a piece.  (Trading values between lanes until
        // rows leave in 64-byte pieces took 4900 cycles a segment at head_dim 128, all of it
        // instructions; 16 bytes a lane straight to rows of fp32 10000.)
        const bool none = e <= u.j;  // no tiles here: O is not this segment's
        unsigned char* out = a.out + (row * a.o_ts + head * a.o_hs) * 2;
        float4* pieces = reinterpret_cast<float4*>(part.o) +
                         slot * (HD / 4) * (NQ * 128) + part_row;
        const int d0 = half * (HD / HALVES);
        float o[32];
        tmem_ld32(lanes + 256 + s * HD + d0, o);
#pragma unroll 1
        for (int d = d0; d < d0 + HD / HALVES; d += 32) {
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            pin(o[i]);
            if (none || !ok) o[i] = ok ? 0.f : l;
          }
          if (live && whole) {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              mul2(o[i], o[i + 1], inv, inv);
              w[i / 2] = RowType<T>::pack2(o[i], o[i + 1]);
            }
            store32(out + d * 2, w);
            store32(out + d * 2 + 32, w + 8);
          } else if (live) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              pieces[(d + i) / 4 * (NQ * 128)] = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          }
          if (d + 32 < d0 + HD / HALVES) tmem_ld32(lanes + 256 + s * HD + d + 32, o);
        }
        if (live && half == 0) {
          if (!whole)
            part.ml[slot * (NQ * 128) + part_row] = make_float2(m, l);
          else if (a.lse)
            a.lse[row * a.q_heads + head] = row_lse(m, l);
        }
      }
      if (s == 0 && half == 0 && r == 0 && u.j == 0 && !whole) {
        const int tokens = u.s.n_new - u.i * NQ * tq1;
        Left left = {(u.n - seg + f.per - 1) / f.per, u.s.first + u.i * NQ * tq1, u.h,
                     (tokens < NQ * tq1 ? tokens : NQ * tq1) * a.group};
        part.left[blockIdx.x] = left;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&f.o_empty[s]);
    }
  } else if constexpr (E8) {
    // ---- converters of an e4m3 cache (and of bf16 queries that meet it)
    fewer_registers<F::REGS_REST>();
    const int ct = tid - 128 - F::SOFT_WARPS * 32;
    constexpr int N = F::STAGE / 32 / 128;  // 16-code pieces of a thread and stage
    int it = 0, seg_no = 0, tiles = 0;
    while (at.left > 0) {
      const int seg = at.segment(line), end = at.j + seg, ns = streams(at);
      bool ok = true;
      if constexpr (RESCALE_Q) {
        ok = flash_wait(&f.q_full, seg_no & 1, &f.gave_up);
        if (!ok) break;
        for (int s = 0; s < ns; ++s) {
          const uint32_t row = sq + s * F::Q_TILE + ct * 128;
          float size = 0.f;
#pragma unroll 4
          for (int x = 0; x < CHUNKS * 8; ++x) {  // the lanes' pieces turned: no bank conflicts
            const uint4 w = lds128(row + (x >> 3) * (128 * 128) + (((x + ct) & 7) << 4));
            float v[8];
            RowType<Bf16>::unpack(w, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) size = fmaxf(size, fabsf(v[i]));
          }
          uint32_t ex = __float_as_uint(size) >> 23;
          ex = ex < 1 ? 1 : ex > 253 ? 253 : ex;
          const float down = __uint_as_float((254 - ex) << 23);
          q_size[(seg_no & 3) * NQ * 128 + s * 128 + ct] = __uint_as_float(ex << 23);
#pragma unroll 4
          for (int x = 0; x < CHUNKS * 8; ++x) {
            const uint32_t p = row + (x >> 3) * (128 * 128) + (((x + ct) & 7) << 4);
            const uint4 w = lds128(p);
            float v[8];
            RowType<Bf16>::unpack(w, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= down;
            const uint4 h = RowType<Fp16>::pack(v);
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(p), "r"(h.x), "r"(h.y),
                         "r"(h.z), "r"(h.w)
                         : "memory");
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&f.q_ready);
      }
      // (plain loads of the table, codes and scales: this kernel is there before the one in
      // front has written them, so they are not constant while it lives)
      // stage n of the segment in the order in which the issuer takes them
      const int len = at.s.len, j0 = at.j;
      auto what = [&](int n, bool& v, int& j, int& p) {
        const int x = n / PARTS;
        p = n % PARTS;
        if (NQ == 2) {
          v = x & 1;
          j = j0 + (x >> 1);
        } else if (x & 1) {
          v = (x + 1) / 2 >= seg;
          j = v ? end - 1 : j0 + (x + 1) / 2;
        } else {
          v = x > 0;
          j = x > 0 ? j0 + x / 2 - 1 : j0;
        }
      };
      auto place = [&](int x, bool v, int& row, int& pc) {
        const int per = v ? CHUNKS * 4 : F::KC * 4;
        row = x / per;
        pc = x % per;
      };
      auto page_of = [&](int key) {
        const int page =
            key < len ? a.table[(long long)at.b * a.table_stride + (key >> a.c.page_shift)] : -1;
        return page < a.c.n_pages ? page : -1;
      };
      auto load = [&](int n, uint4 (&w)[N]) {
        bool v;
        int j, p;
        what(n, v, j, p);
        const unsigned char* src = v ? a.c.v : a.c.k;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          int row, pc;
          place(i * 128 + ct, v, row, pc);
          const int key = j * KEYS + (v ? p * F::VK : 0) + row;
          const int page = page_of(key);
          w[i] = make_uint4(0, 0, 0, 0);
          if (page >= 0)
            w[i] = *reinterpret_cast<const uint4*>(
                src + page * a.c.page_stride + at.h * a.c.head_stride +
                (key & (a.c.page_size - 1)) * a.c.pos_stride + (v ? 0 : p * F::KC * 64) + pc * 16);
        }
      };
      uint4 cur[N], next[N];
      load(0, cur);
      for (int n = 0; n < 2 * seg * PARTS; ++n, ++it) {
        bool v;
        int j, p;
        what(n, v, j, p);
        float ks = 0.f, vs = 1.f;
        const bool first = !v && p == 0;
        if (first) {
          const int key = j * KEYS + ct, page = page_of(key);
          if (page >= 0) {
            const long long at_scale =
                (((long long)page * a.c.kv_heads + at.h) << a.c.page_shift) +
                (key & (a.c.page_size - 1));
            ks = a.c.k_scale[at_scale];
            vs = a.c.v_scale[at_scale];
          }
        }
        if (n + 1 < 2 * seg * PARTS) load(n + 1, next);
        const int st = it % STAGES;
        ok = it < STAGES || flash_wait(&f.empty[st], (it / STAGES - 1) & 1, &f.gave_up);
        if (!ok) break;
        const int rows = v ? F::VK : KEYS;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          int row, pc;
          place(i * 128 + ct, v, row, pc);
          const uint32_t to = ring + st * F::STAGE + ((pc >> 2) * rows + row) * 128;
          const uint32_t x = (pc & 3) * 2, turn = row & 7;
          asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(to + ((x ^ turn) << 4)),
                       "r"(e4m3_to_half2(cur[i].x)), "r"(e4m3_to_half2(cur[i].x >> 16)),
                       "r"(e4m3_to_half2(cur[i].y)), "r"(e4m3_to_half2(cur[i].y >> 16))
                       : "memory");
          asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(to + (((x + 1) ^ turn) << 4)),
                       "r"(e4m3_to_half2(cur[i].z)), "r"(e4m3_to_half2(cur[i].z >> 16)),
                       "r"(e4m3_to_half2(cur[i].w)), "r"(e4m3_to_half2(cur[i].w >> 16))
                       : "memory");
        }
        if (first) {
          const int slot = (tiles + j - j0) & 7;
          float* to = scales + slot * 3 * KEYS + ct;
          to[0] = ks;
          to[KEYS] = log2f(vs);
          to[2 * KEYS] = 1.0f / vs;
          __syncwarp();
          if (lane == 0) mbar_arrive(&f.sc_full[slot]);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&f.full[v][st]);
#pragma unroll
        for (int i = 0; i < N; ++i) cur[i] = next[i];
      }
      if (!ok) break;
      tiles += seg;
      at.skip(line, seg);
      make_uniform(at);
      ++seg_no;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(f.tmem, 512);
}

}  // namespace at
}  // namespace mk
