// mk_ops.cu -- host side of the operators of an attention layer over a paged
// cache (include/mk.h): argument checks and launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "mk.h"
#include "mk_attn.cuh"
#include "mk_flash.cuh"
#include "mk_kvcache.cuh"
#include "mk_paged.cuh"
#include "mk_rope.cuh"

namespace {

int launched() {
  const cudaError_t r = cudaGetLastError();
  if (r == cudaSuccess) return MK_OK;
  return r == cudaErrorInvalidConfiguration || r == cudaErrorLaunchOutOfResources ? MK_ERR_LAUNCH
                                                                                 : MK_ERR_CUDA;
}

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool half_type(int dtype) { return dtype == MK_BF16 || dtype == MK_FP16; }
int value_size(int dtype) { return dtype == MK_FP32 ? 4 : dtype == MK_E4M3 ? 1 : 2; }

// Rows whose 16-byte pieces the kernels read and write.
bool rows_ok(const void* p, int64_t ts, int64_t hs, int size) {
  return p && aligned(p, 16) && ts >= 0 && hs >= 0 && (ts * size) % 16 == 0 &&
         (hs * size) % 16 == 0 && ts < (int64_t(1) << 38) && hs < (int64_t(1) << 38);
}

bool head_dim_ok(int hd) { return hd == 64 || hd == 128 || hd == 256; }

// MK_OK and the kernels' view of a cache, or the error of a bad one.
int cache_view(const mk_kv_cache* c, mk::PagedView* v) {
  if (!c || c->n_pages <= 0 || c->kv_heads <= 0 || c->page_size <= 0) return MK_ERR_ARG;
  if (c->dtype != MK_BF16 && c->dtype != MK_FP16 && c->dtype != MK_E4M3) return MK_ERR_ARG;
  if (!head_dim_ok(c->head_dim)) return MK_ERR_UNSUPPORTED;
  int shift = 0;
  while ((1 << shift) < c->page_size) ++shift;
  if ((1 << shift) != c->page_size || c->page_size < 16 || c->page_size > 256)
    return MK_ERR_UNSUPPORTED;
  const int size = value_size(c->dtype);
  if (!rows_ok(c->k, c->page_stride, c->head_stride, size) ||
      !rows_ok(c->v, c->page_stride, c->pos_stride, size))
    return MK_ERR_ARG;
  // rows must not overlap
  if (c->pos_stride < c->head_dim || (c->kv_heads > 1 && c->head_stride < c->head_dim) ||
      (c->n_pages > 1 && c->page_stride < c->head_dim))
    return MK_ERR_ARG;
  if (c->dtype == MK_E4M3 && (!c->k_scale || !c->v_scale || !aligned(c->k_scale, 4) ||
                              !aligned(c->v_scale, 4)))
    return MK_ERR_ARG;
  v->k = static_cast<unsigned char*>(c->k);
  v->v = static_cast<unsigned char*>(c->v);
  v->k_scale = c->k_scale;
  v->v_scale = c->v_scale;
  v->page_stride = c->page_stride;
  v->head_stride = c->head_stride;
  v->pos_stride = c->pos_stride;
  v->n_pages = c->n_pages;
  v->page_size = c->page_size;
  v->page_shift = shift;
  v->kv_heads = c->kv_heads;
  v->head_dim = c->head_dim;
  return MK_OK;
}

template <class T>
struct Tag {
  using type = T;
};
template <int N>
struct Num {
  static constexpr int value = N;
};

// f(Tag of the row type); f(Num of the head dim)
template <class F>
void by_row_type(int dtype, F f) {
  if (dtype == MK_BF16) f(Tag<mk::Bf16>{});
  else if (dtype == MK_FP16) f(Tag<mk::Fp16>{});
  else f(Tag<mk::Fp32>{});
}
template <class F>
void by_half_type(int dtype, F f) {
  if (dtype == MK_BF16) f(Tag<mk::Bf16>{});
  else f(Tag<mk::Fp16>{});
}
template <class F>
void by_cache_type(int dtype, F f) {
  if (dtype == MK_BF16) f(Tag<mk::Bf16>{});
  else if (dtype == MK_FP16) f(Tag<mk::Fp16>{});
  else f(Tag<mk::E4m3>{});
}
template <class F>
void by_head_dim(int hd, F f) {
  if (hd == 64) f(Num<64>{});
  else if (hd == 128) f(Num<128>{});
  else f(Num<256>{});
}

int blocks_for(long long items, int per_block, unsigned* blocks) {
  const long long n = (items + per_block - 1) / per_block;
  if (n > 0x7FFFFFFFll) return MK_ERR_UNSUPPORTED;
  *blocks = unsigned(n);
  return MK_OK;
}

int move_args(const mk_kv_cache* cache, const void* k, int64_t k_ts, int64_t k_hs, const void* v,
              int64_t v_ts, int64_t v_hs, const int64_t* slots, int tokens, int dtype,
              mk::kv::MoveArgs* a, unsigned* blocks) {
  if (dtype != MK_BF16 && dtype != MK_FP16 && dtype != MK_FP32) return MK_ERR_ARG;
  const int rc = cache_view(cache, &a->c);
  if (rc != MK_OK) return rc;
  const int size = value_size(dtype);
  if (tokens < 0) return MK_ERR_ARG;
  if (tokens == 0) return MK_OK;
  if (!slots || !aligned(slots, 8) || !rows_ok(k, k_ts, k_hs, size) ||
      !rows_ok(v, v_ts, v_hs, size))
    return MK_ERR_ARG;
  a->k_ts = k_ts;
  a->k_hs = k_hs;
  a->v_ts = v_ts;
  a->v_hs = v_hs;
  a->slots = reinterpret_cast<const long long*>(slots);
  a->tokens = tokens;
  const int lanes = cache->head_dim * size / 32;
  return blocks_for((long long)tokens * cache->kv_heads, mk::kv::THREADS / lanes, blocks);
}

}  // namespace

extern "C" {

int mk_rope_init(mk_rope* r, int rot_dim, int interleaved, double theta, int scaling,
                 double factor, double original_ctx, double low, double high) {
  if (!r || rot_dim <= 0 || !(theta > 1.0) || !std::isfinite(theta)) return MK_ERR_ARG;
  if (rot_dim % 16 || rot_dim > 256) return MK_ERR_UNSUPPORTED;
  if (scaling < MK_ROPE_NONE || scaling > MK_ROPE_BANDED) return MK_ERR_ARG;
  if (scaling != MK_ROPE_NONE && !(factor >= 1.0 && std::isfinite(factor))) return MK_ERR_ARG;
  const bool bands = scaling == MK_ROPE_YARN || scaling == MK_ROPE_BANDED;
  if (bands && (!(original_ctx >= 1.0) || !std::isfinite(original_ctx) || !(low > 0.0) ||
                !(high > low) || !std::isfinite(high)))
    return MK_ERR_ARG;
  const double two_pi = 6.283185307179586476925;
  if (scaling == MK_ROPE_NTK) theta *= std::pow(factor, double(rot_dim) / (rot_dim - 2));
  double first = 0.0, last = 0.0;
  if (scaling == MK_ROPE_YARN) {
    // the pairs that turn `high` and `low` times over the original context
    first = std::floor(rot_dim * std::log(original_ctx / (two_pi * high)) / (2 * std::log(theta)));
    last = std::ceil(rot_dim * std::log(original_ctx / (two_pi * low)) / (2 * std::log(theta)));
    if (first < 0) first = 0;
    if (last > rot_dim - 1) last = rot_dim - 1;
  }
  r->rot_dim = rot_dim;
  r->interleaved = interleaved ? 1 : 0;
  r->magnitude = scaling == MK_ROPE_YARN ? float(0.1 * std::log(factor) + 1.0) : 1.0f;
  for (int i = 0; i < 128; ++i) r->turns[i] = 0.0;
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(theta, -2.0 * i / rot_dim);
    if (scaling == MK_ROPE_LINEAR) f /= factor;
    if (bands) {
      double keep;  // share of the unscaled frequency
      if (scaling == MK_ROPE_YARN) {
        keep = 1.0 - (i - first) / (last - first > 1e-3 ? last - first : 1e-3);
      } else {
        keep = (original_ctx * f / two_pi - low) / (high - low);
      }
      keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
      f = f / factor * (1.0 - keep) + f * keep;
    }
    r->turns[i] = f / two_pi;
  }
  return MK_OK;
}

int mk_qk_norm_rope(const mk_rope* rope, const void* q, int64_t q_ts, int64_t q_hs, const void* k,
                    int64_t k_ts, int64_t k_hs, const void* q_gain, const void* k_gain,
                    const int32_t* positions, void* q_out, int64_t qo_ts, int64_t qo_hs,
                    void* k_out, int64_t ko_ts, int64_t ko_hs, int tokens, int q_heads,
                    int kv_heads, int head_dim, float eps, int dtype, void* stream) {
  if (!rope || tokens < 0 || q_heads <= 0 || kv_heads < 0) return MK_ERR_ARG;
  if (dtype != MK_BF16 && dtype != MK_FP16 && dtype != MK_FP32) return MK_ERR_ARG;
  if (!head_dim_ok(head_dim)) return MK_ERR_UNSUPPORTED;
  if (rope->rot_dim <= 0 || rope->rot_dim % 16 || rope->rot_dim > head_dim) return MK_ERR_ARG;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return MK_ERR_ARG;
  if (tokens == 0) return MK_OK;
  const int size = value_size(dtype);
  if (!positions || !aligned(positions, 4) || !rows_ok(q, q_ts, q_hs, size) ||
      !rows_ok(q_out, qo_ts, qo_hs, size))
    return MK_ERR_ARG;
  if (kv_heads > 0 && (!rows_ok(k, k_ts, k_hs, size) || !rows_ok(k_out, ko_ts, ko_hs, size)))
    return MK_ERR_ARG;
  if ((q_gain && !aligned(q_gain, 16)) || (k_gain && !aligned(k_gain, 16))) return MK_ERR_ARG;
  mk::rp::RopeArgs a;
  a.q = static_cast<const unsigned char*>(q);
  a.k = static_cast<const unsigned char*>(k);
  a.q_out = static_cast<unsigned char*>(q_out);
  a.k_out = static_cast<unsigned char*>(k_out);
  a.q_gain = static_cast<const unsigned char*>(q_gain);
  a.k_gain = static_cast<const unsigned char*>(k_gain);
  a.positions = positions;
  a.q_ts = q_ts;
  a.q_hs = q_hs;
  a.k_ts = k_ts;
  a.k_hs = k_hs;
  a.qo_ts = qo_ts;
  a.qo_hs = qo_hs;
  a.ko_ts = ko_ts;
  a.ko_hs = ko_hs;
  a.tokens = tokens;
  a.q_heads = q_heads;
  a.kv_heads = kv_heads;
  a.per_group = q_heads + kv_heads;
  a.rot_dim = rope->rot_dim;
  a.interleaved = rope->interleaved;
  a.eps = eps;
  a.magnitude = rope->magnitude;
  for (int i = 0; i < 128; ++i) a.turns[i] = rope->turns[i];
  const int groups = mk::rp::THREADS / (head_dim * size / 32);
  const int parts = (q_heads + kv_heads + a.per_group - 1) / a.per_group;
  unsigned blocks;
  const int rc = blocks_for((long long)tokens * parts, groups, &blocks);
  if (rc != MK_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  by_row_type(dtype, [&](auto t) {
    by_head_dim(head_dim, [&](auto d) {
      mk::rp::qk_norm_rope_kernel<typename decltype(t)::type, decltype(d)::value>
          <<<blocks, mk::rp::THREADS, 0, st>>>(a);
    });
  });
  return launched();
}

int mk_kv_write(const mk_kv_cache* cache, const void* k, int64_t k_ts, int64_t k_hs, const void* v,
                int64_t v_ts, int64_t v_hs, const int64_t* slots, int tokens, int dtype,
                void* stream) {
  mk::kv::MoveArgs a = {};
  unsigned blocks;
  const int rc = move_args(cache, k, k_ts, k_hs, v, v_ts, v_hs, slots, tokens, dtype, &a, &blocks);
  if (rc != MK_OK || tokens == 0) return rc;
  a.k = static_cast<const unsigned char*>(k);
  a.v = static_cast<const unsigned char*>(v);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  by_row_type(dtype, [&](auto t) {
    by_cache_type(cache->dtype, [&](auto c) {
      by_head_dim(cache->head_dim, [&](auto d) {
        mk::kv::kv_write_kernel<typename decltype(t)::type, typename decltype(c)::type,
                                decltype(d)::value><<<blocks, mk::kv::THREADS, 0, st>>>(a);
      });
    });
  });
  return launched();
}

int mk_kv_read(const mk_kv_cache* cache, const int64_t* slots, int tokens, void* k, int64_t k_ts,
               int64_t k_hs, void* v, int64_t v_ts, int64_t v_hs, int dtype, void* stream) {
  mk::kv::MoveArgs a = {};
  unsigned blocks;
  const int rc = move_args(cache, k, k_ts, k_hs, v, v_ts, v_hs, slots, tokens, dtype, &a, &blocks);
  if (rc != MK_OK || tokens == 0) return rc;
  a.k_out = static_cast<unsigned char*>(k);
  a.v_out = static_cast<unsigned char*>(v);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  by_row_type(dtype, [&](auto t) {
    by_cache_type(cache->dtype, [&](auto c) {
      by_head_dim(cache->head_dim, [&](auto d) {
        mk::kv::kv_read_kernel<typename decltype(t)::type, typename decltype(c)::type,
                               decltype(d)::value><<<blocks, mk::kv::THREADS, 0, st>>>(a);
      });
    });
  });
  return launched();
}

}  // extern "C"

namespace {

// What both attention calls check and fill in.
int attn_args(const void* q, int64_t q_ts, int64_t q_hs, const int32_t* cu_q, void* out,
              int64_t o_ts, int64_t o_hs, float* lse, int rows, int batch, int q_heads,
              int kv_heads, int head_dim, float scale, int dtype, const void* workspace,
              size_t ws_bytes, mk::at::AttnArgs* a) {
  if (rows < 0 || batch < 0 || q_heads <= 0 || kv_heads <= 0 || !half_type(dtype))
    return MK_ERR_ARG;
  if (!head_dim_ok(head_dim)) return MK_ERR_UNSUPPORTED;
  if (q_heads % kv_heads) return MK_ERR_ARG;
  if (q_heads / kv_heads > 128) return MK_ERR_UNSUPPORTED;
  if (!(scale > 0.0f) || !std::isfinite(scale)) return MK_ERR_ARG;
  if (rows == 0 || batch == 0) return MK_OK;
  if (!rows_ok(q, q_ts, q_hs, 2) || !rows_ok(out, o_ts, o_hs, 2) || !cu_q || !aligned(cu_q, 4) ||
      (lse && !aligned(lse, 4)))
    return MK_ERR_ARG;
  if (!workspace || !aligned(workspace, 256) || ws_bytes < mk_attn_ws_bytes(head_dim))
    return MK_ERR_ARG;
  a->q = static_cast<const unsigned char*>(q);
  a->out = static_cast<unsigned char*>(out);
  a->lse = lse;
  a->q_ts = q_ts;
  a->q_hs = q_hs;
  a->o_ts = o_ts;
  a->o_hs = o_hs;
  a->cu_q = cu_q;
  a->rows = rows;
  a->batch = batch;
  a->q_heads = q_heads;
  a->kv_heads = kv_heads;
  a->group = q_heads / kv_heads;
  a->scale_log2 = scale * 1.4426950408889634f;
  return MK_OK;
}

constexpr int kMaxDevices = 64;

// The current device and its number of multiprocessors.
int device_sms(int* dev, int* sms) {
  static int known[kMaxDevices] = {};
  if (cudaGetDevice(dev) != cudaSuccess || *dev < 0 || *dev >= kMaxDevices) {
    cudaGetLastError();
    return MK_ERR_CUDA;
  }
  if (!known[*dev] && cudaDeviceGetAttribute(&known[*dev], cudaDevAttrMultiProcessorCount, *dev) !=
                          cudaSuccess) {
    cudaGetLastError();
    return MK_ERR_CUDA;
  }
  *sms = known[*dev];
  return MK_OK;
}

// The join of partial results, launched so that its CTAs are in place when the
// kernel before it ends.
template <class T, int HD>
int launch_join(const mk::at::AttnArgs& a, const mk::at::Partials& p, int ctas, int rows, int tq,
                cudaStream_t st) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(ctas, (tq * a.group + mk::at::JOIN_ROWS - 1) / mk::at::JOIN_ROWS);
  c.blockDim = dim3(mk::at::JOIN_ROWS * 32);
  c.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &at;
  c.numAttrs = 1;
  if (cudaLaunchKernelEx(&c, mk::at::join_kernel<T, HD>, a, p, rows, tq) != cudaSuccess) {
    return launched();
  }
  return launched();
}

template <class T, class C, int HD, int NT>
int launch_few(const mk::at::AttnArgs& a, void* ws, int dev, int sms, cudaStream_t st) {
  using F = mk::at::FewCfg<C, HD, NT>;
  auto* kernel = &mk::at::attn_few_kernel<T, C, HD, NT>;
  static bool done[kMaxDevices] = {};
  if (!done[dev]) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(F::SMEM)) !=
        cudaSuccess) {
      cudaGetLastError();
      return MK_ERR_CUDA;
    }
    done[dev] = true;
  }
  int ctas = sms;
  while (mk::at::partial_bytes(ctas, F::ROWS, HD) > mk_attn_ws_bytes(HD)) --ctas;
  const mk::at::Partials p = mk::at::carve(ws, ctas, F::ROWS, HD);
  const int tq = F::ROWS / a.group;
  kernel<<<ctas, mk::at::FEW_THREADS, F::SMEM, st>>>(a, p, tq, 1);
  const int rc = launched();
  return rc != MK_OK ? rc : launch_join<T, HD>(a, p, ctas, F::ROWS, tq, st);
}

// cuTensorMapEncodeTiled through the runtime (no link against the driver library).
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encode_tiled() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      p = nullptr;
    }
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// A 4D view of 16-bit values, strides in values for the dims 1 .. 3, boxes of
// 64 values by b1 by b2, in the 128-byte swizzle; outside the view reads as zero.
bool encode_map(CUtensorMap* m, const void* base, bool bf16, long long d0, long long d1,
                long long d2, long long d3, long long s1, long long s2, long long s3, int b1,
                int b2) {
  const EncodeFn fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t dims[4] = {cuuint64_t(d0), cuuint64_t(d1), cuuint64_t(d2), cuuint64_t(d3)};
  // the stride of a dim of one is never walked; zero is not a valid one
  const cuuint64_t strides[3] = {s1 > 0 ? cuuint64_t(s1) * 2 : 16, s2 > 0 ? cuuint64_t(s2) * 2 : 16,
                                 s3 > 0 ? cuuint64_t(s3) * 2 : 16};
  const cuuint32_t box[4] = {64u, cuuint32_t(b1), cuuint32_t(b2), 1u}, step[4] = {1u, 1u, 1u, 1u};
  return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
            const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class T, class C, int HD, bool PAGED>
int launch_flash(const mk::at::AttnArgs& a, void* ws, int dev, int sms, cudaStream_t st) {
  using F = mk::at::FlashCfg<C, HD>;
  auto* kernel = &mk::at::flash_kernel<T, C, HD, PAGED>;
  static bool done[kMaxDevices] = {};
  if (!done[dev]) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(F::SMEM)) !=
        cudaSuccess) {
      cudaGetLastError();
      return MK_ERR_CUDA;
    }
    done[dev] = true;
  }
  constexpr bool BF = __is_same(T, mk::Bf16);
  mk::at::FlashArgs fa;
  fa.a = a;
  fa.tq1 = 128 / a.group;
  fa.least = 1;
  fa.box_shift = 7;
  if (!encode_map(&fa.q, a.q, BF, HD, a.group, a.rows, a.kv_heads, a.q_hs, a.q_ts,
                  a.group * a.q_hs, a.group, fa.tq1))
    return MK_ERR_UNSUPPORTED;
  if (!F::E8) {
    bool ok;
    if (PAGED) {
      if (a.c.page_shift < 7) fa.box_shift = a.c.page_shift;
      const int kb = 1 << fa.box_shift, vb = kb < F::VK ? kb : F::VK;
      ok = encode_map(&fa.k, a.c.k, BF, HD, a.c.page_size, a.c.kv_heads, a.c.n_pages,
                      a.c.pos_stride, a.c.head_stride, a.c.page_stride, kb, 1) &&
           encode_map(&fa.v, a.c.v, BF, HD, a.c.page_size, a.c.kv_heads, a.c.n_pages,
                      a.c.pos_stride, a.c.head_stride, a.c.page_stride, vb, 1);
    } else {
      ok = encode_map(&fa.k, a.k, BF, HD, a.rows, a.kv_heads, 1, a.k_ts, a.k_hs, 0, mk::at::KEYS,
                      1) &&
           encode_map(&fa.v, a.v, BF, HD, a.rows, a.kv_heads, 1, a.v_ts, a.v_hs, 0, F::VK, 1);
    }
    if (!ok) return MK_ERR_UNSUPPORTED;
  } else {
    fa.k = fa.v = fa.q;
  }
  int ctas = sms;
  constexpr int ROWS = F::NQ * 128;
  while (mk::at::partial_bytes(ctas, ROWS, HD) > mk_attn_ws_bytes(HD)) --ctas;
  const mk::at::Partials p = mk::at::carve(ws, ctas, ROWS, HD);
  kernel<<<ctas, F::THREADS, F::SMEM, st>>>(fa, p);
  const int rc = launched();
  return rc != MK_OK ? rc : launch_join<T, HD>(a, p, ctas, ROWS, F::NQ * fa.tq1, st);
}

}  // namespace

extern "C" {

size_t mk_attn_ws_bytes(int head_dim) {
  if (!head_dim_ok(head_dim)) return 0;
  return size_t(40) << 20;
}

int mk_attn_paged(const mk_kv_cache* cache, const void* q, int64_t q_ts, int64_t q_hs,
                  const int32_t* block_table, int table_stride, const int32_t* seq_lens,
                  const int32_t* cu_q, void* out, int64_t o_ts, int64_t o_hs, float* lse, int rows,
                  int batch, int q_heads, float scale, int dtype, void* workspace, size_t ws_bytes,
                  void* stream) {
  mk::at::AttnArgs a = {};
  int rc = cache_view(cache, &a.c);
  if (rc != MK_OK) return rc;
  rc = attn_args(q, q_ts, q_hs, cu_q, out, o_ts, o_hs, lse, rows, batch, q_heads, cache->kv_heads,
                 cache->head_dim, scale, dtype, workspace, ws_bytes, &a);
  if (rc != MK_OK) return rc;
  if (cache->dtype != MK_E4M3 && cache->dtype != dtype) return MK_ERR_ARG;
  if (rows == 0 || batch == 0) return MK_OK;
  if (!block_table || !aligned(block_table, 4) || table_stride <= 0 || !seq_lens ||
      !aligned(seq_lens, 4))
    return MK_ERR_ARG;
  a.table = block_table;
  a.table_stride = table_stride;
  a.seq_lens = seq_lens;
  int dev, sms;
  rc = device_sms(&dev, &sms);
  if (rc != MK_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const long long unit = (long long)a.group * ((rows + batch - 1) / batch);
  by_half_type(dtype, [&](auto t) {
    by_head_dim(cache->head_dim, [&](auto d) {
      using T = typename decltype(t)::type;
      constexpr int HD = decltype(d)::value;
      const bool e8 = cache->dtype == MK_E4M3;
      if (unit <= 8)
        rc = e8 ? launch_few<T, mk::E4m3, HD, 1>(a, workspace, dev, sms, st)
                : launch_few<T, T, HD, 1>(a, workspace, dev, sms, st);
      else if (unit <= 16)
        rc = e8 ? launch_few<T, mk::E4m3, HD, 2>(a, workspace, dev, sms, st)
                : launch_few<T, T, HD, 2>(a, workspace, dev, sms, st);
      else
        rc = e8 ? launch_flash<T, mk::E4m3, HD, true>(a, workspace, dev, sms, st)
                : launch_flash<T, T, HD, true>(a, workspace, dev, sms, st);
    });
  });
  return rc;
}

int mk_attn_packed(const void* q, int64_t q_ts, int64_t q_hs, const void* k, int64_t k_ts,
                   int64_t k_hs, const void* v, int64_t v_ts, int64_t v_hs,
                   const int32_t* cu_seqlens, void* out, int64_t o_ts, int64_t o_hs, float* lse,
                   int rows, int batch, int q_heads, int kv_heads, int head_dim, float scale,
                   int dtype, void* workspace, size_t ws_bytes, void* stream) {
  mk::at::AttnArgs a = {};
  int rc = attn_args(q, q_ts, q_hs, cu_seqlens, out, o_ts, o_hs, lse, rows, batch, q_heads,
                     kv_heads, head_dim, scale, dtype, workspace, ws_bytes, &a);
  if (rc != MK_OK || rows == 0 || batch == 0) return rc;
  if (!rows_ok(k, k_ts, k_hs, 2) || !rows_ok(v, v_ts, v_hs, 2)) return MK_ERR_ARG;
  a.k = static_cast<const unsigned char*>(k);
  a.v = static_cast<const unsigned char*>(v);
  a.k_ts = k_ts;
  a.k_hs = k_hs;
  a.v_ts = v_ts;
  a.v_hs = v_hs;
  int dev, sms;
  rc = device_sms(&dev, &sms);
  if (rc != MK_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  by_half_type(dtype, [&](auto t) {
    by_head_dim(head_dim, [&](auto d) {
      using T = typename decltype(t)::type;
      rc = launch_flash<T, T, decltype(d)::value, false>(a, workspace, dev, sms, st);
    });
  });
  return rc;
}

}  // extern "C"
