// mk_ops.cuh -- what the host sides of the operators share: status of a
// launch, checks of rows and caches, choice of a kernel by type and head dim.
#pragma once
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "mk.h"
#include "mk_rows.cuh"

namespace {

inline int launched() {
  const cudaError_t r = cudaGetLastError();
  if (r == cudaSuccess) return MK_OK;
  return r == cudaErrorInvalidConfiguration || r == cudaErrorLaunchOutOfResources ? MK_ERR_LAUNCH
                                                                                 : MK_ERR_CUDA;
}

inline bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline bool half_type(int dtype) { return dtype == MK_BF16 || dtype == MK_FP16; }
inline int value_size(int dtype) { return dtype == MK_FP32 ? 4 : dtype == MK_E4M3 ? 1 : 2; }

// Rows whose 16-byte pieces the kernels read and write.
inline bool rows_ok(const void* p, int64_t ts, int64_t hs, int size) {
  return p && aligned(p, 16) && ts >= 0 && hs >= 0 && (ts * size) % 16 == 0 &&
         (hs * size) % 16 == 0 && ts < (int64_t(1) << 38) && hs < (int64_t(1) << 38);
}

// Rows that a call writes: no two tokens or heads may share theirs.
inline bool out_rows_ok(const void* p, int64_t ts, int64_t hs, int tokens, int heads, int head_dim,
                        int size) {
  return rows_ok(p, ts, hs, size) && (tokens == 1 || ts >= head_dim) &&
         (heads == 1 || hs >= head_dim);
}

inline bool head_dim_ok(int hd) { return hd == 64 || hd == 128 || hd == 256; }

// MK_OK and the kernels' view of a cache, or the error of a bad one.
inline int cache_view(const mk_kv_cache* c, mk::PagedView* v) {
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
  if (c->dtype == MK_E4M3 && (!c->k_scale || !c->v_scale || !aligned(c->k_scale, 16) ||
                              !aligned(c->v_scale, 16)))
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

// Launch `kernel` so that its CTAs may start while the kernel before it in the
// stream ends, if that one allows it; it waits (griddep_wait) before it touches memory.
template <class... P, class... A>
int launch(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, void* stream,
           const A&... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &at;
  c.numAttrs = 1;
  cudaLaunchKernelEx(&c, kernel, args...);
  return launched();
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

inline int blocks_for(long long items, int per_block, unsigned* blocks) {
  const long long n = (items + per_block - 1) / per_block;
  if (n > 0x7FFFFFFFll) return MK_ERR_UNSUPPORTED;
  *blocks = unsigned(n);
  return MK_OK;
}

}  // namespace
