// mk_attn_ops.cu -- host side of attention over a paged cache and over packed
// prompts (include/mk.h): checks, tensor maps, choice of a kernel, launches.
#include "mk_flash.cuh"
#include "mk_ops.cuh"
#include "mk_paged.cuh"

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
  // (more than 2^30 sequences: their numbers in rounds of 32 would pass 32 bits)
  if (q_heads / kv_heads > 128 || batch > 1 << 30) return MK_ERR_UNSUPPORTED;
  if (!(scale > 0.0f) || !std::isfinite(scale)) return MK_ERR_ARG;
  if (rows == 0 || batch == 0) return MK_OK;
  if (!rows_ok(q, q_ts, q_hs, 2) || !out_rows_ok(out, o_ts, o_hs, rows, q_heads, head_dim, 2) ||
      !cu_q || !aligned(cu_q, 4) || (lse && !aligned(lse, 4)))
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

// The tensor maps of the many-row kernel walk the tokens and heads of q, and the tokens of
// packed keys and values: a distance of 0 between several is not theirs.
bool walked(int64_t ts, int rows, int64_t hs = 1, int heads = 1) {
  return (ts > 0 || rows == 1) && (hs > 0 || heads == 1);
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

// What a unit costs besides its key tiles, in key tiles (mk_split.cuh), by sweeps in long
// runs, under the power cap: two for tiles of rows (8 prompts of up to 4096 tokens at head_dim
// 128: 428 us at 0, 412 at 1, 407 at 2, 411 at 3, 415 at 4), two for few rows (64 sequences of
// up to 4096 over an e4m3 cache: 40.8 us at 0, 39.5 at 1, 36.9 at 2, 36.6 at 3, 37.2 at 4;
// at head_dim 128 31.8, 31.2, 29.3, 30.1, 31.0).
constexpr int kFewExtra = 2, kFlashExtra = 2;

// Calls whose sequences hold at most so many keys do not divide units over CTAs, and
// have no join. Measured whole / divided (head_dim 256, 8 + 2 heads): one prompt of 520
// tokens 13.8 / 15.4 us, of 780 17.1 / 17.0; 5 tokens over 128 keys 8.7 / 12.0, over 260
// 11.8 / 12.4, over 520 15.5 / 12.3; one token over 64 keys 5.1 / 7.1, over 128 6.1 / 6.9,
// over 260 9.0 / 7.2.  (64 sequences of exactly 520 would gain too, 14.6 / 17.5, but not
// ragged ones, and the call knows no more than the longest.)  The longest is what the table
// (of a packed call, its rows) has room for: the lengths are on the device.
constexpr int kWholePrompt = 640, kWholeChunk = 256, kWholeFew = 128;

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
// A stride of 0 is no map's: only a dim of one, which is never walked, may have it.
bool encode_map(CUtensorMap* m, const void* base, bool bf16, long long d0, long long d1,
                long long d2, long long d3, long long s1, long long s2, long long s3, int b1,
                int b2) {
  const EncodeFn fn = encode_tiled();
  if (!fn || (s1 <= 0 && d1 > 1) || (s2 <= 0 && d2 > 1) || (s3 <= 0 && d3 > 1)) return false;
  const cuuint64_t dims[4] = {cuuint64_t(d0), cuuint64_t(d1), cuuint64_t(d2), cuuint64_t(d3)};
  const cuuint64_t strides[3] = {s1 > 0 ? cuuint64_t(s1) * 2 : 16, s2 > 0 ? cuuint64_t(s2) * 2 : 16,
                                 s3 > 0 ? cuuint64_t(s3) * 2 : 16};
  const cuuint32_t box[4] = {64u, cuuint32_t(b1), cuuint32_t(b2), 1u}, step[4] = {1u, 1u, 1u, 1u};
  return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
            const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A paged cache's rows as boxes of (128 bytes, 16 positions, all columns of 128 bytes):
// 64-byte rows as one column of 64.
bool encode_rows(CUtensorMap* m, const void* base, const mk::PagedView& c, int row) {
  const EncodeFn fn = encode_tiled();
  if (!fn) return false;
  const bool e8 = row == c.head_dim;
  const int size = e8 ? 1 : 2, col = row < 128 ? row : 128;  // bytes
  const cuuint64_t dims[5] = {cuuint64_t(col / size), cuuint64_t(c.page_size),
                              cuuint64_t(row / col), cuuint64_t(c.kv_heads),
                              cuuint64_t(c.n_pages)};
  auto stride = [&](long long s) { return s > 0 ? cuuint64_t(s) * size : cuuint64_t(16); };
  const cuuint64_t strides[4] = {stride(c.pos_stride), cuuint64_t(col), stride(c.head_stride),
                                 stride(c.page_stride)};
  const cuuint32_t box[5] = {cuuint32_t(col / size), 16u, cuuint32_t(row / col), 1u, 1u};
  const cuuint32_t step[5] = {1u, 1u, 1u, 1u, 1u};
  return fn(m, e8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5,
            const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            col == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class T, class C, int HD, int NT>
int launch_few(const mk::at::AttnArgs& a, long long longest, void* ws, int dev, int sms, cudaStream_t st) {
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
  mk::at::FewArgs fa;
  fa.a = a;
  fa.tq = tq;
  fa.extra = kFewExtra;
  fa.least = 1;
  fa.whole = longest <= kWholeFew;
  if (!encode_rows(&fa.k, a.c.k, a.c, F::ROW) || !encode_rows(&fa.v, a.c.v, a.c, F::ROW))
    return MK_ERR_UNSUPPORTED;
  const int rc = launch(kernel, dim3(ctas), F::THREADS, F::SMEM, st, fa, p);
  if (rc != MK_OK || fa.whole) return rc;
  return launch(mk::at::join_kernel<T, HD>, dim3(ctas, tq * a.group),
                mk::at::JOIN_SPLIT * 32, 0, st, a, p, int(F::ROWS));
}

template <class T, class C, int HD, bool PAGED>
int launch_flash(const mk::at::AttnArgs& a, long long longest, void* ws, int dev, int sms, cudaStream_t st) {
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
  fa.extra = kFlashExtra;
  fa.least = 1;
  fa.whole = longest <= (PAGED ? kWholeChunk : kWholePrompt);
  fa.box_shift = 7;
  fa.k_head = fa.v_head = ~0;
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
      // heads that share their rows (a distance of 0) are one head to the map
      fa.k_head = a.k_hs ? ~0 : 0;
      fa.v_head = a.v_hs ? ~0 : 0;
      ok = encode_map(&fa.k, a.k, BF, HD, a.rows, a.k_hs ? a.kv_heads : 1, 1, a.k_ts, a.k_hs, 0,
                      mk::at::KEYS, 1) &&
           encode_map(&fa.v, a.v, BF, HD, a.rows, a.v_hs ? a.kv_heads : 1, 1, a.v_ts, a.v_hs, 0,
                      F::VK, 1);
    }
    if (!ok) return MK_ERR_UNSUPPORTED;
  } else {
    fa.k = fa.v = fa.q;
  }
  int ctas = sms;
  constexpr int ROWS = F::NQ * 128;
  while (mk::at::partial_bytes(ctas, ROWS, HD) > mk_attn_ws_bytes(HD)) --ctas;
  const mk::at::Partials p = mk::at::carve(ws, ctas, ROWS, HD);
  const int rc = launch(kernel, dim3(ctas), F::THREADS, F::SMEM, st, fa, p);
  const int tq = F::NQ * fa.tq1;
  const dim3 join(ctas, (tq * a.group + 31) / 32 * (HD / 64));
  if (rc != MK_OK || fa.whole) return rc;
  return launch(mk::at::join_tiles_kernel<T, HD>, join, 128, 0, st, a, p, int(ROWS));
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
  const long long unit = a.group * (((long long)rows + batch - 1) / batch);
  if (unit > 16 && !walked(q_ts, rows, q_hs, q_heads)) return MK_ERR_UNSUPPORTED;
  a.table = block_table;
  a.table_stride = table_stride;
  a.seq_lens = seq_lens;
  int dev, sms;
  rc = device_sms(&dev, &sms);
  if (rc != MK_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // By the rows of a unit on average: up to 8 or 16 the few-row kernel. It serves the whole
  // batch, so that one chunk of 512 among 256 single tokens walks its keys four tokens at a
  // time (contexts of up to 8192, 8 + 2 heads of 256: 774 us, 427 + 40 as two calls; 16 + 4
  // heads of 128: 524, 420 + 48).
  const long long longest = (long long)table_stride * cache->page_size;
  by_half_type(dtype, [&](auto t) {
    by_head_dim(cache->head_dim, [&](auto d) {
      using T = typename decltype(t)::type;
      constexpr int HD = decltype(d)::value;
      const bool e8 = cache->dtype == MK_E4M3;
      if (unit <= 8)
        rc = e8 ? launch_few<T, mk::E4m3, HD, 1>(a, longest, workspace, dev, sms, st)
                : launch_few<T, T, HD, 1>(a, longest, workspace, dev, sms, st);
      else if (unit <= 16)
        rc = e8 ? launch_few<T, mk::E4m3, HD, 2>(a, longest, workspace, dev, sms, st)
                : launch_few<T, T, HD, 2>(a, longest, workspace, dev, sms, st);
      else
        rc = e8 ? launch_flash<T, mk::E4m3, HD, true>(a, longest, workspace, dev, sms, st)
                : launch_flash<T, T, HD, true>(a, longest, workspace, dev, sms, st);
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
  if (!walked(q_ts, rows, q_hs, q_heads) || !walked(k_ts, rows) || !walked(v_ts, rows))
    return MK_ERR_UNSUPPORTED;
  a.k = static_cast<const unsigned char*>(k);
  a.v = static_cast<const unsigned char*>(v);
  a.k_ts = k_ts;
  a.k_hs = k_hs;
  a.v_ts = v_ts;
  a.v_hs = v_hs;
  int dev, sms;
  rc = device_sms(&dev, &sms);
  if (rc != MK_OK) return rc;
  const long long longest = rows;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  by_half_type(dtype, [&](auto t) {
    by_head_dim(head_dim, [&](auto d) {
      using T = typename decltype(t)::type;
      rc = launch_flash<T, T, decltype(d)::value, false>(a, longest, workspace, dev, sms, st);
    });
  });
  return rc;
}

}  // extern "C"
