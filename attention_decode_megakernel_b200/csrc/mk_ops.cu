// mk_ops.cu -- host side of the row-wise operators of an attention layer
// (include/mk.h): head norm and rotation, cache write and read.
#include "mk_kvcache.cuh"
#include "mk_ops.cuh"
#include "mk_rope.cuh"

namespace {

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
  if (cache->kv_heads > 65535) return MK_ERR_UNSUPPORTED;  // heads are the grid's second dimension
  return blocks_for(tokens, mk::kv::THREADS / (cache->head_dim * size / 32), blocks);
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
  for (int i = 0; i < 128; ++i) r->turns[i] = 0;
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
    r->turns[i] = uint64_t(std::ldexp(f / two_pi, 64));  // below 2^62: f is at most 1
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
      !out_rows_ok(q_out, qo_ts, qo_hs, tokens, q_heads, head_dim, size))
    return MK_ERR_ARG;
  if (kv_heads > 0 && (!rows_ok(k, k_ts, k_hs, size) ||
                       !out_rows_ok(k_out, ko_ts, ko_hs, tokens, kv_heads, head_dim, size)))
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
  a.rot_dim = rope->rot_dim;
  a.interleaved = rope->interleaved;
  a.eps = eps;
  a.magnitude = rope->magnitude;
  std::memcpy(a.turns, rope->turns, sizeof(a.turns));
  // Blocks are (tokens, parts of the heads).  The angles are computed for each
  // part, so heads are divided only while there are too few blocks to fill the
  // device (two a multiprocessor), and into no fewer rows than a lane has in flight.
  const int groups = mk::rp::THREADS / (head_dim * size / 32), heads = q_heads + kv_heads;
  unsigned blocks;
  const int rc = blocks_for(tokens, groups, &blocks);
  if (rc != MK_OK) return rc;
  int parts = int(blocks) < 296 ? int((296 + blocks - 1) / blocks) : 1;
  if (parts > (heads + mk::rp::UNROLL - 1) / mk::rp::UNROLL)
    parts = (heads + mk::rp::UNROLL - 1) / mk::rp::UNROLL;
  a.per_group = (heads + parts - 1) / parts;
  parts = (heads + a.per_group - 1) / a.per_group;
  if (parts > 65535) return MK_ERR_UNSUPPORTED;
  const dim3 grid(blocks, parts);
  const size_t smem = size_t(groups) * rope->rot_dim * 4;
  // (Launched to start while the kernel before it ends, as the other operators are, 520
  // tokens took 7.7 us one after another in a graph, not 5.1.)
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  by_row_type(dtype, [&](auto t) {
    by_head_dim(head_dim, [&](auto d) {
      mk::rp::qk_norm_rope_kernel<typename decltype(t)::type, decltype(d)::value>
          <<<grid, mk::rp::THREADS, smem, st>>>(a);
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
  int status = MK_OK;
  by_row_type(dtype, [&](auto t) {
    by_cache_type(cache->dtype, [&](auto c) {
      by_head_dim(cache->head_dim, [&](auto d) {
        status = launch(mk::kv::kv_write_kernel<typename decltype(t)::type,
                                             typename decltype(c)::type, decltype(d)::value>,
                        dim3(blocks, cache->kv_heads), mk::kv::THREADS, 0, stream, a);
      });
    });
  });
  return status;
}

int mk_kv_read(const mk_kv_cache* cache, const int64_t* slots, int tokens, void* k, int64_t k_ts,
               int64_t k_hs, void* v, int64_t v_ts, int64_t v_hs, int dtype, void* stream) {
  mk::kv::MoveArgs a = {};
  unsigned blocks;
  const int rc = move_args(cache, k, k_ts, k_hs, v, v_ts, v_hs, slots, tokens, dtype, &a, &blocks);
  if (rc != MK_OK || tokens == 0) return rc;
  const int size = value_size(dtype);
  if (!out_rows_ok(k, k_ts, k_hs, tokens, cache->kv_heads, cache->head_dim, size) ||
      !out_rows_ok(v, v_ts, v_hs, tokens, cache->kv_heads, cache->head_dim, size))
    return MK_ERR_ARG;
  a.k_out = static_cast<unsigned char*>(k);
  a.v_out = static_cast<unsigned char*>(v);
  int status = MK_OK;
  by_row_type(dtype, [&](auto t) {
    by_cache_type(cache->dtype, [&](auto c) {
      by_head_dim(cache->head_dim, [&](auto d) {
        status = launch(mk::kv::kv_read_kernel<typename decltype(t)::type,
                                             typename decltype(c)::type, decltype(d)::value>,
                        dim3(blocks, cache->kv_heads), mk::kv::THREADS, 0, stream, a);
      });
    });
  });
  return status;
}

}  // extern "C"
