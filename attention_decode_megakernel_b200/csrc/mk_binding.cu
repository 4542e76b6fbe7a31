// mk_binding.cu -- the Python binding's quick way into five entries of
// include/mk.h, for calls that take the device a few microseconds.
//
// A tensor's pointer, shape, strides, type and device cost Python a
// microsecond, seven tensors more than a decode step's kernel.  Here they come
// from DLPack's C exchange interface (a table of functions that a tensor
// class publishes; the caller hands over the table and holds the interpreter
// lock), and the tensors arrive as the objects they are.  A call whose
// arguments are not exactly what the entry takes, or whose device is not the
// current one, is answered with MKP_SLOW: the binding then goes through its own
// checks, which name what is wrong or make the call the long way.
#include <cuda_runtime.h>

#include <cstdint>

#include "mk.h"

namespace {

// DLPack's descriptions, as its standard lays them out.
struct DlTensor {
  void* data;
  int32_t device_type, device;
  int32_t ndim;
  uint8_t code, bits;
  uint16_t lanes;
  int64_t* shape;
  int64_t* strides;
  uint64_t byte_offset;
};
struct DlExchange {
  uint32_t major, minor;
  void* previous;
  void *allocate, *from_object, *to_object;
  int (*view)(void* object, DlTensor* out);  // the object's tensor, not owned
  int (*stream)(int device_type, int32_t device, void** out);
};

constexpr int MKP_SLOW = -1;
constexpr int kCuda = 2, kInt = 0, kUint = 1, kFloat = 2, kBfloat = 4;

// The head of every Python object.
struct PyHead {
  intptr_t references;
  void* type;
};

const DlExchange* g_dl = nullptr;
void* g_none = nullptr;
void* g_tensor_type = nullptr;  // the exchange functions take objects of this class alone

struct Slow {};  // thrown and caught in this file

int row_type(const DlTensor& t) {
  if (t.lanes == 1 && t.code == kBfloat && t.bits == 16) return MK_BF16;
  if (t.lanes == 1 && t.code == kFloat && t.bits == 16) return MK_FP16;
  if (t.lanes == 1 && t.code == kFloat && t.bits == 32) return MK_FP32;
  throw Slow{};
}

// The arguments of one call: all tensors on one device, the current one.
struct Args {
  int device = -1;

  DlTensor view(void* object) {
    DlTensor t;
    if (!g_dl || static_cast<PyHead*>(object)->type != g_tensor_type ||
        g_dl->view(object, &t) != 0 || t.device_type != kCuda || !t.strides) throw Slow{};
    if (device < 0) {
      int now;
      if (cudaGetDevice(&now) != cudaSuccess || now != t.device) throw Slow{};
      device = now;
    }
    if (t.device != device) throw Slow{};
    return t;
  }

  struct Rows {
    char* p = nullptr;
    int64_t ts = 0, hs = 0;
    int tokens = 0, heads = 0, dim = 0, type = 0;
  };
  // [token][head][dim], dims side by side; the shape of `like` where given, its type always
  Rows rows(void* object, const Rows* like = nullptr, bool same_shape = true) {
    const DlTensor t = view(object);
    if (t.ndim != 3 || t.strides[2] != 1) throw Slow{};
    for (int i = 0; i < 3; ++i)
      if (t.shape[i] > 0x7FFFFFFF) throw Slow{};
    Rows r;
    r.p = static_cast<char*>(t.data) + t.byte_offset;
    r.tokens = int(t.shape[0]);
    r.heads = int(t.shape[1]);
    r.dim = int(t.shape[2]);
    r.ts = r.tokens > 1 ? t.strides[0] : 0;  // a distance that is never walked may be anything
    r.hs = r.heads > 1 ? t.strides[1] : 0;
    r.type = row_type(t);
    if (like && (r.type != like->type || r.tokens != like->tokens || r.dim != like->dim ||
                 (same_shape && r.heads != like->heads)))
      throw Slow{};
    return r;
  }
  // A contiguous array of n0 (by n1) numbers; null for None where that is allowed.
  void* array(void* object, int code, int bits, int64_t n0, int64_t n1 = -1, bool or_none = false) {
    if (object == g_none) {
      if (or_none) return nullptr;
      throw Slow{};
    }
    const DlTensor t = view(object);
    const int dims = n1 < 0 ? 1 : 2;
    if (t.ndim != dims || t.code != code || t.bits != bits || t.lanes != 1 || t.shape[0] != n0 ||
        (dims == 2 && t.shape[1] != n1))
      throw Slow{};
    const int64_t inner = dims == 2 ? n1 : 1;
    if ((n0 > 1 && t.strides[0] != inner) || (dims == 2 && n1 > 1 && t.strides[1] != 1))
      throw Slow{};
    return static_cast<char*>(t.data) + t.byte_offset;
  }
  void* gain(void* object, const Rows& r) {
    return array(object, r.type == MK_BF16 ? kBfloat : kFloat, r.type == MK_FP32 ? 32 : 16, r.dim,
                 -1, true);
  }
  void* workspace(void* object, size_t* bytes) {
    if (object == g_none) throw Slow{};
    const DlTensor t = view(object);
    if (t.ndim != 1 || t.strides[0] != 1) throw Slow{};
    *bytes = size_t(t.shape[0]) * (t.bits / 8);
    return static_cast<char*>(t.data) + t.byte_offset;
  }
  void* stream() {
    void* s = nullptr;
    if (g_dl->stream(kCuda, device, &s) != 0) throw Slow{};
    return s;
  }
};

template <class F>
int quick(F f) {
  try {
    return f();
  } catch (...) {
    return MKP_SLOW;
  }
}

}  // namespace

extern "C" {

// The exchange table of the tensor class, that class, and the object that stands for
// nothing.
int mkp_init(const void* exchange, void* tensor_type, void* none) {
  const DlExchange* dl = static_cast<const DlExchange*>(exchange);
  if (!dl || dl->major != 1 || !dl->view || !dl->stream) return MKP_SLOW;
  g_tensor_type = tensor_type;
  g_none = none;
  g_dl = dl;
  return 0;
}

int mkp_qk_norm_rope(const mk_rope* rope, void* q, void* k, void* positions, void* q_out,
                     void* k_out, void* q_gain, void* k_gain, double eps) {
  return quick([&] {
    Args a;
    const Args::Rows rq = a.rows(q), oq = q_out == g_none ? rq : a.rows(q_out, &rq);
    Args::Rows rk, ok;
    if (k != g_none) {
      rk = a.rows(k, &rq, false);
      ok = k_out == g_none ? rk : a.rows(k_out, &rk);
    }
    const void* qg = a.gain(q_gain, rq);
    const void* kg = a.gain(k_gain, rq);
    const void* pos = a.array(positions, kInt, 32, rq.tokens);
    return mk_qk_norm_rope(rope, rq.p, rq.ts, rq.hs, rk.p, rk.ts, rk.hs, qg, kg,
                           static_cast<const int32_t*>(pos), oq.p, oq.ts, oq.hs, ok.p, ok.ts,
                           ok.hs, rq.tokens, rq.heads, rk.heads, rq.dim, float(eps), rq.type,
                           a.stream());
  });
}

int mkp_kv_write(const mk_kv_cache* cache, int device, void* k, void* v, void* slots) {
  return quick([&] {
    Args a;
    const Args::Rows rk = a.rows(k), rv = a.rows(v, &rk);
    if (a.device != device || rk.heads != cache->kv_heads || rk.dim != cache->head_dim) throw Slow{};
    const void* s = a.array(slots, kInt, 64, rk.tokens);
    return mk_kv_write(cache, rk.p, rk.ts, rk.hs, rv.p, rv.ts, rv.hs,
                       static_cast<const int64_t*>(s), rk.tokens, rk.type, a.stream());
  });
}

int mkp_kv_read(const mk_kv_cache* cache, int device, void* slots, void* k, void* v) {
  return quick([&] {
    Args a;
    const Args::Rows rk = a.rows(k), rv = a.rows(v, &rk);
    if (a.device != device || rk.heads != cache->kv_heads || rk.dim != cache->head_dim) throw Slow{};
    const void* s = a.array(slots, kInt, 64, rk.tokens);
    return mk_kv_read(cache, static_cast<const int64_t*>(s), rk.tokens, rk.p, rk.ts, rk.hs, rv.p,
                      rv.ts, rv.hs, rk.type, a.stream());
  });
}

int mkp_attn_paged(const mk_kv_cache* cache, int device, void* q, void* block_table, void* seq_lens,
                   void* cu_q, void* out, void* lse, double scale, void* workspace) {
  return quick([&] {
    Args a;
    const Args::Rows rq = a.rows(q), ro = a.rows(out, &rq);
    if (a.device != device || rq.dim != cache->head_dim) throw Slow{};
    const DlTensor t = a.view(block_table);
    if (t.ndim != 2 || t.shape[0] > 0x7FFFFFFE || t.shape[1] > 0x7FFFFFFF) throw Slow{};
    const int batch = int(t.shape[0]), pages = int(t.shape[1]);
    const void* table = a.array(block_table, kInt, 32, batch, pages);
    const void* lens = a.array(seq_lens, kInt, 32, batch);
    const void* cu = a.array(cu_q, kInt, 32, int64_t(batch) + 1);
    void* l = a.array(lse, kFloat, 32, rq.tokens, rq.heads, true);
    size_t bytes;
    void* ws = a.workspace(workspace, &bytes);
    return mk_attn_paged(cache, rq.p, rq.ts, rq.hs, static_cast<const int32_t*>(table), pages,
                         static_cast<const int32_t*>(lens), static_cast<const int32_t*>(cu), ro.p,
                         ro.ts, ro.hs, static_cast<float*>(l), rq.tokens, batch, rq.heads,
                         float(scale), rq.type, ws, bytes, a.stream());
  });
}

int mkp_attn_packed(void* q, void* k, void* v, void* cu_seqlens, void* out, void* lse, double scale,
                    void* workspace) {
  return quick([&] {
    Args a;
    const Args::Rows rq = a.rows(q), ro = a.rows(out, &rq), rk = a.rows(k, &rq, false),
                     rv = a.rows(v, &rk);
    const DlTensor t = a.view(cu_seqlens);
    if (t.ndim != 1 || t.shape[0] < 1 || t.shape[0] > 0x7FFFFFFF) throw Slow{};
    const int batch = int(t.shape[0]) - 1;
    const void* cu = a.array(cu_seqlens, kInt, 32, t.shape[0]);
    void* l = a.array(lse, kFloat, 32, rq.tokens, rq.heads, true);
    size_t bytes;
    void* ws = a.workspace(workspace, &bytes);
    return mk_attn_packed(rq.p, rq.ts, rq.hs, rk.p, rk.ts, rk.hs, rv.p, rv.ts, rv.hs,
                          static_cast<const int32_t*>(cu), ro.p, ro.ts, ro.hs,
                          static_cast<float*>(l), rq.tokens, batch, rq.heads, rk.heads, rq.dim,
                          float(scale), rq.type, ws, bytes, a.stream());
  });
}

}  // extern "C"
