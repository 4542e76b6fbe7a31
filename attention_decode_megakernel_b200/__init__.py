"""Python binding of the single-launch decode engine (include/mk.h).

The functions below carry the C ABI's names and only marshal arguments:
every step of the forward pass runs in the CUDA kernels of ``libmk.so``.
PyTorch provides device memory and the current stream.  There is no CPU
fallback: without the built library every call raises.
"""
from __future__ import annotations

import ctypes as C
import os
import re
from typing import Dict, Optional

import numpy as np

from . import synth

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmk.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "mk.h")
MAX_LAYERS = 64

MK_OK, MK_ERR_ARG, MK_ERR_CTX_OVERFLOW, MK_ERR_STATE = 0, 1, 2, 3
MK_ERR_LAUNCH, MK_ERR_TIMEOUT, MK_ERR_CUDA, MK_ERR_UNSUPPORTED = 4, 5, 6, 7
MK_ERR_RANGE = 8


class MkError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__("%s: %s (status %d)" % (what, mk_strerror(code), code))


class mk_config(C.Structure):
    _fields_ = [("n_layers", C.c_int32), ("layer_is_attn", C.c_uint8 * MAX_LAYERS),
                ("hidden", C.c_int32), ("vocab", C.c_int32), ("mlp", C.c_int32),
                ("dn_heads", C.c_int32), ("dn_dk", C.c_int32), ("dn_dv", C.c_int32),
                ("conv_k", C.c_int32), ("q_heads", C.c_int32), ("kv_heads", C.c_int32),
                ("head_dim", C.c_int32), ("rope_theta", C.c_float), ("rms_eps", C.c_float),
                ("max_ctx", C.c_int32), ("max_verify", C.c_int32)]


_LAYER_FIELDS = ("attn_norm", "in_proj", "conv_w", "A_log", "dt_bias", "out_norm",
                 "out_proj", "w_q", "w_k", "w_v", "w_o", "mlp_norm", "w_gate", "w_up",
                 "w_down")


class mk_layer_weights(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in _LAYER_FIELDS]


class mk_weights(C.Structure):
    _fields_ = [("embed", C.c_void_p), ("final_norm", C.c_void_p),
                ("layers", C.POINTER(mk_layer_weights))]


class mk_rope(C.Structure):
    _fields_ = [("rot_dim", C.c_int32), ("interleaved", C.c_int32), ("magnitude", C.c_float),
                ("turns", C.c_uint64 * 128)]


class mk_kv_cache(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("k_scale", C.c_void_p),
                ("v_scale", C.c_void_p), ("page_stride", C.c_int64), ("head_stride", C.c_int64),
                ("pos_stride", C.c_int64), ("n_pages", C.c_int32), ("page_size", C.c_int32),
                ("kv_heads", C.c_int32), ("head_dim", C.c_int32), ("dtype", C.c_int32)]


_lib = None


def lib():
    """Load libmk.so; raise if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("the CUDA engine library %s is not built; run "
                               "attention_decode_megakernel_b200.build.build()" % LIB_PATH)
        L = C.CDLL(LIB_PATH)
        vp, i32, i64, sz = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t
        sig = {
            "mk_workspace_bytes": (sz, [C.POINTER(mk_config)]),
            "mk_create": (C.c_int, [C.POINTER(mk_config), C.POINTER(mk_weights), vp, sz, vp,
                                    C.POINTER(vp)]),
            "mk_destroy": (None, [vp]),
            "mk_reset": (C.c_int, [vp]),
            "mk_prefill": (C.c_int, [vp, vp, C.c_int, vp]),
            "mk_decode_step": (C.c_int, [vp, i32, vp]),
            "mk_generate": (C.c_int, [vp, i32, C.c_int, vp, vp]),
            "mk_verify": (C.c_int, [vp, vp, C.c_int, vp]),
            "mk_accept": (C.c_int, [vp, C.c_int]),
            "mk_position": (C.c_int, [vp]),
            "mk_sync": (C.c_int, [vp]),
            "mk_last_argmax": (i32, [vp]),
            "mk_set_state": (C.c_int, [vp, C.c_int, vp, vp, vp, vp]),
            "mk_get_state": (C.c_int, [vp, vp, vp, vp, vp]),
            "mk_get_hidden": (C.c_int, [vp, vp]),
            "mk_launch_count": (i64, [vp]),
            "mk_debug_set_wait_limit": (C.c_int, [vp, i64, C.c_int]),
            "mk_delta_step": (C.c_int, [vp, vp, vp, vp, vp, vp, vp, C.c_int, C.c_int,
                                        C.c_int, C.c_int, vp]),
            "mk_delta_chunked_ws_bytes": (sz, [C.c_int, C.c_int, C.c_int]),
            "mk_delta_chunked": (C.c_int, [vp, vp, vp, vp, vp, vp, vp, C.c_int, C.c_int,
                                           C.c_int, C.c_int, vp, sz, vp]),
            "mk_debug_gemm": (C.c_int, [vp, vp, vp, C.c_int, C.c_int, C.c_int, vp]),
            "mk_debug_gemm_noalloc": (C.c_int, [vp, vp, vp, C.c_int, C.c_int, C.c_int, vp]),
            "mk_quantize_w4": (C.c_int, [vp, C.c_int, C.c_int, vp, vp, vp]),
            "mk_gemv_w4": (C.c_int, [vp, vp, vp, C.c_int, C.c_int, C.c_int, vp, vp]),
            "mk_rope_init": (C.c_int, [C.POINTER(mk_rope), C.c_int, C.c_int, C.c_double, C.c_int,
                                       C.c_double, C.c_double, C.c_double, C.c_double]),
            "mk_qk_norm_rope": (C.c_int, [vp, vp, i64, i64, vp, i64, i64, vp, vp, vp, vp, i64, i64,
                                          vp, i64, i64, C.c_int, C.c_int, C.c_int, C.c_int,
                                          C.c_float, C.c_int, vp]),
            "mk_kv_write": (C.c_int, [vp, vp, i64, i64, vp, i64, i64, vp, C.c_int, C.c_int, vp]),
            "mk_kv_read": (C.c_int, [vp, vp, C.c_int, vp, i64, i64, vp, i64, i64, C.c_int, vp]),
            "mk_attn_ws_bytes": (sz, [C.c_int]),
            "mk_attn_paged": (C.c_int, [vp, vp, i64, i64, vp, C.c_int, vp, vp, vp, i64, i64, vp,
                                        C.c_int, C.c_int, C.c_int, C.c_float, C.c_int, vp, sz,
                                        vp]),
            "mk_attn_packed": (C.c_int, [vp, i64, i64, vp, i64, i64, vp, i64, i64, vp, vp, i64,
                                         i64, vp, C.c_int, C.c_int, C.c_int, C.c_int, C.c_int,
                                         C.c_float, C.c_int, vp, sz, vp]),
            "mk_strerror": (C.c_char_p, [C.c_int]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def header_symbols():
    """Names of the functions include/mk.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(mk_[a-z_0-9]+)\s*\(", text)))


def mk_strerror(code: int) -> str:
    return lib().mk_strerror(int(code)).decode()


def _check(rc: int, what: str):
    if rc != MK_OK:
        raise MkError(rc, what)


def make_config(cfg: synth.ModelConfig) -> mk_config:
    c = mk_config()
    c.n_layers = cfg.n_layers
    for i, a in enumerate(cfg.layer_is_attn):
        c.layer_is_attn[i] = 1 if a else 0
    c.hidden, c.vocab, c.mlp = cfg.hidden, cfg.vocab, cfg.mlp
    c.dn_heads, c.dn_dk, c.dn_dv, c.conv_k = cfg.dn_heads, cfg.dn_dk, cfg.dn_dv, cfg.conv_k
    c.q_heads, c.kv_heads, c.head_dim = cfg.q_heads, cfg.kv_heads, cfg.head_dim
    c.rope_theta, c.rms_eps = cfg.rope_theta, cfg.rms_eps
    c.max_ctx, c.max_verify = cfg.max_ctx, cfg.max_verify
    return c


def mk_workspace_bytes(cfg: synth.ModelConfig) -> int:
    return int(lib().mk_workspace_bytes(C.byref(make_config(cfg))))


def _ptr(t) -> Optional[int]:
    return None if t is None else int(t.data_ptr())


def upload_weights(cfg: synth.ModelConfig, w: Dict, device="cuda"):
    """Pack the numpy weights into one device blob (128-byte aligned
    tensors) with a single host->device copy.  Returns (blob, offsets)."""
    import torch
    items = [("embed", w["embed"]), ("final_norm", w["final_norm"])]
    for l, d in enumerate(w["layers"]):
        for name in _LAYER_FIELDS:
            if name in d:
                items.append(("%d.%s" % (l, name), d[name]))
    offs, total = {}, 0
    for name, arr in items:
        offs[name] = total
        total += (arr.nbytes + 127) // 128 * 128
    blob = np.zeros(total, np.uint8)
    for name, arr in items:
        blob[offs[name]:offs[name] + arr.nbytes] = np.ascontiguousarray(arr).view(np.uint8).ravel()
    dev = torch.from_numpy(blob).to(device)
    return dev, offs


class Engine:
    """One engine over device-resident weights; every method is a C-ABI call."""

    def __init__(self, cfg: synth.ModelConfig, weights: Dict, device="cuda"):
        import torch
        self.cfg = cfg
        self.torch = torch
        self.blob, offs = upload_weights(cfg, weights, device)
        base = self.blob.data_ptr()
        self._layers = (mk_layer_weights * cfg.n_layers)()
        for l, d in enumerate(weights["layers"]):
            for name in _LAYER_FIELDS:
                key = "%d.%s" % (l, name)
                if key in offs:
                    setattr(self._layers[l], name, base + offs[key])
        self._w = mk_weights(base + offs["embed"], base + offs["final_norm"], self._layers)
        self._cfg = make_config(cfg)
        nbytes = int(lib().mk_workspace_bytes(C.byref(self._cfg)))
        if nbytes == 0:
            raise MkError(MK_ERR_ARG, "mk_workspace_bytes")
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.stream = torch.cuda.current_stream(self.ws.device)
        h = C.c_void_p()
        _check(lib().mk_create(C.byref(self._cfg), C.byref(self._w), self.ws.data_ptr(), nbytes,
                               self.stream.cuda_stream, C.byref(h)), "mk_create")
        self._h = h

    def close(self):
        if getattr(self, "_h", None):
            lib().mk_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- calls ----------------------------------------------------------------
    def reset(self):
        _check(lib().mk_reset(self._h), "mk_reset")

    @property
    def position(self) -> int:
        return lib().mk_position(self._h)

    def sync(self):
        _check(lib().mk_sync(self._h), "mk_sync")

    def prefill(self, tokens, logits=None):
        t = np.ascontiguousarray(tokens, dtype=np.int32)
        _check(lib().mk_prefill(self._h, t.ctypes.data, int(t.size), _ptr(logits)), "mk_prefill")

    def decode_step(self, token: int, logits=None):
        _check(lib().mk_decode_step(self._h, int(token), _ptr(logits)), "mk_decode_step")

    def generate(self, first_token: int, n: int, tokens_out, logits=None):
        _check(lib().mk_generate(self._h, int(first_token), int(n), _ptr(tokens_out),
                                 _ptr(logits)), "mk_generate")

    def verify(self, tokens, logits):
        t = np.ascontiguousarray(tokens, dtype=np.int32)
        _check(lib().mk_verify(self._h, t.ctypes.data, int(t.size), _ptr(logits)), "mk_verify")

    def accept(self, n_keep: int):
        _check(lib().mk_accept(self._h, int(n_keep)), "mk_accept")

    def last_argmax(self) -> int:
        return int(lib().mk_last_argmax(self._h))

    def launch_count(self) -> int:
        return int(lib().mk_launch_count(self._h))

    def set_wait_limit(self, ns: int, fail_phase: int = -1):
        _check(lib().mk_debug_set_wait_limit(self._h, int(ns), int(fail_phase)),
               "mk_debug_set_wait_limit")

    def set_state(self, st: Dict):
        """st: device tensors dn_state f32, conv_state f32, k_cache/v_cache
        (16-bit bf16 patterns), plus 'pos'."""
        _check(lib().mk_set_state(self._h, int(st["pos"]), _ptr(st["dn_state"]),
                                  _ptr(st["conv_state"]), _ptr(st.get("k_cache")),
                                  _ptr(st.get("v_cache"))), "mk_set_state")

    def get_state(self, with_kv=False):
        torch, cfg = self.torch, self.cfg
        dev = self.ws.device
        dn = torch.empty((cfg.n_dn, cfg.dn_heads, cfg.dn_dv, cfg.dn_dk), dtype=torch.float32,
                         device=dev)
        conv = torch.empty((cfg.n_dn, cfg.conv_channels, cfg.conv_k - 1), dtype=torch.float32,
                           device=dev)
        kc = vc = None
        if with_kv:
            shape = (cfg.n_attn, cfg.kv_heads, self.position, cfg.head_dim)
            kc = torch.empty(shape, dtype=torch.int16, device=dev)
            vc = torch.empty(shape, dtype=torch.int16, device=dev)
        _check(lib().mk_get_state(self._h, _ptr(dn), _ptr(conv), _ptr(kc), _ptr(vc)),
               "mk_get_state")
        return dn, conv, kc, vc

    def get_hidden(self):
        torch, cfg = self.torch, self.cfg
        h = torch.empty((cfg.n_layers, cfg.hidden), dtype=torch.float32, device=self.ws.device)
        _check(lib().mk_get_hidden(self._h, _ptr(h)), "mk_get_hidden")
        return h


def mk_delta_step(S, q, k, v, alpha, beta, o, stream=None):
    """Isolated gated delta step (in place on S) through the C ABI."""
    B, heads, dv, dk = S.shape
    st = stream if stream is not None else 0
    _check(lib().mk_delta_step(_ptr(S), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                               _ptr(o), int(B), int(heads), int(dk), int(dv), st),
           "mk_delta_step")


def mk_delta_chunked(S, q, k, v, alpha, beta, o, workspace=None, stream=None):
    """The gated delta rule over T positions in chunkwise form (in place on
    S [heads][dv][dk]); q, k [heads][T][dk], v and o [heads][T][dv], alpha,
    beta [heads][T], all float32 device tensors.  `workspace` (a device
    tensor) may be given; otherwise one is allocated with torch."""
    heads, dv, dk = S.shape
    T = q.shape[1]
    need = lib().mk_delta_chunked_ws_bytes(int(T), int(heads), int(dk))
    if need == 0:
        raise MkError(MK_ERR_ARG, "mk_delta_chunked_ws_bytes")
    if workspace is None:
        import torch
        workspace = torch.empty(need, dtype=torch.uint8, device=S.device)
    st = stream if stream is not None else 0
    _check(lib().mk_delta_chunked(_ptr(S), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                                  _ptr(o), int(T), int(heads), int(dk), int(dv), _ptr(workspace),
                                  int(workspace.numel() * workspace.element_size()), st),
           "mk_delta_chunked")


def mk_debug_gemm(W, X, Cout, stream=None):
    """C = X W^T on the prompt path's tensor-core GEMM (bf16 in, fp32 out)."""
    n_out, K = W.shape
    if X.numel() % (2 * K):
        raise ValueError("X must hold [2][T][K] bf16 (hi then lo operands)")
    T = X.numel() // (2 * K)
    if Cout.numel() != T * n_out:
        raise ValueError("C must hold [T][n_out] float32")
    st = stream if stream is not None else 0
    _check(lib().mk_debug_gemm(_ptr(W), _ptr(X), _ptr(Cout), int(n_out), int(T), int(K), st),
           "mk_debug_gemm")


def mk_debug_gemm_noalloc(W, X, Cout, stream=None):
    """mk_debug_gemm through the allocation-free entry point (static scratch)."""
    n_out, K = W.shape
    if X.numel() % (2 * K):
        raise ValueError("X must hold [2][T][K] bf16 (hi then lo operands)")
    T = X.numel() // (2 * K)
    if Cout.numel() != T * n_out:
        raise ValueError("C must hold [T][n_out] float32")
    st = stream if stream is not None else 0
    _check(lib().mk_debug_gemm_noalloc(_ptr(W), _ptr(X), _ptr(Cout), int(n_out), int(T), int(K),
                                       st), "mk_debug_gemm_noalloc")


def quantize_w4(W, codes, scales, stream=None):
    """4-bit group-wise quantisation of W (bf16 bits [rows][cols] as an int16
    device tensor) into codes (uint8 [rows][cols / 2]) and scales (float32
    [rows][cols / 64]), device tensors the caller provides."""
    rows, cols = W.shape
    if codes.numel() != rows * cols // 2 or scales.numel() != rows * cols // 64:
        raise ValueError("codes must hold [rows][cols/2] bytes, scales [rows][cols/64] floats")
    st = stream if stream is not None else 0
    _check(lib().mk_quantize_w4(_ptr(W), int(rows), int(cols), _ptr(codes), _ptr(scales), st),
           "mk_quantize_w4")


def gemv_w4(codes, scales, x, y, stream=None):
    """y [T][rows] = x [T][cols] times the dequantised 4-bit weights, transposed."""
    T, cols = x.shape
    rows = codes.numel() * 2 // cols
    if y.numel() != T * rows or scales.numel() != rows * cols // 64:
        raise ValueError("y must hold [T][rows] floats and scales [rows][cols/64]")
    st = stream if stream is not None else 0
    _check(lib().mk_gemv_w4(_ptr(codes), _ptr(scales), _ptr(x), int(T), int(rows), int(cols),
                            _ptr(y), st), "mk_gemv_w4")


# ---- an attention layer over a paged cache ------------------------------------
#
# Tensors are device tensors; rows are [token][head][dim] views with any token
# and head distance (a slice of a fused projection, say).  Without `stream` a
# call runs on torch's current stream of the tensors' device.  The calls serve
# only: they record nothing for autograd, whatever requires a gradient.
#
# A decoded token's calls take a few microseconds on the device, less than
# Python needs to look at seven tensors.  So a call first goes, as it is, to
# libmk.so's mkp_ entry (csrc/mk_binding.cu), which looks at the tensors through
# DLPack's C interface and refuses whatever does not fit exactly; what it
# refuses is checked here, where the error says what is wrong.

_ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "banded": 4}
_torch = None
_DTYPES = {}


def _torch_types():
    """Import torch for the calls below; code of each row type."""
    global _torch
    import torch
    _torch = torch
    _DTYPES.update({torch.bfloat16: 0, torch.float16: 1, torch.float32: 2,
                    torch.float8_e4m3fn: 3})
    return _DTYPES


def _code(dtype, what):
    code = (_DTYPES or _torch_types()).get(dtype)
    if code is None:
        raise ValueError("%s: %s is not a supported type" % (what, dtype))
    return code


def _counted(what, *numbers):
    """What the C entries count in 32 bits (ctypes would cut a larger number)."""
    if max(numbers) > 0x7FFFFFFF:
        raise ValueError("%s: more than 2^31 - 1 in a dimension" % what)


def _rows(t, what, shape, dtype, device):
    """(pointer, token distance, head distance) of a [token][head][dim] view."""
    _counted(what, *shape)
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device:
        raise ValueError("%s must be [token][head][dim] = %s of %s on the device of the other "
                         "rows, got %s of %s" % (what, tuple(shape), dtype, tuple(t.shape), t.dtype))
    ts, hs, ds = t.stride()
    if ds != 1:
        raise ValueError("the dims of a head of %s must lie side by side" % what)
    # a distance that is never walked is whatever torch left there
    return t.data_ptr(), ts if shape[0] > 1 else 0, hs if shape[1] > 1 else 0


def _vector(t, what, dtype, shape, device):
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device \
            or not t.is_contiguous():
        raise ValueError("%s must be contiguous, %s of %s on the device of the rows, got %s of %s"
                         % (what, tuple(shape), dtype, tuple(t.shape), t.dtype))
    return t.data_ptr()


def _head_rows(t, what):
    """Shape [token][head][dim], type, its code and device index of the leading tensor."""
    if t.dim() != 3:
        raise ValueError("%s must be [token][head][dim], got %s" % (what, tuple(t.shape)))
    device = t.get_device()
    if device < 0:
        raise ValueError("%s must be on a CUDA device" % what)
    return t.shape, t.dtype, _code(t.dtype, what), device


class _Call:
    """One entry of the C ABI: quick(...) hands the objects over and is True when
    the call was made; slow(...) makes it with plain numbers."""

    def __init__(self, name, quick_args):
        self.name, self.quick_args, self.fn = name, quick_args, None

    def _load(self):
        self.fn = _no_quick_way
        L = _quick_lib()
        if L is not None:
            fn = getattr(L, self.name.replace("mk_", "mkp_"))
            kinds = {"p": C.c_void_p, "i": C.c_int, "o": C.py_object, "d": C.c_double}
            fn.restype, fn.argtypes = C.c_int, [kinds[k] for k in self.quick_args]
            self.fn = fn

    def quick(self, *args):
        if self.fn is None:
            self._load()
        try:
            rc = self.fn(*args)
        except Exception:  # an object that is no tensor, or one that DLPack cannot describe
            return False
        if rc > MK_OK:
            raise MkError(rc, self.name)
        return rc == MK_OK

    def slow(self, device, stream, *args):
        if stream is None:
            stream = _torch.cuda.current_stream(device).cuda_stream
        with _torch.cuda.device(device):
            _check(getattr(lib(), self.name)(*args, stream), self.name)


def _no_quick_way(*args):
    return -1


_quick = None


def _quick_lib():
    """libmk.so called with the interpreter lock held, or None without DLPack's C
    interface (a tensor class of an older torch)."""
    global _quick
    if _quick is None:
        _torch_types()
        _quick = False
        capsule = getattr(_torch.Tensor, "__dlpack_c_exchange_api__", None)
        if capsule is not None:
            get = C.pythonapi.PyCapsule_GetPointer
            get.restype, get.argtypes = C.c_void_p, [C.py_object, C.c_char_p]
            lib()
            L = C.PyDLL(LIB_PATH)
            L.mkp_init.restype = C.c_int
            L.mkp_init.argtypes = [C.c_void_p, C.py_object, C.py_object]
            if L.mkp_init(get(capsule, b"dlpack_exchange_api"), _torch.Tensor, None) == 0:
                _quick = L
    return _quick or None


_norm_rope_call = _Call("mk_qk_norm_rope", "poooooood")
_kv_write_call = _Call("mk_kv_write", "piooo")
_kv_read_call = _Call("mk_kv_read", "piooo")
_paged_call = _Call("mk_attn_paged", "pioooooodo")
_packed_call = _Call("mk_attn_packed", "oooooodo")


class Rope:
    """How positions turn the first `rot_dim` values of a head: pairs
    (i, i + rot_dim / 2), or (2i, 2i + 1) when interleaved; frequencies
    theta^(-2i / rot_dim), scaled for contexts beyond `original_ctx` ("linear",
    "ntk", "yarn", "banded"; see mk_rope_scaling in include/mk.h)."""

    def __init__(self, rot_dim, theta, interleaved=False, scaling="none", factor=1.0,
                 original_ctx=0.0, low=1.0, high=32.0):
        if scaling not in _ROPE_SCALINGS:
            raise ValueError("scaling must be one of %s" % ", ".join(_ROPE_SCALINGS))
        self.c = mk_rope()
        _check(lib().mk_rope_init(C.byref(self.c), int(rot_dim), int(bool(interleaved)),
                                  float(theta), _ROPE_SCALINGS[scaling], float(factor),
                                  float(original_ctx), float(low), float(high)), "mk_rope_init")
        self.address = C.addressof(self.c)


def qk_norm_rope(rope, q, k, positions, q_out=None, k_out=None, q_gain=None, k_gain=None,
                 eps=1e-6, stream=None):
    """RMSNorm (where a gain [head_dim] is given) and rotation of every head of
    q [tokens][q_heads][head_dim] and k [tokens][kv_heads][head_dim] (or None),
    by positions int32 [tokens]; in place where no output is given."""
    if stream is None and _norm_rope_call.quick(rope.address, q, k, positions, q_out, k_out, q_gain,
                                                k_gain, eps):
        return
    shape, dtype, code, dev = _head_rows(q, "q")
    tokens, heads, hd = shape
    qp, qts, qhs = _rows(q, "q", shape, dtype, dev)
    op, ots, ohs = (qp, qts, qhs) if q_out is None else _rows(q_out, "q_out", shape, dtype, dev)
    kp = kts = khs = okp = okts = okhs = kv_heads = 0
    if k is not None:
        kshape = k.shape
        kv_heads = kshape[1]
        if kshape != (tokens, kv_heads, hd):
            raise ValueError("k must be [tokens][kv_heads][head_dim] beside q")
        kp, kts, khs = _rows(k, "k", kshape, dtype, dev)
        okp, okts, okhs = (kp, kts, khs) if k_out is None else _rows(k_out, "k_out", kshape, dtype,
                                                                     dev)
    qg = 0 if q_gain is None else _vector(q_gain, "q_gain", dtype, (hd,), dev)
    kg = 0 if k_gain is None else _vector(k_gain, "k_gain", dtype, (hd,), dev)
    pos = _vector(positions, "positions", _torch.int32, (tokens,), dev)
    _norm_rope_call.slow(dev, stream, rope.address, qp, qts, qhs, kp, kts, khs, qg, kg, pos, op, ots,
                    ohs, okp, okts, okhs, tokens, heads, kv_heads, hd, eps, code)


class KvCache:
    """A paged cache over the caller's tensors k and v, views
    [page][kv_head][position][dim] with the same distances, bfloat16, float16 or
    float8_e4m3fn; the latter with float32 scales [page][kv_head][position]."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype \
                or k.device != v.device or k.stride(3) != 1:
            raise ValueError("k and v must be [page][kv_head][position][dim] views alike, "
                             "dims side by side")
        n, heads, size, hd = k.shape
        code = _code(k.dtype, "cache")
        self.device = k.get_device()
        for s in (k_scale, v_scale):
            if (code == 3) != (s is not None):
                raise ValueError("scales belong to a float8_e4m3fn cache")
            if s is not None:
                _vector(s, "scales", _torch.float32, (n, heads, size), self.device)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.kv_heads, self.head_dim, self.page_size = heads, hd, size
        ps, hs, ts = k.stride()[:3]
        self.c = mk_kv_cache(k.data_ptr(), v.data_ptr(), _ptr(k_scale), _ptr(v_scale),
                             ps if n > 1 else 0, hs if heads > 1 else 0, ts, n, size, heads, hd,
                             code)
        self.address = C.addressof(self.c)


def _move_args(cache, k, v, slots):
    shape, dtype, code, dev = _head_rows(k, "k")
    tokens = shape[0]
    if dev != cache.device or shape != (tokens, cache.kv_heads, cache.head_dim):
        raise ValueError("rows of this cache must be [tokens][%d][%d] on its device"
                         % (cache.kv_heads, cache.head_dim))
    kp, kts, khs = _rows(k, "k", shape, dtype, dev)
    vp, vts, vhs = _rows(v, "v", shape, dtype, dev)
    sp = _vector(slots, "slots", _torch.int64, (tokens,), dev)
    return dev, (kp, kts, khs, vp, vts, vhs), sp, tokens, code


def kv_write(cache, k, v, slots, stream=None):
    """Rows k, v [tokens][kv_heads][head_dim] (bfloat16, float16 or float32) into
    the cache: token t to slot slots[t] = page * page_size + position (int64);
    a slot outside the cache (-1) skips its token."""
    if stream is None and _kv_write_call.quick(cache.address, cache.device, k, v, slots):
        return
    dev, rows, sp, tokens, code = _move_args(cache, k, v, slots)
    _kv_write_call.slow(dev, stream, cache.address, *rows, sp, tokens, code)


def kv_read(cache, slots, k_out, v_out, stream=None):
    """The rows of `slots` as values into k_out, v_out [tokens][kv_heads][head_dim];
    rows of slots outside the cache stay as they were."""
    if stream is None and _kv_read_call.quick(cache.address, cache.device, slots, k_out, v_out):
        return
    dev, rows, sp, tokens, code = _move_args(cache, k_out, v_out, slots)
    _kv_read_call.slow(dev, stream, cache.address, sp, tokens, *rows, code)


def attn_workspace(head_dim, device="cuda"):
    """A workspace for attn_paged and attn_packed; calls that may overlap (other
    streams, graphs replayed at once) need one each."""
    import torch
    n = int(lib().mk_attn_ws_bytes(int(head_dim)))
    if n == 0:
        raise MkError(MK_ERR_UNSUPPORTED, "mk_attn_ws_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _call_workspace(head_dim, dev, stream):
    """A workspace for one call on `stream`.  It belongs to that stream in the allocator's
    books, so that its memory is handed out again behind the call, in the stream's order."""
    device = "cuda:%d" % dev
    if stream is None:
        return attn_workspace(head_dim, device)
    if stream in (0, 1):  # names of the default stream (NULL, cudaStreamLegacy)
        stream = _torch.cuda.default_stream(device)
    else:
        stream = _torch.cuda.ExternalStream(stream, device=device)
    with _torch.cuda.stream(stream):
        return attn_workspace(head_dim, device)


def _attn_outputs(shape, dtype, dev, stream, out, lse, workspace):
    """(pointer, distances of out, pointer of lse, the workspace: held until the call is made)"""
    op, ots, ohs = _rows(out, "out", shape, dtype, dev)
    lp = 0 if lse is None else _vector(lse, "lse", _torch.float32, (shape[0], shape[1]), dev)
    if workspace is None:
        workspace = _call_workspace(shape[2], dev, stream)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("the workspace must be contiguous, on the rows' device")
    return op, ots, ohs, lp, workspace


def attn_paged(q, cache, block_table, seq_lens, cu_q, out, lse=None, scale=None, workspace=None,
               stream=None):
    """Attention of new tokens over a paged cache: rows cu_q[b] .. cu_q[b+1]-1 of
    q [rows][q_heads][head_dim] are the newest of sequence b's seq_lens[b] keys,
    which lie in the pages block_table[b] (int32).  out as q; lse float32
    [rows][q_heads] or None; scale head_dim ** -0.5 by default.  Rows behind
    cu_q[-1] stay as they were.  An expanded q is taken for few rows only (see
    mk_attn_paged in include/mk.h)."""
    if scale is None:
        scale = cache.head_dim ** -0.5
    if stream is None and workspace is not None and _paged_call.quick(
            cache.address, cache.device, q, block_table, seq_lens, cu_q, out, lse, scale, workspace):
        return
    shape, dtype, code, dev = _head_rows(q, "q")
    rows, heads, hd = shape
    if hd != cache.head_dim or dev != cache.device:
        raise ValueError("q must have the cache's head_dim and device")
    qp, qts, qhs = _rows(q, "q", shape, dtype, dev)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [batch][pages]")
    batch, pages = block_table.shape
    _counted("block_table", batch, pages)
    i32 = _torch.int32
    tp = _vector(block_table, "block_table", i32, (batch, pages), dev)
    sp = _vector(seq_lens, "seq_lens", i32, (batch,), dev)
    cp = _vector(cu_q, "cu_q", i32, (batch + 1,), dev)
    op, ots, ohs, lp, ws = _attn_outputs(shape, dtype, dev, stream, out, lse, workspace)
    _paged_call.slow(dev, stream, cache.address, qp, qts, qhs, tp, pages, sp, cp, op, ots, ohs, lp,
                     rows, batch, heads, scale, code, ws.data_ptr(), ws.nbytes)


def attn_packed(q, k, v, cu_seqlens, out, lse=None, scale=None, workspace=None, stream=None):
    """Causal attention of whole prompts packed one after another: rows
    cu_seqlens[b] .. cu_seqlens[b+1]-1 of q [rows][q_heads][head_dim] and of k, v
    [rows][kv_heads][head_dim] are sequence b.  k and v may be expanded over their
    heads; q may not be expanded."""
    if scale is None:
        scale = q.shape[-1] ** -0.5
    if stream is None and workspace is not None and _packed_call.quick(
            q, k, v, cu_seqlens, out, lse, scale, workspace):
        return
    shape, dtype, code, dev = _head_rows(q, "q")
    rows, heads, hd = shape
    kshape = k.shape
    if len(kshape) != 3 or kshape != (rows, kshape[1], hd):
        raise ValueError("k must be [rows][kv_heads][head_dim] beside q")
    qp, qts, qhs = _rows(q, "q", shape, dtype, dev)
    kp, kts, khs = _rows(k, "k", kshape, dtype, dev)
    vp, vts, vhs = _rows(v, "v", kshape, dtype, dev)
    batch = cu_seqlens.shape[0] - 1
    _counted("cu_seqlens", batch)
    cp = _vector(cu_seqlens, "cu_seqlens", _torch.int32, (batch + 1,), dev)
    op, ots, ohs, lp, ws = _attn_outputs(shape, dtype, dev, stream, out, lse, workspace)
    _packed_call.slow(dev, stream, qp, qts, qhs, kp, kts, khs, vp, vts, vhs, cp, op, ots, ohs, lp,
                      rows, batch, heads, kshape[1], hd, scale, code, ws.data_ptr(), ws.nbytes)
