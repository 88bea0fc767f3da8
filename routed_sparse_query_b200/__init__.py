"""Python binding of libgqe.so, the B200 (sm_100a) GQE prefill layer.

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels. Tensors are torch CUDA tensors (torch supplies device memory and
streams); each function has the name and argument order of the C entry point
it calls (see include/gqe.h) and raises ``GQEError`` on a non-OK status.

There is no CPU fallback: importing this module fails loudly when libgqe.so
is missing or cannot be loaded.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgqe.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libgqe.so not built ({LIB_PATH}); run python -m routed_sparse_query_b200.build")
_lib = ctypes.CDLL(LIB_PATH)

GQE_OK, GQE_ERR_INVALID, GQE_ERR_UNSUPPORTED, GQE_ERR_WORKSPACE = 0, 1, 2, 3
GQE_ERR_CUDA, GQE_ERR_TIMEOUT, GQE_ERR_DEVICE_CHECK = 4, 5, 6
GQE_WS_DISPATCH, GQE_WS_LAYER, GQE_WS_DENSE, GQE_WS_ATTENTION = 1, 2, 3, 4
GQE_WS_DECODE, GQE_WS_DENSE_DECODE, GQE_WS_BACKWARD = 5, 6, 7
GQE_WS_QK_ROPE, GQE_WS_BALANCE, GQE_WS_KV4, GQE_WS_DECODE_KV4, GQE_WS_BACKWARD_AUX = 8, 9, 10, 11, 12
GQE_ROPE_NORM, GQE_ROPE_ADJACENT = 1, 2
GQE_FLAG_WS_CLEAN, GQE_FLAG_EXPERT_MAJOR = 1, 2
# Output constructions (at most one): see include/gqe.h.
GQE_FLAG_SLOT_GROUP_MEAN, GQE_FLAG_OUT_HARD, GQE_FLAG_OUT_WEIGHTED_CONCAT = 4, 8, 16
GQE_FLAG_NO_SHARED_HEAD = 32  # a shard of the layer split over KV groups (no shared head)
OUTPUT_MODE_FLAGS = {"gqe": 0, "group_mean": GQE_FLAG_SLOT_GROUP_MEAN, "hard": GQE_FLAG_OUT_HARD,
                     "weighted_concat": GQE_FLAG_OUT_WEIGHTED_CONCAT}
ITEMS = {"idx": 1, "r": 2, "omega": 3, "counts": 4, "offsets": 5, "tok": 6, "slot_pos": 7,
         "Qv": 8, "Qs": 9, "K": 10, "V": 11, "slots": 12, "dispatch_ws": 13, "attention_ws": 14,
         "dense_Q": 32, "dense_O": 33}

EXPORTED = ("gqe_workspace_bytes", "gqe_workspace_offset", "gqe_router_topk", "gqe_dispatch",
            "gqe_kv_proj", "gqe_attention_fwd", "gqe_output_proj", "gqe_layer_fwd",
            "gqa_dense_fwd", "gqe_read_status", "gqe_selftest_wait_timeout",
            "gqe_status_string", "gqe_version", "gqe_dispatch_noalloc", "gqe_attention_fwd_compact",
            "gqe_decode_step", "gqa_dense_decode_step", "gqe_layer_bwd", "gqe_qk_rope", "gqe_qk_rope_bwd",
            "gqe_router_logits", "gqe_balance_stats", "gqe_balance_loss", "gqe_kv4_append", "gqe_kv4_read",
            "gqe_kv4_attention", "gqe_layer_fwd_rope", "gqe_layer_bwd_aux", "gqe_decode_step_rope",
            "gqe_decode_step_kv4")


class GQEConfig(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("d_model", ctypes.c_int32),
                ("G", ctypes.c_int32), ("M", ctypes.c_int32), ("k", ctypes.c_int32),
                ("d_head", ctypes.c_int32), ("flags", ctypes.c_uint32)]

    @classmethod
    def of(cls, shape, flags: int = 0) -> "GQEConfig":
        return cls(shape.B, shape.T, shape.d_model, shape.G, shape.M, shape.k, shape.d_head, flags)


# torch's own cheap accessors where it has them (a Stream object costs 3 us to make).
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _first_device(*tensors) -> int:
    """The CUDA device of the first tensor given (of none: the current one)."""
    for t in tensors:
        if t is not None:
            dev = t.get_device()
            if dev < 0:
                raise ValueError("tensors must be contiguous CUDA tensors")
            return dev
    return _current_device()


def _arg(t, dtype, n, dev, name):
    """Pointer of an optional argument: contiguous, on CUDA device `dev`, of the
    given type and (n not None) element count."""
    if t is None:
        return None
    if t.get_device() != dev or t.dtype is not dtype or (n is not None and t.numel() != n) or not t.is_contiguous():
        _refuse(t, dtype, n, dev, name)
    return t.data_ptr()


def _refuse(t, dtype, n, dev, name):
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: tensors must be contiguous CUDA tensors")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on cuda:{t.get_device()}, the call's other tensors on cuda:{dev}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: {t.dtype}, {dtype} is needed")
    raise ValueError(f"{name}: {t.numel()} elements, {n} are needed")


class GQERope(ctypes.Structure):
    """gqe_rope: the norm and rotation of queries and keys (see include/gqe.h).
    Made by ``of`` from CUDA tensors, which it keeps alive."""
    _fields_ = [("d_rot", ctypes.c_int32), ("axes", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("eps", ctypes.c_float), ("scale", ctypes.c_float), ("pos", ctypes.c_void_p),
                ("inv_freq", ctypes.c_void_p), ("axis", ctypes.c_void_p), ("w_q", ctypes.c_void_p),
                ("w_k", ctypes.c_void_p)]

    @classmethod
    def of(cls, d_rot: int, inv_freq, pos=None, axis=None, w_q=None, w_k=None, eps: float = 0.0, scale: float = 1.0,
           flags: int = 0, axes: int | None = None) -> "GQERope":
        """inv_freq [d_rot/2] fp64; pos int32 [axes, tokens] (or [tokens]); axis int32 [d_rot/2]; w_q, w_k fp32
        [d_head]. `axes` is taken from pos where it has two dimensions."""
        if axes is None:
            axes = pos.shape[0] if pos is not None and pos.dim() == 2 else 1
        half = d_rot // 2
        tensors = [(pos, torch.int32, None, "pos"), (inv_freq, torch.float64, half, "inv_freq"),
                   (axis, torch.int32, half, "axis"), (w_q, torch.float32, None, "w_q"), (w_k, torch.float32, None, "w_k")]
        given = [t for t, _, _, _ in tensors if t is not None]
        dev = _first_device(*given) if given else -1
        self = cls(d_rot, axes, flags, eps, scale, *(_arg(t, d, n, dev, what) for t, d, n, what in tensors))
        self._refs, self._dev = given, dev
        self._n_pos = None if pos is None else pos.numel()
        self._n_w = {t.numel() for t in (w_q, w_k) if t is not None}
        return self


class GQEKv4(ctypes.Structure):
    """gqe_kv4: a 4-bit K/V cache (see include/gqe.h). Made by ``of`` from its
    CUDA tensors, which it keeps alive: k_codes, v_codes uint8 [B, G, capacity,
    d_head/2], meta bf16 [B, G, capacity, 4]."""
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p), ("meta", ctypes.c_void_p),
                ("capacity", ctypes.c_int32)]

    @classmethod
    def of(cls, k_codes, v_codes, meta) -> "GQEKv4":
        if k_codes.dim() != 4:
            raise ValueError("k_codes is [B, G, capacity, d_head/2]")
        B, G, cap, half = k_codes.shape
        dev = _first_device(k_codes)
        self = cls(_arg(k_codes, torch.uint8, None, dev, "k_codes"),
                   _arg(v_codes, torch.uint8, k_codes.numel(), dev, "v_codes"),
                   _arg(meta, torch.bfloat16, B * G * cap * 4, dev, "meta"), cap)
        self._refs, self._dev, self._shape = (k_codes, v_codes, meta), dev, (B, G, 2 * half)
        return self


class GQEBalance(ctypes.Structure):
    """gqe_balance: the balance loss of gqe_layer_bwd_aux (see include/gqe.h).
    Made by ``of`` from CUDA tensors, which it keeps alive."""
    _fields_ = [("mask", ctypes.c_void_p), ("c_balance", ctypes.c_float), ("c_z", ctypes.c_float),
                ("counts", ctypes.c_void_p), ("sums", ctypes.c_void_p), ("loss", ctypes.c_void_p)]

    @classmethod
    def of(cls, counts, sums, loss=None, mask=None, c_balance: float = 0.0, c_z: float = 0.0) -> "GQEBalance":
        dev = _first_device(counts)
        self = cls(_arg(mask, torch.uint8, None, dev, "mask"), c_balance, c_z,
                   _arg(counts, torch.int32, None, dev, "counts"), _arg(sums, torch.float32, counts.numel(), dev, "sums"),
                   _arg(loss, torch.float32, 3, dev, "loss"))
        self._refs, self._dev, self._n = (counts, sums, loss, mask), dev, counts.numel()
        self._n_mask = None if mask is None else mask.numel()
        return self


class GQEError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = _lib.gqe_status_string(status).decode()
        super().__init__(f"{where}: {msg} (status {status})")
        self.status = status


_P = ctypes.c_void_p
_CFG = ctypes.POINTER(GQEConfig)
_ROPE, _KV4, _BAL = ctypes.POINTER(GQERope), ctypes.POINTER(GQEKv4), ctypes.POINTER(GQEBalance)
_sig = {
    "gqe_workspace_bytes": (ctypes.c_size_t, [_CFG, ctypes.c_int]),
    "gqe_workspace_offset": (ctypes.c_size_t, [_CFG, ctypes.c_int, ctypes.c_int]),
    "gqe_router_topk": (ctypes.c_int, [_CFG, _P, _P, _P, _P, _P, _P, _P]),
    "gqe_dispatch": (ctypes.c_int, [_CFG, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                    ctypes.c_size_t, _P]),
    "gqe_dispatch_noalloc": (ctypes.c_int, [_CFG, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "gqe_kv_proj": (ctypes.c_int, [_CFG, _P, _P, _P, _P, _P, _P]),
    "gqe_attention_fwd": (ctypes.c_int, [_CFG, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "gqe_attention_fwd_compact": (ctypes.c_int, [_CFG, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "gqe_output_proj": (ctypes.c_int, [_CFG, _P, _P, _P, _P, _P]),
    "gqe_layer_fwd": (ctypes.c_int, [_CFG, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                     ctypes.c_size_t, _P]),
    "gqa_dense_fwd": (ctypes.c_int, [_CFG, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "gqe_decode_step": (ctypes.c_int, [_CFG, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_int32,
                                       _P, _P, ctypes.c_size_t, _P]),
    "gqa_dense_decode_step": (ctypes.c_int, [_CFG, _P, _P, _P, _P, _P, _P, _P, ctypes.c_int32, _P,
                                             _P, ctypes.c_size_t, _P]),
    "gqe_layer_bwd": (ctypes.c_int, [_CFG] + [_P] * 18 + [ctypes.c_size_t, _P]),
    "gqe_qk_rope": (ctypes.c_int, [_CFG, _ROPE] + [_P] * 8),
    "gqe_qk_rope_bwd": (ctypes.c_int, [_CFG, _ROPE] + [_P] * 13 + [ctypes.c_size_t, _P]),
    "gqe_router_logits": (ctypes.c_int, [_CFG] + [_P] * 5),
    "gqe_balance_stats": (ctypes.c_int, [_CFG] + [_P] * 6 + [ctypes.c_size_t, _P]),
    "gqe_balance_loss": (ctypes.c_int, [_CFG] + [_P] * 4 + [ctypes.c_float, ctypes.c_float, _P, _P, ctypes.c_int, _P]),
    "gqe_kv4_append": (ctypes.c_int, [_CFG] + [_P] * 4 + [_KV4, _P]),
    "gqe_kv4_read": (ctypes.c_int, [_CFG, _KV4] + [_P] * 5),
    "gqe_kv4_attention": (ctypes.c_int, [_CFG, _P, _P, _KV4, _P, _P, ctypes.c_int32, _P, ctypes.c_size_t, _P]),
    "gqe_layer_fwd_rope": (ctypes.c_int, [_CFG, _ROPE] + [_P] * 10 + [ctypes.c_size_t, _P]),
    "gqe_layer_bwd_aux": (ctypes.c_int, [_CFG, _ROPE, _BAL] + [_P] * 20 + [ctypes.c_size_t, _P]),
    "gqe_decode_step_rope": (ctypes.c_int, [_CFG, _ROPE] + [_P] * 10 + [ctypes.c_int32, _P, _P, ctypes.c_size_t, _P]),
    "gqe_decode_step_kv4": (ctypes.c_int, [_CFG, _ROPE] + [_P] * 8 + [_KV4, _P, _P, _P, ctypes.c_size_t, _P]),
    "gqe_read_status": (ctypes.c_int, [ctypes.POINTER(ctypes.c_int32)]),
    "gqe_selftest_wait_timeout": (ctypes.c_int, [ctypes.c_uint64, _P]),
    "gqe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "gqe_version": (ctypes.c_int, []),
}
for _name, (_res, _args) in _sig.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


def lib():
    return _lib


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("tensors must be contiguous CUDA tensors")
    return t.data_ptr()


def _stream(stream):
    return _raw_stream(_current_device()) if stream is None else stream.cuda_stream


def _check(status: int, where: str):
    if status != GQE_OK:
        raise GQEError(status, where)


def _cfg(cfg):
    return ctypes.byref(cfg if isinstance(cfg, GQEConfig) else GQEConfig.of(cfg))


def gqe_workspace_bytes(cfg, which: int) -> int:
    return int(_lib.gqe_workspace_bytes(_cfg(cfg), which))


def gqe_workspace_offset(cfg, which: int, item) -> int:
    item = ITEMS[item] if isinstance(item, str) else item
    return int(_lib.gqe_workspace_offset(_cfg(cfg), which, item))


def gqe_router_topk(cfg, x, W_r, b_r, idx, r, omega, stream=None):
    _check(_lib.gqe_router_topk(_cfg(cfg), _ptr(x), _ptr(W_r), _ptr(b_r), _ptr(idx), _ptr(r),
                                _ptr(omega), _stream(stream)), "gqe_router_topk")


def gqe_dispatch(cfg, idx, x, W_q, W_qs, counts, offsets, tok, slot_pos, Qv, Qs, ws, stream=None):
    _check(_lib.gqe_dispatch(_cfg(cfg), _ptr(idx), _ptr(x), _ptr(W_q), _ptr(W_qs), _ptr(counts),
                             _ptr(offsets), _ptr(tok), _ptr(slot_pos), _ptr(Qv), _ptr(Qs),
                             _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "gqe_dispatch")


def gqe_dispatch_noalloc(cfg, idx, x, W_q, W_qs, counts, offsets, tok, slot_pos, Qv, Qs,
                         stream=None):
    """gqe_dispatch for callers that cannot allocate a workspace: the scratch is
    a fixed device array of the library (see include/gqe.h)."""
    _check(_lib.gqe_dispatch_noalloc(_cfg(cfg), _ptr(idx), _ptr(x), _ptr(W_q), _ptr(W_qs),
                                     _ptr(counts), _ptr(offsets), _ptr(tok), _ptr(slot_pos),
                                     _ptr(Qv), _ptr(Qs), _stream(stream)), "gqe_dispatch_noalloc")


def gqe_kv_proj(cfg, x, W_k, W_v, K, V, stream=None):
    _check(_lib.gqe_kv_proj(_cfg(cfg), _ptr(x), _ptr(W_k), _ptr(W_v), _ptr(K), _ptr(V),
                            _stream(stream)), "gqe_kv_proj")


def gqe_attention_fwd(cfg, Qv, Qs, K, V, slots, ws, stream=None):
    _check(_lib.gqe_attention_fwd(_cfg(cfg), _ptr(Qv), _ptr(Qs), _ptr(K), _ptr(V), _ptr(slots),
                                  _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "gqe_attention_fwd")


def gqe_attention_fwd_compact(cfg, Qe, Qs, K, V, idx, offsets, tok, slots, stream=None):
    _check(_lib.gqe_attention_fwd_compact(_cfg(cfg), _ptr(Qe), _ptr(Qs), _ptr(K), _ptr(V), _ptr(idx),
                                          _ptr(offsets), _ptr(tok), _ptr(slots), _stream(stream)),
           "gqe_attention_fwd_compact")


def gqe_output_proj(cfg, slots, omega, W_o, y, stream=None):
    _check(_lib.gqe_output_proj(_cfg(cfg), _ptr(slots), _ptr(omega), _ptr(W_o), _ptr(y),
                                _stream(stream)), "gqe_output_proj")


def gqe_layer_fwd(cfg, x, W_r, b_r, W_q, W_qs, W_k, W_v, W_o, y, ws, stream=None):
    _check(_lib.gqe_layer_fwd(_cfg(cfg), _ptr(x), _ptr(W_r), _ptr(b_r), _ptr(W_q), _ptr(W_qs),
                              _ptr(W_k), _ptr(W_v), _ptr(W_o), _ptr(y), _ptr(ws),
                              ws.numel() * ws.element_size(), _stream(stream)), "gqe_layer_fwd")


def gqe_layer_bwd(cfg, x, W_r, b_r, W_q, W_qs, W_k, W_v, W_o, dy, dx, dW_r, db_r, dW_q, dW_qs, dW_k, dW_v,
                  dW_o, ws, stream=None):
    _check(_lib.gqe_layer_bwd(_cfg(cfg), _ptr(x), _ptr(W_r), _ptr(b_r), _ptr(W_q), _ptr(W_qs), _ptr(W_k),
                              _ptr(W_v), _ptr(W_o), _ptr(dy), _ptr(dx), _ptr(dW_r), _ptr(db_r), _ptr(dW_q),
                              _ptr(dW_qs), _ptr(dW_k), _ptr(dW_v), _ptr(dW_o), _ptr(ws),
                              ws.numel() * ws.element_size(), _stream(stream)), "gqe_layer_bwd")


def gqa_dense_fwd(cfg, x, W_q, W_k, W_v, W_o_dense, y, ws, stream=None):
    _check(_lib.gqa_dense_fwd(_cfg(cfg), _ptr(x), _ptr(W_q), _ptr(W_k), _ptr(W_v),
                              _ptr(W_o_dense), _ptr(y), _ptr(ws), ws.numel() * ws.element_size(),
                              _stream(stream)), "gqa_dense_fwd")


def gqe_decode_step(cfg, x, W_r, b_r, W_q, W_qs, W_k, W_v, W_o, K_cache, V_cache, y, ws,
                    stream=None):
    """cfg.T = keys after the step (the new token at T - 1); the cache capacity
    is K_cache.shape[2]."""
    _check(_lib.gqe_decode_step(_cfg(cfg), _ptr(x), _ptr(W_r), _ptr(b_r), _ptr(W_q), _ptr(W_qs),
                                _ptr(W_k), _ptr(W_v), _ptr(W_o), _ptr(K_cache), _ptr(V_cache),
                                int(K_cache.shape[2]), _ptr(y), _ptr(ws),
                                ws.numel() * ws.element_size(), _stream(stream)), "gqe_decode_step")


def gqa_dense_decode_step(cfg, x, W_q, W_k, W_v, W_o_dense, K_cache, V_cache, y, ws, stream=None):
    _check(_lib.gqa_dense_decode_step(_cfg(cfg), _ptr(x), _ptr(W_q), _ptr(W_k), _ptr(W_v),
                                      _ptr(W_o_dense), _ptr(K_cache), _ptr(V_cache),
                                      int(K_cache.shape[2]), _ptr(y), _ptr(ws),
                                      ws.numel() * ws.element_size(), _stream(stream)),
           "gqa_dense_decode_step")


_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
_byref = ctypes.byref


def _call(fn, dev, stream, *args):
    """The C entry point `fn` on device `dev` and on `stream` (default: that
    device's current stream)."""
    if dev == _current_device():
        status = fn(*args, _raw_stream(dev) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _stream(stream))
    if status:
        raise GQEError(status, fn.__name__)


def _config(cfg) -> GQEConfig:
    return cfg if type(cfg) is GQEConfig else GQEConfig.of(cfg)


def _ws(ws, dev):
    return _arg(ws, ws.dtype, None, dev, "ws"), ws.nbytes


def _rope(rope, c, rows, dev):
    """`rope` (or None) checked against a call of `rows` tokens on `dev`."""
    if rope is None:
        return None
    if rope._dev != dev and rope._dev != -1:
        raise ValueError(f"rope: on cuda:{rope._dev}, the call's other tensors on cuda:{dev}")
    if rope._n_pos is not None and rope._n_pos != rope.axes * rows:
        raise ValueError(f"rope.pos: {rope._n_pos} elements, {rope.axes * rows} are needed")
    if rope._n_w and rope._n_w != {c.d_head}:
        raise ValueError(f"rope.w_q, rope.w_k: {c.d_head} elements are needed")
    return _byref(rope)


def _kv4(cache, c, dev):
    if cache._dev != dev:
        raise ValueError(f"cache: on cuda:{cache._dev}, the call's other tensors on cuda:{dev}")
    if cache._shape != (c.B, c.G, c.d_head):
        raise ValueError(f"cache: made for (B, G, d_head) = {cache._shape}, not {(c.B, c.G, c.d_head)}")
    return _byref(cache)


def gqe_qk_rope(cfg, rope, Q, Qs, K, slot_pos, Qo, Qso, Ko, stream=None):
    c = _config(cfg)
    R, G, dh = c.B * c.T, c.G, c.d_head
    dev, nq, ns, nk = _first_device(Q, Qs, K), R * G * c.k * dh, R * dh, R * G * dh
    _call(_lib.gqe_qk_rope, dev, stream, _byref(c), _rope(rope, c, R, dev), _arg(Q, _BF16, nq, dev, "Q"),
          _arg(Qs, _BF16, ns, dev, "Qs"), _arg(K, _BF16, nk, dev, "K"),
          None if slot_pos is None else _arg(slot_pos, _I32, R * G * c.k, dev, "slot_pos"),
          _arg(Qo, _BF16, nq, dev, "Qo"), _arg(Qso, _BF16, ns, dev, "Qso"), _arg(Ko, _BF16, nk, dev, "Ko"))


def gqe_qk_rope_bwd(cfg, rope, Q, Qs, K, slot_pos, dQo, dQso, dKo, dQ, dQs, dK, dw_q, dw_k, ws, stream=None):
    c = _config(cfg)
    R, G, dh = c.B * c.T, c.G, c.d_head
    dev, nq, ns, nk = _first_device(dQo, dQso, dKo), R * G * c.k * dh, R * dh, R * G * dh
    _call(_lib.gqe_qk_rope_bwd, dev, stream, _byref(c), _rope(rope, c, R, dev), _arg(Q, _BF16, nq, dev, "Q"),
          _arg(Qs, _BF16, ns, dev, "Qs"), _arg(K, _BF16, nk, dev, "K"),
          None if slot_pos is None else _arg(slot_pos, _I32, R * G * c.k, dev, "slot_pos"),
          _arg(dQo, _F32, nq, dev, "dQo"), _arg(dQso, _F32, ns, dev, "dQso"), _arg(dKo, _F32, nk, dev, "dKo"),
          _arg(dQ, _F32, nq, dev, "dQ"), _arg(dQs, _F32, ns, dev, "dQs"), _arg(dK, _F32, nk, dev, "dK"),
          _arg(dw_q, _F32, dh, dev, "dw_q"), _arg(dw_k, _F32, dh, dev, "dw_k"), *_ws(ws, dev))


def gqe_router_logits(cfg, x, W_r, b_r, z, stream=None):
    c = _config(cfg)
    dev, R, N = _first_device(x), c.B * c.T, c.G * c.M
    _call(_lib.gqe_router_logits, dev, stream, _byref(c), _arg(x, _BF16, R * c.d_model, dev, "x"),
          _arg(W_r, _F32, c.d_model * N, dev, "W_r"), _arg(b_r, _F32, N, dev, "b_r"), _arg(z, _F32, R * N, dev, "z"))


def gqe_balance_stats(cfg, z, idx, mask, counts, sums, ws, stream=None):
    c = _config(cfg)
    dev, R, G = _first_device(z), c.B * c.T, c.G
    N = G * c.M
    _call(_lib.gqe_balance_stats, dev, stream, _byref(c), _arg(z, _F32, R * N, dev, "z"),
          _arg(idx, _I32, R * G * c.k, dev, "idx"), _arg(mask, _U8, R, dev, "mask"),
          _arg(counts, _I32, N + 1, dev, "counts"), _arg(sums, _F32, N + 1, dev, "sums"), *_ws(ws, dev))


def gqe_balance_loss(cfg, z, mask, counts, sums, c_balance, c_z, loss, dz, accumulate=False, stream=None):
    c = _config(cfg)
    dev, R, N = _first_device(counts), c.B * c.T, c.G * c.M
    _call(_lib.gqe_balance_loss, dev, stream, _byref(c), _arg(z, _F32, R * N, dev, "z"),
          _arg(mask, _U8, R, dev, "mask"), _arg(counts, _I32, N + 1, dev, "counts"),
          _arg(sums, _F32, N + 1, dev, "sums"), c_balance, c_z, _arg(loss, _F32, 3, dev, "loss"),
          _arg(dz, _F32, R * N, dev, "dz"), 1 if accumulate else 0)


def gqe_kv4_append(cfg, K, V, start, count, cache, stream=None):
    c = _config(cfg)
    B = c.B
    dev, n = _first_device(K), B * c.G * c.T * c.d_head
    _call(_lib.gqe_kv4_append, dev, stream, _byref(c), _arg(K, _BF16, n, dev, "K"), _arg(V, _BF16, n, dev, "V"),
          _arg(start, _I32, B, dev, "start"), _arg(count, _I32, B, dev, "count"), _kv4(cache, c, dev))


def gqe_kv4_read(cfg, cache, start, count, K, V, stream=None):
    c = _config(cfg)
    B = c.B
    dev, n = _first_device(K), B * c.G * c.T * c.d_head
    _call(_lib.gqe_kv4_read, dev, stream, _byref(c), _kv4(cache, c, dev), _arg(start, _I32, B, dev, "start"),
          _arg(count, _I32, B, dev, "count"), _arg(K, _BF16, n, dev, "K"), _arg(V, _BF16, n, dev, "V"))


def gqe_kv4_attention(cfg, Q, Qs, cache, lens, out, ws, stream=None):
    """out [B, ldo]: ldo is its row length."""
    c = _config(cfg)
    B, dh, ldo = c.B, c.d_head, out.shape[-1]
    dev = _first_device(Q)
    _call(_lib.gqe_kv4_attention, dev, stream, _byref(c), _arg(Q, _BF16, B * c.G * c.k * dh, dev, "Q"),
          _arg(Qs, _BF16, B * dh, dev, "Qs"), _kv4(cache, c, dev), _arg(lens, _I32, B, dev, "lens"),
          _arg(out, _BF16, B * ldo, dev, "out"), ldo, *_ws(ws, dev))


def _layer_args(c, rows, dev, x, W_r, b_r, W_q, W_qs, W_k, W_v, W_o):
    d, dh, N = c.d_model, c.d_head, c.G * c.M
    weighted = (c.flags & (GQE_FLAG_OUT_HARD | GQE_FLAG_OUT_WEIGHTED_CONCAT)) == 0
    slots = c.G * c.k + (1 if weighted else 0) + (1 if weighted and not c.flags & GQE_FLAG_NO_SHARED_HEAD else 0)
    return (_arg(x, _BF16, rows * d, dev, "x"), _arg(W_r, _F32, d * N, dev, "W_r"), _arg(b_r, _F32, N, dev, "b_r"),
            _arg(W_q, _BF16, d * N * dh, dev, "W_q"), _arg(W_qs, _BF16, d * dh, dev, "W_qs"),
            _arg(W_k, _BF16, d * c.G * dh, dev, "W_k"), _arg(W_v, _BF16, d * c.G * dh, dev, "W_v"),
            _arg(W_o, _BF16, slots * dh * d, dev, "W_o"))


def gqe_layer_fwd_rope(cfg, rope, x, W_r, b_r, W_q, W_qs, W_k, W_v, W_o, y, ws, stream=None):
    c = _config(cfg)
    dev, R = _first_device(x), c.B * c.T
    _call(_lib.gqe_layer_fwd_rope, dev, stream, ctypes.byref(c), _rope(rope, c, R, dev),
          *_layer_args(c, R, dev, x, W_r, b_r, W_q, W_qs, W_k, W_v, W_o), _arg(y, _BF16, R * c.d_model, dev, "y"),
          *_ws(ws, dev))


def gqe_layer_bwd_aux(cfg, rope, balance, x, W_r, b_r, W_q, W_qs, W_k, W_v, W_o, dy, dx, dW_r, db_r, dW_q, dW_qs, dW_k,
                      dW_v, dW_o, dw_qn, dw_kn, ws, stream=None):
    """gqe_layer_bwd with positions (GQERope or None) and the router's balance loss (GQEBalance or None)."""
    c = _config(cfg)
    dev, R, d, dh, N = _first_device(x), c.B * c.T, c.d_model, c.d_head, c.G * c.M
    if balance is not None and (balance._dev != dev or balance._n != N + 1 or balance._n_mask not in (None, R)):
        raise ValueError(f"balance: counts and sums of {N + 1}, a mask of {R} on cuda:{dev} are needed")
    grads = [(dy, R * d, "dy"), (dx, R * d, "dx"), (dW_r, d * N, "dW_r"), (db_r, N, "db_r"), (dW_q, d * N * dh, "dW_q"),
             (dW_qs, d * dh, "dW_qs"), (dW_k, d * c.G * dh, "dW_k"), (dW_v, d * c.G * dh, "dW_v"),
             (dW_o, (c.k * c.G + 2) * dh * d, "dW_o"), (dw_qn, dh, "dw_qn"), (dw_kn, dh, "dw_kn")]
    _call(_lib.gqe_layer_bwd_aux, dev, stream, ctypes.byref(c), _rope(rope, c, R, dev),
          None if balance is None else ctypes.byref(balance),
          *_layer_args(c, R, dev, x, W_r, b_r, W_q, W_qs, W_k, W_v, W_o),
          *(_arg(t, _F32, n, dev, what) for t, n, what in grads), *_ws(ws, dev))


def gqe_decode_step_rope(cfg, rope, x, W_r, b_r, W_q, W_qs, W_k, W_v, W_o, K_cache, V_cache, y, ws, stream=None):
    """gqe_decode_step with positions; the cache capacity is K_cache.shape[2]."""
    c = _config(cfg)
    dev, cap = _first_device(x), int(K_cache.shape[2])
    n = c.B * c.G * cap * c.d_head
    _call(_lib.gqe_decode_step_rope, dev, stream, ctypes.byref(c), _rope(rope, c, c.B, dev),
          *_layer_args(c, c.B, dev, x, W_r, b_r, W_q, W_qs, W_k, W_v, W_o), _arg(K_cache, _BF16, n, dev, "K_cache"),
          _arg(V_cache, _BF16, n, dev, "V_cache"), cap, _arg(y, _BF16, c.B * c.d_model, dev, "y"), *_ws(ws, dev))


def gqe_decode_step_kv4(cfg, rope, x, W_r, b_r, W_q, W_qs, W_k, W_v, W_o, cache, lens, y, ws, stream=None):
    c = _config(cfg)
    dev = _first_device(x)
    _call(_lib.gqe_decode_step_kv4, dev, stream, ctypes.byref(c), _rope(rope, c, c.B, dev),
          *_layer_args(c, c.B, dev, x, W_r, b_r, W_q, W_qs, W_k, W_v, W_o), _kv4(cache, c, dev),
          _arg(lens, _I32, c.B, dev, "lens"), _arg(y, _BF16, c.B * c.d_model, dev, "y"), *_ws(ws, dev))


def gqe_read_status() -> int:
    out = ctypes.c_int32(0)
    _check(_lib.gqe_read_status(ctypes.byref(out)), "gqe_read_status")
    return int(out.value)


def gqe_selftest_wait_timeout(limit_ns: int, stream=None):
    _check(_lib.gqe_selftest_wait_timeout(int(limit_ns), _stream(stream)),
           "gqe_selftest_wait_timeout")


def gqe_status_string(status: int) -> str:
    return _lib.gqe_status_string(status).decode()


def gqe_version() -> int:
    return int(_lib.gqe_version())


def workspace_view(ws: torch.Tensor, cfg, which: int, item, dtype, shape) -> torch.Tensor:
    """A typed view of one item of a layer / dense workspace (for inspection)."""
    off = gqe_workspace_offset(cfg, which, item)
    if off == 2 ** 64 - 1:
        raise ValueError(f"no item {item} in workspace {which}")
    n = 1
    for s in shape:
        n *= s
    nbytes = n * torch.empty((), dtype=dtype).element_size()
    return ws[off:off + nbytes].view(dtype).view(*shape)
