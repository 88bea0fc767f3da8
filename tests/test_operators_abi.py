"""The position, balance and 4-bit cache entry points refuse bad arguments on
the host, before anything is launched (CPU only; the pointers are never
dereferenced)."""
import ctypes

import pytest

A = ctypes.c_void_p(0x1000_0000)   # aligned
B4 = ctypes.c_void_p(0x1000_0004)  # 4-byte aligned only
ODD = ctypes.c_void_p(0x1000_0001)


@pytest.fixture(scope="module")
def rsq():
    from routed_sparse_query_b200 import build
    build.build()
    import routed_sparse_query_b200 as m
    return m


def _cfg(rsq, **kw):
    base = dict(B=1, T=64, d_model=256, G=4, M=2, k=1, d_head=64, flags=0)
    base.update(kw)
    return rsq.GQEConfig(*(base[n] for n in ("B", "T", "d_model", "G", "M", "k", "d_head", "flags")))


def _rope(rsq, **kw):
    base = dict(d_rot=64, axes=1, flags=rsq.GQE_ROPE_NORM, eps=1e-6, scale=1.0, pos=None, inv_freq=0x1000_0000, axis=None,
                w_q=None, w_k=None)
    base.update(kw)
    return rsq.GQERope(*(base[n] for n, _ in rsq.GQERope._fields_))


def _kv4(rsq, **kw):
    base = dict(k_codes=0x1000_0000, v_codes=0x1000_0000, meta=0x1000_0000, capacity=64)
    base.update(kw)
    return rsq.GQEKv4(*(base[n] for n, _ in rsq.GQEKv4._fields_))


R = ctypes.byref


def _fwd(rsq, c, r, Q=A, Qs=A, K=A, sp=None, Qo=A, Qso=A, Ko=A):
    return rsq.lib().gqe_qk_rope(R(c) if c is not None else None, R(r) if r is not None else None, Q, Qs, K, sp, Qo, Qso,
                                 Ko, None)


@pytest.mark.parametrize("bad", [dict(d_rot=-8), dict(d_rot=72), dict(axes=0), dict(axes=5), dict(flags=4), dict(eps=-1.0),
                                 dict(eps=float("nan")), dict(inv_freq=None), dict(inv_freq=0x1000_0004),
                                 dict(pos=0x1000_0002), dict(axis=0x1000_0001), dict(w_q=0x1000_0002),
                                 dict(w_k=0x1000_0002)])
def test_rope_descriptions_refused(rsq, bad):
    assert _fwd(rsq, _cfg(rsq), _rope(rsq, **bad)) == rsq.GQE_ERR_INVALID


def test_rope_arguments_refused(rsq):
    c, r = _cfg(rsq), _rope(rsq)
    assert _fwd(rsq, None, r) == rsq.GQE_ERR_INVALID
    assert _fwd(rsq, c, None) == rsq.GQE_ERR_INVALID
    assert _fwd(rsq, c, _rope(rsq, d_rot=12)) == rsq.GQE_ERR_UNSUPPORTED
    assert _fwd(rsq, _cfg(rsq, d_head=32), r) == rsq.GQE_ERR_INVALID  # d_rot > d_head
    assert _fwd(rsq, _cfg(rsq, d_head=128), r) == rsq.GQE_ERR_UNSUPPORTED
    assert _fwd(rsq, c, r, Q=None) == rsq.GQE_ERR_INVALID  # an output without its input
    assert _fwd(rsq, c, r, Ko=None) == rsq.GQE_ERR_INVALID
    assert _fwd(rsq, c, r, None, None, None, None, None, None, None) == rsq.GQE_ERR_INVALID
    assert _fwd(rsq, c, r, Q=B4) == rsq.GQE_ERR_INVALID
    assert _fwd(rsq, c, r, sp=ODD) == rsq.GQE_ERR_INVALID
    # More rows than int32 counts.
    assert _fwd(rsq, _cfg(rsq, B=1 << 15, T=1 << 15), r) == rsq.GQE_ERR_UNSUPPORTED


def test_rope_backward_arguments_refused(rsq):
    c, r = _cfg(rsq), _rope(rsq)
    need = rsq.gqe_workspace_bytes(c, rsq.GQE_WS_QK_ROPE)
    assert need > 0

    def bwd(r=r, Q=A, dQo=A, dQ=A, dw=A, ws=A, n=need):
        return rsq.lib().gqe_qk_rope_bwd(R(c), R(r), Q, A, A, None, dQo, A, A, dQ, A, A, dw, None, ws, n, None)

    assert bwd(n=need - 1) == rsq.GQE_ERR_WORKSPACE
    assert bwd(ws=None) == rsq.GQE_ERR_INVALID
    assert bwd(dQ=None) == rsq.GQE_ERR_INVALID
    assert bwd(Q=None) == rsq.GQE_ERR_INVALID  # the norm's backward reads it
    assert bwd(r=_rope(rsq, flags=0)) == rsq.GQE_ERR_INVALID  # weight gradients without a norm
    assert bwd(dw=ODD) == rsq.GQE_ERR_INVALID
    assert bwd(dQo=B4) == rsq.GQE_ERR_INVALID


def test_balance_arguments_refused(rsq):
    c = _cfg(rsq)
    need = rsq.gqe_workspace_bytes(c, rsq.GQE_WS_BALANCE)
    lib = rsq.lib()
    assert lib.gqe_balance_stats(R(c), A, A, None, A, A, A, need - 1, None) == rsq.GQE_ERR_WORKSPACE
    assert lib.gqe_balance_stats(R(c), A, A, None, A, A, None, need, None) == rsq.GQE_ERR_INVALID
    assert lib.gqe_balance_stats(R(c), A, None, None, A, A, A, need, None) == rsq.GQE_ERR_INVALID
    assert lib.gqe_balance_stats(R(c), B4, A, None, A, A, A, need, None) == rsq.GQE_ERR_INVALID
    assert lib.gqe_balance_stats(R(_cfg(rsq, k=3)), A, A, None, A, A, A, need, None) == rsq.GQE_ERR_INVALID
    assert lib.gqe_balance_loss(R(c), A, None, A, A, 1.0, 0.0, None, None, 0, None) == rsq.GQE_ERR_INVALID
    assert lib.gqe_balance_loss(R(c), None, None, A, A, 1.0, 0.0, A, A, 0, None) == rsq.GQE_ERR_INVALID
    assert lib.gqe_balance_loss(R(c), A, None, None, A, 1.0, 0.0, A, A, 0, None) == rsq.GQE_ERR_INVALID
    assert lib.gqe_router_logits(R(c), A, A, None, None, None) == rsq.GQE_ERR_INVALID
    assert lib.gqe_router_logits(R(c), A, A, ODD, A, None) == rsq.GQE_ERR_INVALID


def test_kv4_arguments_refused(rsq):
    c, lib = _cfg(rsq), rsq.lib()

    def append(c=c, K=A, start=None, kv=None):
        return lib.gqe_kv4_append(R(c), K, A, start, None, R(kv if kv is not None else _kv4(rsq)), None)

    for bad in (dict(k_codes=None), dict(v_codes=0x1000_0008), dict(meta=None), dict(capacity=0), dict(capacity=-16),
                dict(capacity=24)):
        assert append(kv=_kv4(rsq, **bad)) == rsq.GQE_ERR_INVALID
        assert lib.gqe_kv4_read(R(c), R(_kv4(rsq, **bad)), None, None, A, A, None) == rsq.GQE_ERR_INVALID
    assert lib.gqe_kv4_append(R(c), A, A, None, None, None, None) == rsq.GQE_ERR_INVALID
    assert append(K=None) == rsq.GQE_ERR_INVALID
    assert append(start=ODD) == rsq.GQE_ERR_INVALID
    assert append(c=_cfg(rsq, T=0)) == rsq.GQE_ERR_INVALID

    need = rsq.gqe_workspace_bytes(c, rsq.GQE_WS_KV4)

    def attn(c=c, Q=A, Qs=A, kv=None, lens=None, out=A, ldo=5 * 64, ws=A, n=need):
        return lib.gqe_kv4_attention(R(c), Q, Qs, R(kv if kv is not None else _kv4(rsq)), lens, out, ldo, ws, n, None)

    assert attn(n=0) == rsq.GQE_ERR_WORKSPACE
    assert attn(ws=None) == rsq.GQE_ERR_INVALID
    assert attn(Q=None) == rsq.GQE_ERR_INVALID
    assert attn(Qs=B4) == rsq.GQE_ERR_INVALID
    assert attn(lens=ODD) == rsq.GQE_ERR_INVALID
    assert attn(ldo=4 * 64) == rsq.GQE_ERR_INVALID   # no column for the shared head
    assert attn(ldo=5 * 64 + 4) == rsq.GQE_ERR_INVALID
    assert attn(kv=_kv4(rsq, capacity=48)) == rsq.GQE_ERR_INVALID  # shorter than T
    big = _cfg(rsq, G=1, M=17, k=17)
    assert rsq.gqe_workspace_bytes(big, rsq.GQE_WS_KV4) == 0
    assert attn(c=big, ldo=18 * 64) == rsq.GQE_ERR_UNSUPPORTED
    wide = _cfg(rsq, B=1 << 14, T=16)
    assert rsq.gqe_workspace_bytes(wide, rsq.GQE_WS_KV4) == 0
    assert attn(c=wide) == rsq.GQE_ERR_UNSUPPORTED


def test_layer_calls_refused(rsq):
    lib, c, r, kv = rsq.lib(), _cfg(rsq), _rope(rsq), _kv4(rsq)
    w = (A, None, A, A, A, A, A)  # W_r, b_r, W_q, W_qs, W_k, W_v, W_o
    need = rsq.gqe_workspace_bytes(c, rsq.GQE_WS_LAYER)
    assert lib.gqe_layer_fwd_rope(R(c), R(r), A, *w, A, A, need - 1, None) == rsq.GQE_ERR_WORKSPACE
    assert lib.gqe_layer_fwd_rope(R(c), None, A, *w, A, A, need, None) == rsq.GQE_ERR_INVALID
    assert lib.gqe_layer_fwd_rope(R(c), R(_rope(rsq, d_rot=4)), A, *w, A, A, need, None) == rsq.GQE_ERR_UNSUPPORTED

    need = rsq.gqe_workspace_bytes(c, rsq.GQE_WS_BACKWARD_AUX)
    assert need > rsq.gqe_workspace_bytes(c, rsq.GQE_WS_BACKWARD)
    bal = rsq.GQEBalance(None, 0.1, 0.0, 0x1000_0000, 0x1000_0000, None)

    def bwd(c=c, r=r, b=bal, dw=None, n=need):
        return lib.gqe_layer_bwd_aux(R(c), R(r) if r is not None else None, R(b) if b is not None else None, A, *w,
                                     *[A] * 9, dw, None, A, n, None)

    assert bwd(n=need - 1) == rsq.GQE_ERR_WORKSPACE
    assert bwd(r=None, dw=A) == rsq.GQE_ERR_INVALID
    assert bwd(r=_rope(rsq, flags=0), dw=A) == rsq.GQE_ERR_INVALID
    assert bwd(b=rsq.GQEBalance(None, 0.1, 0.0, None, 0x1000_0000, None)) == rsq.GQE_ERR_INVALID
    for flags in (rsq.GQE_FLAG_OUT_HARD, rsq.GQE_FLAG_EXPERT_MAJOR):
        assert bwd(c=_cfg(rsq, flags=flags)) == rsq.GQE_ERR_UNSUPPORTED
        assert rsq.gqe_workspace_bytes(_cfg(rsq, flags=flags), rsq.GQE_WS_BACKWARD_AUX) == 0

    need = rsq.gqe_workspace_bytes(c, rsq.GQE_WS_DECODE_KV4)

    def step(c=c, r=None, kv=kv, n=need, lens=None):
        return lib.gqe_decode_step_kv4(R(c), r, A, *w, R(kv), lens, A, A, n, None)

    assert step(n=need - 1) == rsq.GQE_ERR_WORKSPACE
    assert step(kv=_kv4(rsq, capacity=32)) == rsq.GQE_ERR_INVALID
    assert step(lens=ODD) == rsq.GQE_ERR_INVALID
    assert step(r=R(_rope(rsq, axes=9))) == rsq.GQE_ERR_INVALID
    for flags in (rsq.GQE_FLAG_OUT_HARD, rsq.GQE_FLAG_EXPERT_MAJOR, rsq.GQE_FLAG_NO_SHARED_HEAD):
        assert step(c=_cfg(rsq, flags=flags)) == rsq.GQE_ERR_UNSUPPORTED
    dec = lib.gqe_decode_step_rope
    assert dec(R(c), None, A, *w, A, A, 64, A, A, need, None) == rsq.GQE_ERR_INVALID
    em = _cfg(rsq, flags=rsq.GQE_FLAG_EXPERT_MAJOR)
    assert dec(R(em), R(r), A, *w, A, A, 64, A, A, need, None) == rsq.GQE_ERR_UNSUPPORTED
    assert dec(R(c), R(r), A, *w, A, A, 63, A, A, need, None) == rsq.GQE_ERR_INVALID  # capacity < T


def test_binding_refuses_cpu_tensors(rsq):
    import torch
    x = torch.zeros(4, dtype=torch.float64)
    with pytest.raises(ValueError):
        rsq.GQERope.of(8, x)
    with pytest.raises(ValueError):
        rsq.GQEKv4.of(*(torch.zeros(1, 1, 16, 32, dtype=torch.uint8),) * 2, torch.zeros(1, 1, 16, 4, dtype=torch.bfloat16))
