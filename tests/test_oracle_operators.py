"""Pins of the fp64 operator definitions (oracle.operators), CPU only:
gradients against central differences, invariants of the rotation, the
balance loss and the 4-bit rows."""
import numpy as np
import pytest

from oracle import operators as op


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("d_rot", [0, 8, 16, 32])
def test_rope_rotation_keeps_pair_norms_and_relative_angles(adjacent, d_rot):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 5, 32))
    inv = 100.0 ** (-2.0 * np.arange(d_rot // 2) / max(d_rot, 1))
    pos = np.array([[0, 1, 7, 100000, 3]])
    y = op.rope(x, op.rope_angles(pos, inv, None), norm=False, adjacent=adjacent)
    assert np.allclose(y[..., d_rot:], x[..., d_rot:], rtol=0, atol=0)
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
    assert np.allclose(y[:, 0], x[:, 0])  # position 0
    # <rope(q, p), rope(k, p')> depends on p - p' only.
    q, k = x[0, :1], x[1, :1]
    dots = []
    for p in (0, 11, 5000):
        a = op.rope(q, op.rope_angles(np.array([[p + 4]]), inv, None), norm=False, adjacent=adjacent)
        b = op.rope(k, op.rope_angles(np.array([[p]]), inv, None), norm=False, adjacent=adjacent)
        dots.append(float((a * b).sum()))
    assert np.allclose(dots, dots[0])


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("adjacent", [False, True])
def test_rope_backward_matches_differences(norm, adjacent):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((2, 3, 8))
    g = rng.standard_normal(x.shape)
    w = 1.0 + 0.2 * rng.standard_normal(8)
    pos = rng.integers(0, 50, (2, 3))
    ang = op.rope_angles(pos, np.array([1.0, 0.1]), np.array([1, 0]))
    kw = dict(norm=norm, eps=0.01, scale=1.3, adjacent=adjacent)
    dx, dw = op.rope_backward(x, g, ang, w=w, **kw)
    h = 1e-5

    def f(x_, w_):
        return float((op.rope(x_, ang, w=w_, **kw) * g).sum())

    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[i]) < 1e-8
    if norm:
        for i in range(8):
            e = np.zeros(8)
            e[i] = h
            assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - dw[i]) < 1e-8
    else:
        assert dw is None


def test_balance_gradient_matches_differences():
    rng = np.random.default_rng(3)
    R, G, M, k = 7, 2, 3, 2
    z = rng.standard_normal((R, G * M))
    idx = np.sort(np.argsort(-z.reshape(R, G, M), axis=-1)[..., :k], axis=-1)
    mask = np.array([1, 1, 0, 1, 1, 0, 1])
    ref = op.balance(z, idx, mask, G, M, 0.3, 0.05)
    assert ref["counts"].sum() == 5 * G * k and ref["n"] == 5
    h = 1e-5
    for i in np.ndindex(z.shape):
        e = np.zeros_like(z)
        e[i] = h
        d = (op.balance(z + e, idx, mask, G, M, 0.3, 0.05)["loss"][0]
             - op.balance(z - e, idx, mask, G, M, 0.3, 0.05)["loss"][0]) / (2 * h)
        assert abs(d - ref["dz"][i]) < 1e-9


def test_balance_of_uniform_routing_is_one_and_nothing_counted_is_zero():
    G, M = 2, 4
    z = np.zeros((M, G * M))
    idx = np.repeat(np.arange(M)[:, None, None], G, axis=1)
    ref = op.balance(z, idx, None, G, M, 1.0, 0.0)
    assert np.isclose(ref["loss"][1], 1.0) and np.allclose(ref["dz"], 0)
    off = op.balance(np.full((M, G * M), np.nan), idx, np.zeros(M), G, M, 1.0, 1.0)
    assert (off["loss"] == 0).all() and (off["dz"] == 0).all() and off["counts"].sum() == 0


def test_kv4_rows():
    rng = np.random.default_rng(4)
    x = op.bf16_round(rng.standard_normal((50, 64)))
    codes, scale, zero = op.kv4_quantise(x)
    v = op.kv4_values(codes, scale, zero)
    # Half a step, and what rounding the step to 8 bits moves the last code by
    # (15 steps * 2^-8) -- the row's ends are off by no more than that.
    assert (np.abs(v - x) <= scale[:, None] * (0.5 + 15 * 2.0 ** -8)).all()
    assert np.array_equal(v.min(-1), x.min(-1).astype(np.float64))
    assert np.array_equal(op.kv4_unpack(op.kv4_pack(codes)), codes)
    # A constant row, a row of 16 levels, one past the range of a difference, bad rows.
    c, s, z = op.kv4_quantise(np.full((1, 32), 3.0))
    assert (c == 0).all() and s[0] == 0 and z[0] == 3.0
    lv = np.arange(16, dtype=np.float32).repeat(2)[None]
    assert np.array_equal(op.kv4_values(*op.kv4_quantise(lv)), lv)
    big = np.array([[3.0e38, -3.0e38] * 16], dtype=np.float32)
    assert np.isfinite(op.kv4_values(*op.kv4_quantise(op.bf16_round(big)))).all()
    bad = np.zeros((2, 32), dtype=np.float32)
    bad[0, 3], bad[1, 5] = np.inf, np.nan
    assert np.isnan(op.kv4_values(*op.kv4_quantise(bad))).all()


def test_decode_attention_without_keys_is_zero():
    q = np.ones((2, 32))
    assert (op.decode_attention(q, np.zeros((0, 32)), np.zeros((0, 32))) == 0).all()
