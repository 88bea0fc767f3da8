"""The 4-bit attention's sums, sharply: by how much the outputs miss the fp64
result beyond their own rounding to bf16.

For an output `out` that is the nearest bf16 to the kernel's fp32 value x, the
excess max(0, |out - want| - ulp(out) / 2) is at most |x - want|. What x may be off
by, for one head with weights p (they sum to 1) over values of scale s:
  - each weight p s enters the tensor cores as two bf16 parts: 8 bits cut off, then
    8 bits rounded, 2^-16 of it in all, against codes taken around 8, |n - 8| <= 8.
    Independent and uniform: a standard deviation of 8 * 2^-16 / sqrt(3) *
    sqrt(sum (p s)^2).
  - the tensor cores cut a tile's sums (of up to 31 p s, fresh for every tile) off,
    always downwards: at most 2^-22 of them for each of the four products, 2^-15
    of W = sum p s in all.
  - running sums in fp32, of at most A = 31 W + sum p |zero + 8 s|: each of m
    additions rounds by 2^-24 at most, uniformly. A lane adds a weight for every
    eighth key, twice, a tile's sums once, and the parts are joined: m <= keys / 4 +
    keys / 64 + 400.
  - the scores: sums of d_head products cut off by 2^-20 of their terms' size
    and three roundings, e = 2^-19 * (15 scale_k + |zero_k|) sum|q| / sqrt(d_head),
    and 2^-21 for the exponential; a weight's error (e + 2^-21) p_u moves the output by
    that times V_u - o.
The bound of a head's excess over its elements, as a norm: the cut-off plus four of
the standard deviations, the scores' taken as independent too.

It is sharp enough to see a tile left out: test_a_lost_tile_would_show."""
import numpy as np
import pytest
import torch

from oracle import operators as op
from test_gpu_kv4 import host, new_cache, rsq, run_attention, stored  # noqa: F401


def excess(out, want):
    """|out - want| beyond half a step of the bf16 value out (fp64 arrays)."""
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(out), 2.0 ** -126))) - 7)
    return np.maximum(np.abs(out - want) - step / 2, 0)


def heads_of(q, qs, g):
    k = q.shape[2]
    return [(g * k + s, s) for s in range(k)] + ([(q.shape[1] * k, None)] if g == 0 and qs is not None else [])


def head_bound(p, V, sv, zv, o, kmax, qv):
    """Norm of the excess that the roundings explain (see above)."""
    n, dh = V.shape
    W = (p * sv).sum()
    A = 31 * W + (p * np.abs(zv + 8 * sv)).sum()
    std = np.sqrt(dh * (64 * 2.0 ** -32 / 3 * ((p * sv) ** 2).sum() + 2.0 ** -48 / 3 * (n / 4 + n / 64 + 400) * A * A))
    e = 2.0 ** -19 * kmax * np.abs(qv).sum() / np.sqrt(dh) + 2.0 ** -21
    return np.sqrt(dh) * 2.0 ** -15 * W + 4 * std + 4 * e * np.sqrt((p * p * ((V - o) ** 2).sum(1)).sum())


def reference(q, qs, t, lens):
    """(b, column, o, bound, p, V) of every head with keys."""
    B, G, k, dh = q.shape
    for b in range(B):
        n = lens[b]
        for g in range(G) if n else []:
            K, V = (stored(t[i][b, g, :n], t[2][b, g, :n], 2 * i) for i in range(2))
            m = t[2][b, g, :n].double().numpy()
            kmax = (15 * m[:, 0] + np.abs(m[:, 1])).max()
            for col, s in heads_of(q, qs, g):
                qv = (qs[b] if s is None else q[b, g, s]).double().numpy()
                sc = K @ qv / np.sqrt(dh)
                p = np.exp(sc - sc.max())
                p /= p.sum()
                o = op.decode_attention(qv[None], K, V)[0]
                yield b, col, o, head_bound(p, V, m[:, 2], m[:, 3], o, kmax, qv), p, V


def make(rsq, case, seed=21):  # noqa: F811
    """Even weights over values around 0: the outputs are far smaller than the
    values, and show what the sums lose."""
    B, G, k, shared, dh, T, lens = case
    cap = (T + 15) // 16 * 16
    t, cache = new_cache(rsq, B, G, cap, dh, seed=seed)
    t[2][..., 3] = (-7.5 * t[2][..., 2].float()).to(torch.bfloat16)
    gen = torch.Generator().manual_seed(seed + 1)
    q = (0.05 * torch.randn(B, G, k, dh, generator=gen)).to(torch.bfloat16)
    qs = (0.05 * torch.randn(B, dh, generator=gen)).to(torch.bfloat16) if shared else None
    cfg = rsq.GQEConfig(B, T, 64, G, k, k, dh, 0)
    return t, cache, q, qs, cfg, [T] * B if lens is None else lens


# Heads per group: one column each up to 2, 4 columns, 8 and 16; both head sizes.
# few: a tile or less, where a weight's rounding shows most; unit: a cluster per
# (sequence, group); shares: equal shares and a join.
CASES = {}
for k, shared in ((1, False), (1, True), (2, False), (3, False), (4, False), (5, False), (7, True), (9, False), (15, True)):
    for dh in (32, 64):
        h = f"h{k + shared}_dh{dh}"
        CASES["few_" + h] = (6, 2, k, shared, dh, 200, [2, 16, 47, 64, 65, 200])
        CASES["unit_" + h] = (2, 1, k, shared, dh, 5003, [5003, 1000])
        CASES["shares_" + h] = (2, 1, k, shared, dh, 33001, [33001, 1000])


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(CASES))
def test_even_weights(rsq, name):  # noqa: F811
    t, cache, q, qs, cfg, lens = make(rsq, CASES[name])
    got = run_attention(rsq, cfg, q, qs, cache, CASES[name][-1]).double().numpy()
    worst = 0.0
    for b, col, o, bound, _, _ in reference(q, qs, host(t), lens):
        worst = max(worst, np.linalg.norm(excess(got[b, col], o)) / bound)
    assert worst <= 1, f"{worst:.2f} of the bound"
    assert rsq.gqe_read_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["h1", "h4", "h8_dh32", "h16"])
def test_uneven_weights(rsq, name):  # noqa: F811
    # Scores of a few units and values away from zero.
    k, dh = {"h1": (1, 64), "h4": (4, 64), "h8_dh32": (8, 32), "h16": (16, 64)}[name]
    case = (3, 2, k, False, dh, 9001, [9001, 63, 700])
    t, cache, q, qs, cfg, lens = make(rsq, case, seed=31)
    t[2][..., 3] += 0.5
    q = (20 * q.float()).to(torch.bfloat16)
    got = run_attention(rsq, cfg, q, qs, cache, lens).double().numpy()
    for b, col, o, bound, _, _ in reference(q, qs, host(t), lens):
        e = np.linalg.norm(excess(got[b, col], o))
        assert e <= bound, f"{b} {col}: {e / bound:.2f} of the bound"


class _Host:
    """The parts of the binding that `make` uses, for the CPU."""
    class GQEKv4:
        of = staticmethod(lambda *t: None)
    GQEConfig = staticmethod(lambda *a: None)


@pytest.mark.parametrize("name", [n for n in CASES if n.startswith(("unit", "shares")) and ("h1_" in n or "h16" in n or "h5" in n)])
def test_a_lost_tile_would_show(monkeypatch, name):
    # The fp64 result without one 64-key tile, rounded to bf16, is outside the
    # bound, whichever tile it is.
    monkeypatch.setattr(torch.Tensor, "cuda", lambda self: self)
    t, _, q, qs, _, lens = make(_Host, CASES[name])
    for b, col, o, bound, p, V in reference(q, qs, t, lens):
        starts = np.arange(0, len(p), 64)
        pt = np.add.reduceat(p, starts)
        ot = np.add.reduceat(p[:, None] * V, starts)
        for i in range(len(starts)):
            if lens[b] - starts[i] < 32:  # a tile of a few keys: fewer than the bound resolves
                continue
            lost = (o - ot[i]) / (1 - pt[i])
            out = torch.from_numpy(lost).to(torch.bfloat16).double().numpy()
            assert np.linalg.norm(excess(out, o)) > bound, (b, col, i)
