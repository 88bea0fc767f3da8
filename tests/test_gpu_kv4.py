"""The 4-bit K/V cache: stored rows bit for bit against the format's
definition, and the attention over them against fp64 on the stored values.

Attention tolerance, from three roundings: the output's (2^-8 of the value); the
weights', which may be rounded to bf16 (2^-8) against codes taken around the
middle of their range, |code - 8| <= 8: 2^-8 sum p 8 scale_v; and the scores', fp32
sums of d_head products, at most 2^-17 of the sum of their absolute values
(64 * 2^-24 = 2^-18 for the sum, as much again for the dequantisation): a score error
d moves the output by at most 2 d max|V|."""
import numpy as np
import pytest
import torch

from oracle import operators as op

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rsq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import routed_sparse_query_b200 as m
    return m


def new_cache(rsq, B, G, cap, dh, fill=None, seed=0):
    """A cache of random codes and sensible scales, or of the byte `fill`."""
    gen = torch.Generator().manual_seed(seed)
    if fill is None:
        codes = [torch.randint(0, 256, (B, G, cap, dh // 2), generator=gen, dtype=torch.uint8) for _ in range(2)]
        step = 0.15 + 0.2 * torch.rand(B, G, cap, 2, generator=gen)
        zero = -7.5 * step + 0.3 * torch.randn(B, G, cap, 2, generator=gen)
        meta = torch.stack([step[..., 0], zero[..., 0], step[..., 1], zero[..., 1]], -1).to(torch.bfloat16)
    else:
        codes = [torch.full((B, G, cap, dh // 2), fill, dtype=torch.uint8) for _ in range(2)]
        meta = torch.full((B, G, cap, 8), fill, dtype=torch.uint8).view(torch.bfloat16)
    t = [c.cuda() for c in codes] + [meta.cuda()]
    return t, rsq.GQEKv4.of(*t)


def host(t):
    return [x.cpu() for x in t]


def stored(codes, meta, at):
    """fp64 values of rows [..., dh/2] with meta [..., 4] (at: 0 keys, 2 values)."""
    m = meta.double().numpy()
    return op.kv4_values(op.kv4_unpack(codes.numpy()), m[..., at], m[..., at + 1])


SPECIAL = 12


def rows(B, G, T, dh, seed):
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn(B, G, T, dh, generator=gen) * torch.exp(2 * torch.randn(B, G, T, 1, generator=gen))).to(torch.bfloat16)
    f = x.view(-1, dh)
    if f.shape[0] >= SPECIAL:  # rows that the arithmetic could trip over
        f[0] = 0
        f[1] = 3.5
        f[2] = torch.arange(dh) % 16
        f[3] = torch.tensor([3.0e38, -3.0e38] * (dh // 2)).to(torch.bfloat16)
        f[4, 3] = float("inf")
        f[5, 7] = float("nan")
        f[6] = 1e-40
        f[7, :] = 1.0
        f[7, 0] = 1.0 + 2 ** -7
        f[8] = torch.linspace(-1e-38, 1e-38, dh).to(torch.bfloat16)
        f[9, 0] = -1000
        f[10, dh - 1] = -float("inf")
        f[11] = -0.0
    return x


@pytest.mark.parametrize("B,G,T,dh,cap", [(1, 1, 1, 64, 16), (3, 2, 7, 32, 32), (2, 8, 130, 64, 144), (64, 8, 1, 64, 64),
                                          (1, 3, 1000, 32, 1008)])
def test_append_and_read(rsq, B, G, T, dh, cap):
    K, V = rows(B, G, T, dh, 1), rows(B, G, T, dh, 2)
    gen = torch.Generator().manual_seed(3)
    start = torch.randint(0, cap - T + 1, (B,), generator=gen, dtype=torch.int32)
    count = torch.randint(0, T + 1, (B,), generator=gen, dtype=torch.int32)
    cfg = rsq.GQEConfig(B, T, 64, G, 1, 1, dh, 0)
    for st, ct in ((None, None), (start, None), (start, count)):
        t, cache = new_cache(rsq, B, G, cap, dh, fill=0x5A)
        before = host(t)
        dev = [None if x is None else x.cuda() for x in (st, ct)]
        rsq.gqe_kv4_append(cfg, K.cuda(), V.cuda(), *dev, cache)
        after = host(t)
        want = [x.clone() for x in before]
        Ko, Vo = (torch.full_like(K, 7.0).cuda() for _ in range(2))
        rsq.gqe_kv4_read(cfg, cache, *dev, Ko, Vo)
        Ko, Vo = Ko.cpu(), Vo.cpu()
        for b in range(B):
            s, n = (0 if st is None else int(st[b])), (T if ct is None else int(ct[b]))
            for x, out, ci, at in ((K, Ko, 0, 0), (V, Vo, 1, 2)):
                codes, scale, zero = op.kv4_quantise(x[b, :, :n].float().numpy())
                want[ci][b, :, s:s + n] = torch.from_numpy(op.kv4_pack(codes))
                want[2][b, :, s:s + n, at] = torch.from_numpy(scale).to(torch.bfloat16)
                want[2][b, :, s:s + n, at + 1] = torch.from_numpy(zero).to(torch.bfloat16)
                v = op.kv4_values(codes, scale, zero)
                got = out[b, :, :n].double().numpy()
                bad = np.isnan(v)
                assert np.array_equal(np.isnan(got), bad)
                # fp32, then bf16: half a step of each; 2^-134 for half a step among the subnormals
                assert (np.abs(got - v)[~bad] <= (2.0 ** -8 + 2.0 ** -23) * np.abs(v[~bad]) + 2.0 ** -134).all()
                assert (out[b, :, n:] == 7.0).all()  # rows past the count are left alone
        assert torch.equal(after[0], want[0]) and torch.equal(after[1], want[1])
        a, w = (m[2].view(torch.int16) for m in (after, want))
        nan = torch.isnan(want[2])
        assert torch.equal(torch.isnan(after[2]), nan) and torch.equal(a[~nan], w[~nan])
    assert rsq.gqe_read_status() == 0


@pytest.mark.parametrize("dh", [32, 64])
def test_codes_are_the_definitions(rsq, dh):
    # Bit for bit over many rows: quotients that are halves (codes half to
    # even), next to a half, scales at a border between two bf16, and scales of
    # every magnitude.
    rng = np.random.default_rng(7)
    n = 1 << 16
    x = rng.standard_normal((n, dh))
    x[n // 4: n // 2] = rng.integers(-64, 65, (n // 4, dh)) / 8.0  # few bits: many halves
    x[n // 2: 3 * n // 4] *= np.exp2(rng.integers(-120, 120, (n // 4, 1)))
    x[3 * n // 4:] = rng.standard_normal((n // 4, 1)) * 50 + rng.standard_normal((n // 4, dh))  # far from zero
    # zero -7.5, scale 1: 7.5 + x for small x of both signs, down to what fp32 loses.
    small = np.exp2(-rng.integers(0, 40, (64, dh)).astype(np.float64)) * rng.choice([-1, 1], (64, dh))
    small[:, 0], small[:, 1] = -7.5, 7.5
    # (max - min) / 15 half way between two bf16, and next to it.
    border = rng.random((64, dh)) * 15
    border[:, 0], border[:, 1] = 15.0, -0.05859375 * np.exp2(-(np.arange(64) % 4))
    x = np.concatenate([x, small, border]).astype(np.float32)
    x = op.bf16_round(x)
    T = 64
    B = x.shape[0] // T
    K = torch.from_numpy(x).to(torch.bfloat16).view(B, 1, T, dh)
    V = K.flip(2).contiguous()
    t, cache = new_cache(rsq, B, 1, T, dh, fill=0)
    rsq.gqe_kv4_append(rsq.GQEConfig(B, T, 64, 1, 1, 1, dh, 0), K.cuda(), V.cuda(), None, None, cache)
    got = host(t)
    for data, codes, at in ((K, got[0], 0), (V, got[1], 2)):
        c, s, z = op.kv4_quantise(data.float().numpy())
        meta = got[2].float().numpy()
        assert np.array_equal(meta[..., at], s) and np.array_equal(meta[..., at + 1], z)
        assert np.array_equal(op.kv4_unpack(codes.numpy()), c)
    assert rsq.gqe_read_status() == 0


def test_positions_outside_the_cache(rsq):
    B, G, T, dh, cap = 4, 2, 6, 64, 32
    K, V = rows(B, G, T, dh, 5), rows(B, G, T, dh, 6)
    cfg = rsq.GQEConfig(B, T, 64, G, 1, 1, dh, 0)
    t, cache = new_cache(rsq, B, G, cap, dh, fill=0)
    start = torch.tensor([-3, -100, 0, 26], dtype=torch.int32).cuda()
    rsq.gqe_kv4_append(cfg, K.cuda(), V.cuda(), start, None, cache)
    assert rsq.gqe_read_status() == 0
    touched = (t[0].cpu().view(B, G, cap, -1).any(-1) | t[2].cpu().float().ne(0).any(-1))
    assert touched[0, :, 3:].sum() == 0 and touched[1].sum() == 0 and touched[3, :, :26].sum() == 0
    rsq.gqe_kv4_append(cfg, K.cuda(), V.cuda(), torch.full((B,), 2 ** 31 - 1, dtype=torch.int32).cuda(), None, cache)
    assert rsq.gqe_read_status() == rsq.GQE_ERR_DEVICE_CHECK
    out = torch.full_like(K, 9.0).cuda()
    rsq.gqe_kv4_read(cfg, cache, torch.tensor([28, 0, 0, 0], dtype=torch.int32).cuda(), None, out, out.clone())
    assert rsq.gqe_read_status() == rsq.GQE_ERR_DEVICE_CHECK
    assert (out[0, :, 4:] == 9.0).all()  # positions 32, 33


# B, G, k, shared, dh, T, lens (None: all T)
ATTN = {
    "one_key": (1, 1, 1, True, 64, 1, None),
    "b1_2k": (1, 8, 1, True, 64, 2048, None),
    "ragged_dense4": (9, 2, 4, False, 64, 700, [700, 0, 1, 255, 256, 257, 699, 31, 33]),
    "dh32_k2": (3, 3, 2, True, 32, 515, [515, 17, 129]),
    "heads_8": (2, 2, 8, False, 64, 300, [300, 64]),
    "heads_9": (2, 2, 8, True, 64, 300, [65, 300]),
    "heads_16": (2, 1, 16, False, 64, 1000, [1000, 3]),
    "heads_16_dh32": (2, 2, 15, True, 32, 90, [63, 90]),
    "over_and_under": (4, 2, 1, True, 64, 100, [-5, 400, 100, 2 ** 31 - 1]),
    "spans": (2, 4, 2, True, 64, 9001, [9001, 4095]),
    "many_sequences": (150, 8, 1, True, 64, 70, None),
    "wide_batch": (700, 2, 1, True, 32, 200, [(37 * b) % 201 if b % 3 else 0 for b in range(700)]),
    "one_live_sequence": (300, 1, 2, False, 64, 3000, [0] * 299 + [3000]),
    # A cluster of 8, 4, 2 and 1 CTAs per (sequence, group), then equal shares with a join.
    "unit_8_tiles_per_warp": (2, 1, 1, True, 64, 32768, [32768, 32000]),
    "units_60": (20, 3, 2, True, 64, 1500, [(311 * b) % 1501 for b in range(20)]),
    "units_100": (25, 4, 4, False, 32, 1500, [(311 * b) % 1501 for b in range(25)]),
    "units_200_heads_6": (25, 8, 5, True, 64, 900, [(201 * b) % 901 for b in range(25)]),
    "units_296": (37, 8, 1, True, 64, 4096, [(1009 * b) % 4097 for b in range(37)]),
    "units_297": (297, 1, 4, False, 64, 1000, None),
    "long_k1": (1, 2, 1, True, 64, 40000, None),
    "long_dense4": (2, 1, 4, False, 64, 33001, [33001, 4095]),
    "long_dh32_k2": (2, 1, 2, True, 32, 33001, [17, 33001]),
    "long_heads_8": (1, 1, 8, False, 64, 33001, None),
    "long_heads_9": (1, 2, 8, True, 64, 33001, None),
    "long_heads_16": (1, 1, 16, False, 64, 33001, None),
    "long_heads_16_dh32": (1, 1, 15, True, 32, 33001, None),
    "nothing_live": (5, 2, 1, True, 64, 50, [0, -1, 0, -7, 0]),
}


def attention_reference(q, qs, t, lens, T, k):
    """out [B, heads, dh] and its tolerance, from the stored values."""
    codes_k, codes_v, meta = t
    B, G, dh = q.shape[0], q.shape[1], q.shape[-1]
    n_heads = G * k + (1 if qs is not None else 0)
    out, tol = np.zeros((B, n_heads, dh)), np.zeros((B, n_heads, dh))
    for b in range(B):
        n = min(max(lens[b], 0), T)
        if n == 0:
            continue
        for g in range(G):
            K = stored(codes_k[b, g, :n], meta[b, g, :n], 0)
            V = stored(codes_v[b, g, :n], meta[b, g, :n], 2)
            sv = meta[b, g, :n, 2].double().numpy()
            heads = [(g * k + s, q[b, g, s]) for s in range(k)] + ([(G * k, qs[b])] if g == 0 and qs is not None else [])
            for col, qq in heads:
                qv = qq.double().numpy()
                o = op.decode_attention(qv[None], K, V)[0]
                s = K @ qv / np.sqrt(dh)
                p = np.exp(s - s.max())
                p /= p.sum()
                d = 2.0 ** -17 * (np.abs(K) @ np.abs(qv)).max() / np.sqrt(dh)
                out[b, col] = o
                tol[b, col] = 2.0 ** -8 * np.abs(o) + 2.0 ** -8 * 8 * (p * sv).sum() + 2 * d * np.abs(V).max()
    return out, tol


def run_attention(rsq, cfg, q, qs, cache, lens, extra_cols=0, ws=None):
    B, dh = cfg.B, cfg.d_head
    cols = (cfg.G * cfg.k + (1 if qs is not None else 0)) * dh
    out = torch.full((B, cols + extra_cols), 5.0, dtype=torch.bfloat16, device="cuda")
    if ws is None:  # never written before: nothing in it may matter
        ws = torch.full((rsq.gqe_workspace_bytes(cfg, rsq.GQE_WS_KV4),), 255, dtype=torch.uint8, device="cuda")
    rsq.gqe_kv4_attention(cfg, q.cuda(), None if qs is None else qs.cuda(), cache,
                          None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda(), out, ws)
    assert (out[:, cols:] == 5.0).all()
    return out[:, :cols].cpu().view(B, -1, dh)


@pytest.mark.parametrize("name", list(ATTN))
def test_attention(rsq, name):
    B, G, k, shared, dh, T, lens = ATTN[name]
    cap = (T + 15) // 16 * 16 + 32
    t, cache = new_cache(rsq, B, G, cap, dh, seed=11)
    ls = [T] * B if lens is None else lens
    for b in range(B):  # what lies behind a sequence's keys is not looked at
        n = min(max(ls[b], 0), T)
        t[2][b, :, n:] = float("nan")
    gen = torch.Generator().manual_seed(12)
    q = (torch.randn(B, G, k, dh, generator=gen) * 1.5).to(torch.bfloat16)
    qs = torch.randn(B, dh, generator=gen).to(torch.bfloat16) if shared else None
    cfg = rsq.GQEConfig(B, T, 64, G, max(k, 1), k, dh, 0)
    got = run_attention(rsq, cfg, q, qs, cache, lens, extra_cols=64)
    want, tol = attention_reference(q, qs, host(t), ls, T, k)
    err = np.abs(got.double().numpy() - want)
    assert (err <= tol).all(), f"worst {np.nanmax(err / np.maximum(tol, 1e-30)):.3f} of the tolerance"
    assert torch.equal(got, run_attention(rsq, cfg, q, qs, cache, lens))
    assert rsq.gqe_read_status() == 0


@pytest.mark.parametrize("T", [5000, 200000])
def test_even_weights_over_many_keys(rsq, T):
    # Hardly any score differs: the output is a mean of T values, sqrt(T)
    # smaller than they are, and shows what the sums lose. Two roundings to bf16
    # (the weights', the output's), each uniform within half a step and of
    # 2^-8/sqrt(3) of the value at most as a standard deviation, in the values'
    # own sizes: below 2^-8 together.
    B, G, k, dh = 1, 2, 1, 64
    t, cache = new_cache(rsq, B, G, (T + 15) // 16 * 16, dh, seed=3)
    t[2][..., 3] = (-7.5 * t[2][..., 2].float()).to(torch.bfloat16)
    q = (0.01 * torch.randn(B, G, k, dh, generator=torch.Generator().manual_seed(1))).to(torch.bfloat16)
    cfg = rsq.GQEConfig(B, T, 64, G, 1, k, dh, 0)
    got = run_attention(rsq, cfg, q, None, cache, None)
    want, _ = attention_reference(q, None, host(t), [T], T, k)
    err = got.double().numpy() - want
    assert np.linalg.norm(err) <= 2.0 ** -8 * np.linalg.norm(want)


def test_large_and_small_values(rsq):
    # Queries and rows far from 1: nothing may leave fp32's range on the way.
    B, G, k, dh, T = 2, 2, 1, 64, 330
    for qm, km, vm in ((1e-30, 1e30, 1e30), (1e30, 1e-30, 1e-30), (2.0 ** 20, 2.0 ** -20, 2.0 ** 100), (1.0, 1.0, 2.0 ** -120)):
        t, cache = new_cache(rsq, B, G, 336, dh, seed=2)
        t[2][..., :2] *= km
        t[2][..., 2:] *= vm
        q = (torch.randn(B, G, k, dh, generator=torch.Generator().manual_seed(1)) * qm).to(torch.bfloat16)
        cfg = rsq.GQEConfig(B, T, 64, G, 1, k, dh, 0)
        got = run_attention(rsq, cfg, q, None, cache, None)
        want, tol = attention_reference(q, None, host(t), [T] * B, T, k)
        assert (np.abs(got.double().numpy() - want) <= tol).all(), (qm, km, vm)


def test_one_key_dominates(rsq):
    # A far larger score late and early in the sequence, tiny values on it,
    # large ones on the others.
    B, G, k, dh, T = 1, 1, 1, 64, 1500
    for at in (0, 7, 777, 1499):
        t, cache = new_cache(rsq, B, G, 1504, dh, seed=4)
        t[2][..., 2:] *= 1024.0
        t[2][0, 0, at, 0], t[2][0, 0, at, 1] = 0.0, 4.0   # key 4 everywhere
        t[2][0, 0, at, 2:] *= 2.0 ** -30
        q = torch.full((B, G, k, dh), 2.0).to(torch.bfloat16)
        cfg = rsq.GQEConfig(B, T, 64, G, 1, k, dh, 0)
        got = run_attention(rsq, cfg, q, None, cache, None)
        want, tol = attention_reference(q, None, host(t), [T], T, k)
        assert (np.abs(got.double().numpy() - want) <= tol).all(), at


def test_a_bad_row_reaches_its_own_heads_only(rsq):
    B, G, k, dh, T = 2, 2, 2, 64, 100
    t, cache = new_cache(rsq, B, G, 112, dh, seed=4)
    q = torch.randn(B, G, k, dh, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    cfg = rsq.GQEConfig(B, T, 64, G, 2, k, dh, 0)
    want = run_attention(rsq, cfg, q, None, cache, None)
    t[2][1, 0, 50] = float("nan")
    got = run_attention(rsq, cfg, q, None, cache, None)
    assert torch.isnan(got[1, :k]).all()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1, k:], want[1, k:])
    q[0, 1, 0, 3] = float("nan")
    t[2][1, 0, 50] = 0.25
    got = run_attention(rsq, cfg, q, None, cache, None)
    assert torch.isnan(got[0, k]).all() and torch.isfinite(got[0, k + 1:].float()).all()


def test_capture_with_growing_lengths(rsq):
    # One captured step serves every length: append and attention read start
    # and lens from the device.
    B, G, k, dh, T = 3, 2, 1, 64, 300
    gen = torch.Generator().manual_seed(8)
    K, V = (torch.randn(B, G, T, dh, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.randn(B, G, k, dh, generator=gen).to(torch.bfloat16).cuda()
    t, cache = new_cache(rsq, B, G, 304, dh, fill=0)
    one, cfg = rsq.GQEConfig(B, 1, 64, G, 1, k, dh, 0), rsq.GQEConfig(B, T, 64, G, 1, k, dh, 0)
    ws = torch.empty(rsq.gqe_workspace_bytes(cfg, rsq.GQE_WS_KV4), dtype=torch.uint8, device="cuda")
    kn, vn = torch.empty(B, G, 1, dh, dtype=torch.bfloat16, device="cuda"), torch.empty(B, G, 1, dh, dtype=torch.bfloat16, device="cuda")
    start, lens = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.ones(B, dtype=torch.int32, device="cuda")
    out = torch.empty(B, G * k * dh, dtype=torch.bfloat16, device="cuda")

    def step():
        rsq.gqe_kv4_append(one, kn, vn, start, None, cache)
        rsq.gqe_kv4_attention(cfg, q, None, cache, lens, out, ws)

    kn.copy_(K[:, :, :1])
    vn.copy_(V[:, :, :1])
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in range(T):
        kn.copy_(K[:, :, n:n + 1])
        vn.copy_(V[:, :, n:n + 1])
        start.fill_(n)
        lens.fill_(n + 1)
        graph.replay()
        if n in (0, 1, 63, 64, 255, 256, T - 1):
            got = out.clone()
            t2, c2 = new_cache(rsq, B, G, 304, dh, fill=0)
            rsq.gqe_kv4_append(rsq.GQEConfig(B, n + 1, 64, G, 1, k, dh, 0), K[:, :, :n + 1].contiguous(),
                               V[:, :, :n + 1].contiguous(), None, None, c2)
            ref = run_attention(rsq, cfg, q.cpu(), None, c2, [n + 1] * B)
            assert torch.equal(got.cpu().view(B, -1, dh), ref), n
    assert rsq.gqe_read_status() == 0


def test_two_streams_with_their_own_workspaces(rsq):
    B, G, k, dh, T = 4, 8, 1, 64, 3000
    t, cache = new_cache(rsq, B, G, 3008, dh, seed=6)
    cfg = rsq.GQEConfig(B, T, 64, G, 1, k, dh, 0)
    q = [torch.randn(B, G, k, dh, generator=torch.Generator().manual_seed(s)).to(torch.bfloat16).cuda() for s in range(2)]
    want = [run_attention(rsq, cfg, x.cpu(), None, cache, None) for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    n = rsq.gqe_workspace_bytes(cfg, rsq.GQE_WS_KV4)
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    out = [torch.empty(B, G * k * dh, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for i in range(2):
            rsq.gqe_kv4_attention(cfg, q[i], None, cache, None, out[i], ws[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(out[i].cpu().view(B, -1, dh), want[i])
