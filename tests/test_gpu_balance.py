"""The router's balance loss (gqe_balance_stats, gqe_balance_loss) against the
fp64 definition.

Tolerances. Counts are equal. p and lse come from the hardware's exponential to
base 2, reciprocal and logarithm and a sum of M <= 64 terms: at most 2^-17
relative (64 * 2^-24 = 2^-18 for the sum; the exponential's argument, a difference
of up to 18 times log2 e, two roundings of 2^-24 of 26 and the constant's 2^-26: 2^-18.6
of the term; 2^-22 each for the three functions; together 2^-17.1), lse 2^-17 of
1 + |lse|. sums: those errors plus at most 2^-18 for the fp32 partial sums (of a
thread, a CTA, and the CTAs that one thread of the last step takes). dz: 2^-15 of
the terms' sizes -- with the loads taken around their mean 1/M, as cancellation
would have cost more than that near balance."""
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


# B, T, G, M, k, skew, share of rows counted (None: no mask)
CASES = {
    "one_row": (1, 1, 2, 2, 1, 0.0, None),
    "layer_2k": (1, 2048, 8, 2, 1, 0.0, None),
    "cluster_2560": (1, 2560, 8, 2, 1, 0.0, None),  # as many rows as one cluster takes, and one more
    "cluster_2561": (1, 2561, 8, 2, 1, 0.0, None),
    "pool_masked": (2, 777, 8, 4, 2, 2.0, 0.7),
    "m1": (1, 33, 4, 1, 1, 0.0, None),
    "m3_g5": (3, 41, 5, 3, 2, 0.5, 0.5),
    "m8_all_selected": (1, 100, 2, 8, 8, 0.0, None),
    "m13": (1, 90, 4, 13, 3, 1.0, 0.9),
    "m32_g2": (1, 65, 2, 32, 4, 0.0, None),
    "m64": (2, 50, 1, 64, 5, 1.0, 0.3),
    "m16_all_selected": (1, 77, 2, 16, 16, 1.0, 0.8),
    "m19_k9": (1, 3001, 2, 19, 9, 1.0, 0.8),
    "m20": (3, 301, 3, 20, 2, 1.0, None),
    "m40": (1, 999, 1, 40, 12, 2.0, 0.5),
    "m61": (1, 64, 1, 61, 1, 0.0, 0.9),
    "m64_long": (1, 20011, 1, 64, 8, 2.0, 0.9),
    "g32_m2": (1, 300, 32, 2, 1, 0.0, None),
    "nothing_counted": (1, 40, 4, 2, 1, 0.0, 0.0),
    "long": (1, 70001, 8, 4, 2, 2.0, 0.8),
}


def make(case, seed=9):
    B, T, G, M, k, skew, share = case
    rng = np.random.default_rng(seed)
    z = rng.standard_normal((B * T, G, M)).astype(np.float32) * 2
    z[:, :, 0] += skew
    idx = np.sort(np.argsort(-z, axis=-1, kind="stable")[..., :k], axis=-1).astype(np.int32)
    mask = None if share is None else (rng.random(B * T) < share).astype(np.uint8)
    return z.reshape(B * T, G * M), idx, mask


def call(rsq, case, z, idx, mask, cb, cz, dz=None, accumulate=False):
    B, T, G, M, k = case[:5]
    cfg = rsq.GQEConfig(B, T, 64, G, M, k, 64, 0)
    N = G * M
    dev = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    zc, ic, mc = dev(z), dev(idx), dev(mask)
    counts = torch.full((N + 1,), -1, dtype=torch.int32, device="cuda")
    sums, loss = torch.full((N + 1,), float("nan"), device="cuda"), torch.full((3,), float("nan"), device="cuda")
    ws = torch.full((rsq.gqe_workspace_bytes(cfg, rsq.GQE_WS_BALANCE),), 255, dtype=torch.uint8, device="cuda")
    dz = torch.full((B * T, N), float("nan"), device="cuda") if dz is None else dz
    rsq.gqe_balance_stats(cfg, zc, ic, mc, counts, sums, ws)
    rsq.gqe_balance_loss(cfg, zc, mc, counts, sums, cb, cz, loss, dz, accumulate)
    return {"counts": counts.cpu().numpy(), "sums": sums.double().cpu().numpy(), "loss": loss.double().cpu().numpy(),
            "dz": dz.double().cpu().numpy()}


@pytest.mark.parametrize("name", list(CASES))
def test_matches_the_definition(rsq, name):
    case = CASES[name]
    B, T, G, M, k = case[:5]
    z, idx, mask = make(case)
    cb, cz = 0.02, 0.003
    ref = op.balance(z.astype(np.float64), idx, mask, G, M, cb, cz)
    got = call(rsq, case, z, idx, mask, cb, cz)
    n = ref["n"]
    assert np.array_equal(got["counts"][:-1].reshape(G, M), ref["counts"]) and got["counts"][-1] == n
    assert (np.abs(got["sums"][:-1].reshape(G, M) - ref["psum"]) <= 2.0 ** -16 * ref["psum"]).all()
    lse2 = (1 + np.abs(ref["lse"])) ** 2
    assert abs(got["sums"][-1] - ref["zsum"]) <= 2.0 ** -15 * lse2.sum()
    assert abs(got["loss"][1] - ref["loss"][1]) <= 2.0 ** -15 * abs(ref["loss"][1])
    if n:
        ztol = 2.0 ** -15 * lse2.sum() / (n * G)
        assert abs(got["loss"][2] - ref["loss"][2]) <= ztol
        assert abs(got["loss"][0] - ref["loss"][0]) <= cb * 2.0 ** -14 * abs(ref["loss"][1]) + cz * ztol + 2.0 ** -22 * abs(ref["loss"][0])
        f = ref["counts"] / (k * n) - 1 / M
        size = cb * M / (G * n) * ref["p"] * (np.abs(f) + (ref["p"] * np.abs(f)).sum(-1, keepdims=True))
        size += cz * 2 / (n * G) * ref["p"] * (1 + np.abs(ref["lse"]))[..., None]
        on = np.ones(B * T, dtype=bool) if mask is None else mask != 0
        err = np.abs(got["dz"] - ref["dz"]).reshape(B * T, G, M)
        assert (err[on] <= 2.0 ** -15 * size).all()
        assert (got["dz"][~on] == 0).all()
    else:
        assert (got["loss"] == 0).all() and (got["dz"] == 0).all() and (got["sums"] == 0).all()
    again = call(rsq, case, z, idx, mask, cb, cz)
    assert all(np.array_equal(got[key], again[key]) for key in got)  # the same sums in the same order


def test_masked_rows_may_hold_anything(rsq):
    case = (1, 64, 4, 2, 1, 0.0, 0.5)
    z, idx, mask = make(case)
    want = call(rsq, case, z, idx, mask, 0.1, 0.1)
    z2, idx2 = z.copy(), idx.copy()
    off = mask == 0
    z2[off] = np.array([np.nan, np.inf, -np.inf, np.finfo(np.float32).min] * 2, dtype=np.float32)
    idx2[off] = 2 ** 31 - 1
    got = call(rsq, case, z2, idx2, mask, 0.1, 0.1)
    assert all(np.array_equal(want[key], got[key]) for key in want)


def test_low_logits_and_indices_outside(rsq):
    # Experts switched off by -inf or the type's lowest value get no probability
    # and no gradient; an index outside the group counts for nobody.
    case = (1, 32, 2, 4, 2, 0.0, None)
    z, idx, _ = make(case)
    z.reshape(32, 2, 4)[:, 0, 3] = -np.inf
    z.reshape(32, 2, 4)[:, 1, 2] = np.finfo(np.float32).min
    idx[0, 0] = (-1, 4)
    with np.errstate(invalid="ignore"):
        ref = op.balance(z.astype(np.float64), idx, None, 2, 4, 0.1, 0.1)
    got = call(rsq, case, z, idx, None, 0.1, 0.1)
    assert np.array_equal(got["counts"][:-1].reshape(2, 4), ref["counts"])
    d = got["dz"].reshape(32, 2, 4)
    assert np.isfinite(d).all() and (d[:, 0, 3] == 0).all() and (d[:, 1, 2] == 0).all()
    assert np.allclose(got["dz"], ref["dz"], rtol=2.0 ** -12, atol=2.0 ** -15 * np.abs(ref["dz"]).max())


def test_group_switched_off_and_wide_logits(rsq):
    # A group whose experts all hold the type's lowest value has equal
    # probabilities; lse^2 then passes fp32, and a factor of 0 leaves it out.
    # p: a softmax of z - max, exact here up to one rounding of the difference.
    case = (1, 40, 3, 4, 2, 0.0, None)
    z, idx, _ = make(case)
    zg = z.reshape(40, 3, 4)
    zg[3, 1] = zg[17, 2] = np.finfo(np.float32).min
    zg[5, 0] = (2.0e38, -2.0e38, 1.0, 2.0e38)
    idx[9, 1] = (2, 2)  # an expert named twice counts twice
    ref = op.balance(z.astype(np.float64), idx, None, 3, 4, 0.1, 0.0)
    got = call(rsq, case, z, idx, None, 0.1, 0.0)
    assert np.array_equal(got["counts"][:-1].reshape(3, 4), ref["counts"])
    assert (np.abs(got["sums"][:-1].reshape(3, 4) - ref["psum"]) <= 2.0 ** -16 * ref["psum"]).all()
    assert np.isinf(got["sums"][-1]) and np.isinf(got["loss"][2])
    assert abs(got["loss"][1] - ref["loss"][1]) <= 2.0 ** -15 * ref["loss"][1]
    assert abs(got["loss"][0] - ref["loss"][0]) <= 2.0 ** -14 * ref["loss"][0]
    f = ref["counts"] / 80 - 0.25
    size = 0.1 * 4 / 120 * ref["p"] * (np.abs(f) + (ref["p"] * np.abs(f)).sum(-1, keepdims=True))
    assert (np.abs(got["dz"].reshape(40, 3, 4) - ref["dz"].reshape(40, 3, 4)) <= 2.0 ** -15 * size).all()


def test_accumulates_and_sums_of_two_ranks(rsq):
    # dz += with accumulate; two halves of a batch with added statistics give
    # the whole batch's gradient.
    case = (2, 100, 8, 2, 1, 1.0, 0.9)
    z, idx, mask = make(case)
    whole = call(rsq, case, z, idx, mask, 0.1, 0.01)
    base = torch.randn(200, 16, generator=torch.Generator().manual_seed(2)).cuda()
    acc = call(rsq, case, z, idx, mask, 0.1, 0.01, dz=base.clone(), accumulate=True)
    expect = (base + torch.from_numpy(whole["dz"]).float().cuda()).double().cpu().numpy()
    assert np.array_equal(acc["dz"], expect)
    half = (1, 100) + case[2:]
    cfg = rsq.GQEConfig(1, 100, 64, 8, 2, 1, 64, 0)
    ws = torch.empty(rsq.gqe_workspace_bytes(cfg, rsq.GQE_WS_BALANCE), dtype=torch.uint8, device="cuda")
    parts = []
    for r in (slice(0, 100), slice(100, 200)):
        t = [torch.from_numpy(np.ascontiguousarray(a[r])).cuda() for a in (z, idx, mask)]
        c, s = torch.empty(17, dtype=torch.int32, device="cuda"), torch.empty(17, device="cuda")
        rsq.gqe_balance_stats(cfg, *t, c, s, ws)
        parts.append((t, c, s))
    counts, sums = parts[0][1] + parts[1][1], parts[0][2] + parts[1][2]
    for i, (t, _, _) in enumerate(parts):
        dz, loss = torch.empty(100, 16, device="cuda"), torch.empty(3, device="cuda")
        rsq.gqe_balance_loss(cfg, t[0], t[2], counts, sums, 0.1, 0.01, loss, dz)
        assert np.array_equal(dz.double().cpu().numpy(), whole["dz"][100 * i: 100 * i + 100])
        assert np.allclose(loss.cpu().numpy(), whole["loss"], rtol=1e-6)
    assert half[1] == 100


def test_loss_alone_gradient_alone_and_capture(rsq):
    case = CASES["pool_masked"]
    B, T, G, M, k = case[:5]
    z, idx, mask = make(case)
    want = call(rsq, case, z, idx, mask, 0.1, 0.01)
    cfg = rsq.GQEConfig(B, T, 64, G, M, k, 64, 0)
    t = [torch.from_numpy(a).cuda() for a in (z, idx, mask)]
    N = G * M
    counts, sums = torch.empty(N + 1, dtype=torch.int32, device="cuda"), torch.empty(N + 1, device="cuda")
    loss, dz = torch.empty(3, device="cuda"), torch.empty(B * T, N, device="cuda")
    ws = torch.empty(rsq.gqe_workspace_bytes(cfg, rsq.GQE_WS_BALANCE), dtype=torch.uint8, device="cuda")

    def step():
        rsq.gqe_balance_stats(cfg, *t, counts, sums, ws)
        rsq.gqe_balance_loss(cfg, t[0], t[2], counts, sums, 0.1, 0.01, loss, None)
        rsq.gqe_balance_loss(cfg, t[0], t[2], counts, sums, 0.1, 0.01, None, dz)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for x in (counts, sums, loss, dz):
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(loss.double().cpu().numpy(), want["loss"])
    assert np.array_equal(dz.double().cpu().numpy(), want["dz"])


def test_router_logits(rsq):
    # fp32 sums over d_model of exact bf16 x fp32 products: 4 partial sums of
    # d/4 terms, at most (d/4 + 3) * 2^-24 of the absolute sum.
    gen = torch.Generator().manual_seed(4)
    for R, d, G, M in ((1, 64, 2, 2), (50, 1024, 8, 4), (33, 128, 5, 3)):
        x = torch.randn(R, d, generator=gen).to(torch.bfloat16)
        W, b = torch.randn(d, G * M, generator=gen) / d ** 0.5, torch.randn(G * M, generator=gen)
        cfg = rsq.GQEConfig(1, R, d, G, M, 1, 64, 0)
        for bias in (None, b):
            z = torch.empty(R, G * M, device="cuda")
            rsq.gqe_router_logits(cfg, x.cuda(), W.cuda(), None if bias is None else bias.cuda(), z)
            want = x.double() @ W.double() + (0 if bias is None else bias.double())
            size = x.double().abs() @ W.double().abs() + b.double().abs()
            assert ((z.cpu().double() - want).abs() <= (d / 4 + 4) * 2.0 ** -24 * size).all()
