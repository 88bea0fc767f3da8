"""Norm and rotation of queries and keys (gqe_qk_rope, gqe_qk_rope_bwd) against
the fp64 definition.

Tolerances. Forward: one rounding to bf16 (2^-8 of the value) on fp32 arithmetic
whose error is at most 2^-18 of |a| + |b| of the rotated pair: the mean of d_head
squares at most 2^-18 / 2 = 2^-19 of rstd; the hardware's sine and cosine within
half a turn 2^-21.2 (their stated largest error, absolute); the angle, which
reaches fp32 as a fraction of a turn, 2^-25 turns = 2^-22.3 rad; rsqrt and the
products a few 2^-24: together 2^-18.5. Backward (fp32 out): the same relative
error on the terms of dx = rstd (gw - xh mean(gw xh)); the row's sums of up to 64
terms add 64 * 2^-24 = 2^-18 of their absolute sum; 2^-16 of the terms' sizes covers both. Weight
gradients: the terms' 2^-17 and at most 64 sequential fp32 additions (2^-18) at
these sizes, of the sum of absolute terms: 2^-16."""
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


# B, T, G, k, dh, d_rot, norm, weights, adjacent, axes, far, scale
CASES = {
    "one_token": (1, 1, 2, 1, 64, 64, True, True, False, 1, 0, 1.0),
    "decode_batch_far": (7, 1, 8, 1, 64, 64, True, True, False, 1, 1000000, 1.0),
    "odd_dh32": (2, 37, 4, 2, 32, 32, True, True, False, 1, 0, 1.0),
    "adjacent_axes3": (2, 33, 2, 3, 64, 64, True, True, True, 3, 50, 1.0),
    "partial_rot": (1, 65, 2, 1, 64, 24, True, True, False, 2, 9000, 1.0),
    "partial_adjacent_dh32": (3, 5, 1, 2, 32, 8, True, False, True, 1, 77, 1.0),
    "norm_only": (1, 19, 2, 1, 64, 0, True, True, False, 1, 0, 1.0),
    "rotation_only": (1, 50, 2, 2, 64, 64, False, False, False, 1, 200000, 1.0),
    "scaled_axes4": (1, 129, 1, 1, 32, 32, True, True, False, 4, 3000, 1.25),
    "axes4_default_positions": (3, 40, 2, 1, 32, 32, True, True, True, 4, 0, 1.0),
    "dh32_usual": (2, 300, 3, 2, 32, 32, True, True, False, 2, 64, 1.0),
    "long": (1, 2500, 8, 1, 64, 64, True, True, False, 1, 0, 1.0),
    "tiles_of_many_heads": (5, 1200, 8, 2, 64, 64, True, True, False, 1, 0, 1.0),
}


def make(case, seed=5):
    B, T, G, k, dh, d_rot, norm, weights, adjacent, axes, far, scale = case
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    d = {"Q": r(B, G, k, T, dh), "Qs": r(B, T, dh), "K": r(B, G, T, dh) * 3}
    d = {n: t.to(torch.bfloat16) for n, t in d.items()}
    g = {"Q": r(B, G, k, T, dh), "Qs": r(B, T, dh), "K": r(B, G, T, dh)}
    w_q, w_k = (1 + 0.3 * r(dh), 1 + 0.3 * r(dh)) if weights else (None, None)
    pos = torch.randint(0, far, (axes, B * T), generator=gen, dtype=torch.int32) if far else None
    if far:
        pos[0, 0] = far - 1
    inv = 10000.0 ** (-2.0 * torch.arange(d_rot // 2, dtype=torch.float64) / max(d_rot, 1))
    axis = torch.randint(0, axes, (d_rot // 2,), generator=gen, dtype=torch.int32) if axes > 1 else None
    return d, g, w_q, w_k, pos, inv, axis


def cuda(t):
    return None if t is None else t.cuda()


def f64(t):
    return t.double().numpy()


def description(rsq, case, w_q, w_k, pos, inv, axis):
    _, _, _, _, _, d_rot, norm, _, adjacent, axes, _, scale = case
    flags = (rsq.GQE_ROPE_NORM if norm else 0) | (rsq.GQE_ROPE_ADJACENT if adjacent else 0)
    return rsq.GQERope.of(d_rot, cuda(inv), pos=cuda(pos), axis=cuda(axis), w_q=cuda(w_q), w_k=cuda(w_k), eps=1e-5,
                          scale=scale, flags=flags, axes=axes)


def reference(case, d, g, w_q, w_k, pos, inv, axis):
    B, T, _, _, dh, d_rot, norm, weights, adjacent, axes, far, scale = case
    p = np.tile(np.arange(T), (axes, B)) if pos is None else pos.numpy()
    ang = op.rope_angles(p, inv.numpy(), None if axis is None else axis.numpy()).reshape(B, T, -1)
    fwd, bwd, tol, btol, dws, dwt = {}, {}, {}, {}, {}, {}
    for name in ("Q", "Qs", "K"):
        w = np.ones(dh) if not weights else f64(w_k if name == "K" else w_q)
        x, gr = f64(d[name]), f64(g[name])
        fwd[name], bwd[name] = np.empty_like(x), np.empty_like(x)
        dw = np.zeros(dh)
        dwa = np.zeros(dh)
        for b in range(B):
            kw = dict(norm=norm, w=w, eps=1e-5, scale=scale, adjacent=adjacent)
            fwd[name][b] = op.rope(x[b], ang[b], **kw)
            bwd[name][b], part = op.rope_backward(x[b], gr[b], ang[b], **kw)
            if norm:
                dw += part
                xh = op.rope_norm(x[b], 1.0, 1e-5)
                dwa += (2 * scale * np.abs(gr[b]).max(-1, keepdims=True) * np.abs(xh)).reshape(-1, dh).sum(0)
        n = op.rope_norm(x, w, 1e-5) if norm else x
        top = 2 * max(scale, 1.0) * np.abs(n).max(-1, keepdims=True)
        tol[name] = 2.0 ** -8 * np.abs(fwd[name]) + 2.0 ** -18 * top
        gmax = 2 * max(scale, 1.0) * np.abs(gr).max(-1, keepdims=True) * np.abs(w).max()
        if norm:
            rstd = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5)
            btol[name] = 2.0 ** -16 * rstd * gmax * (1 + np.abs(x * rstd).max(-1, keepdims=True)) + np.zeros_like(x)
            key = "w_k" if name == "K" else "w_q"
            dws[key] = dws.get(key, 0) + dw
            dwt[key] = dwt.get(key, 0) + 2.0 ** -16 * dwa
        else:
            btol[name] = 2.0 ** -18 * gmax + np.zeros_like(x)
    return fwd, tol, bwd, btol, dws, dwt


def within(got, want, tol, what):
    e = np.abs(got.double().cpu().numpy().reshape(want.shape) - want)
    assert (e <= tol).all(), f"{what}: worst {np.nanmax(e / tol):.3f} of the tolerance"


@pytest.mark.parametrize("name", list(CASES))
def test_forward_and_backward_match_the_definition(rsq, name):
    case = CASES[name]
    B, T, G, k, dh = case[:5]
    data = make(case)
    d, g = data[0], data[1]
    rope = description(rsq, case, *data[2:])
    fwd, tol, bwd, btol, dws, dwt = reference(case, *data)
    cfg = rsq.GQEConfig(B, T, 64, G, max(k, 2), k, dh, 0)
    dd = {n: t.cuda() for n, t in d.items()}
    out = {n: torch.full_like(t, float("nan")) for n, t in dd.items()}
    rsq.gqe_qk_rope(cfg, rope, dd["Q"], dd["Qs"], dd["K"], None, out["Q"], out["Qs"], out["K"])
    for n in out:
        within(out[n], fwd[n], tol[n], f"forward {n}")
        assert torch.equal(dd[n].cpu(), d[n])
    # In place, and one operand at a time: the same bits.
    for n in out:
        y = dd[n].clone()
        args = [y if m == n else None for m in ("Q", "Qs", "K")]
        rsq.gqe_qk_rope(cfg, rope, *args, None, *args)
        assert torch.equal(y, out[n]), n

    gg = {n: t.cuda() for n, t in g.items()}
    go = {n: torch.full_like(t, float("nan")) for n, t in gg.items()}
    ws = torch.empty(rsq.gqe_workspace_bytes(cfg, rsq.GQE_WS_QK_ROPE), dtype=torch.uint8, device="cuda")
    norm = case[6]
    dw = {w: torch.full((dh,), float("nan"), device="cuda") for w in ("w_q", "w_k")} if norm else {"w_q": None, "w_k": None}
    rsq.gqe_qk_rope_bwd(cfg, rope, dd["Q"], dd["Qs"], dd["K"], None, gg["Q"], gg["Qs"], gg["K"], go["Q"], go["Qs"],
                        go["K"], dw["w_q"], dw["w_k"], ws)
    for n in go:
        within(go[n], bwd[n], btol[n], f"backward {n}")
    for w in dws:
        within(dw[w], dws[w], dwt[w], f"d{w}")
    # In place over the gradients, twice: the same bits.
    for _ in range(2):
        gi = {n: t.clone() for n, t in gg.items()}
        dw2 = {w: None if t is None else torch.empty_like(t) for w, t in dw.items()}
        rsq.gqe_qk_rope_bwd(cfg, rope, dd["Q"], dd["Qs"], dd["K"], None, gi["Q"], gi["Qs"], gi["K"], gi["Q"], gi["Qs"],
                            gi["K"], dw2["w_q"], dw2["w_k"], ws)
        assert all(torch.equal(gi[n], go[n]) for n in go)
        assert all(t is None or torch.equal(dw2[w], t) for w, t in dw.items())
    assert rsq.gqe_read_status() == 0


def test_token_list_order(rsq):
    # Rows in list order (slot_pos a permutation) give the slot-major results.
    case = (2, 21, 3, 2, 64, 64, True, True, False, 1, 400, 1.0)
    B, T, G, k, dh = case[:5]
    data = make(case)
    d, g = data[0], data[1]
    rope = description(rsq, case, *data[2:])
    cfg = rsq.GQEConfig(B, T, 64, G, 3, k, dh, 0)
    perm = torch.randperm(B * T * G * k, generator=torch.Generator().manual_seed(3)).to(torch.int32)
    sp = perm.view(B * T, G, k).cuda()

    def listed(t):  # [B, G, k, T, dh] -> list order
        rows = t.permute(0, 3, 1, 2, 4).reshape(-1, dh)
        out = torch.empty_like(rows)
        out[perm.long().cuda()] = rows
        return out

    Q, gq = d["Q"].cuda(), g["Q"].cuda()
    want, got = torch.empty_like(Q), torch.empty(B * T * G * k, dh, dtype=Q.dtype, device="cuda")
    rsq.gqe_qk_rope(cfg, rope, Q, None, None, None, want, None, None)
    rsq.gqe_qk_rope(cfg, rope, listed(Q), None, None, sp, got, None, None)
    assert torch.equal(got, listed(want))
    ws = torch.empty(rsq.gqe_workspace_bytes(cfg, rsq.GQE_WS_QK_ROPE), dtype=torch.uint8, device="cuda")
    dq, dql = torch.empty_like(gq), torch.empty(B * T * G * k, dh, device="cuda")
    dw, dwl = torch.empty(dh, device="cuda"), torch.empty(dh, device="cuda")
    rsq.gqe_qk_rope_bwd(cfg, rope, Q, None, None, None, gq, None, None, dq, None, None, dw, None, ws)
    rsq.gqe_qk_rope_bwd(cfg, rope, listed(Q), None, None, sp, listed(gq), None, None, dql, None, None, dwl, None, ws)
    assert torch.equal(dql, listed(dq)) and torch.equal(dw, dwl)
    assert rsq.gqe_read_status() == 0
    # Entries outside the list: their rows are left out and the status says so.
    bad = sp.clone()
    bad.view(-1)[0], bad.view(-1)[7] = -1, B * T * G * k
    left = torch.zeros_like(got)
    rsq.gqe_qk_rope(cfg, rope, listed(Q), None, None, bad, left, None, None)
    torch.cuda.synchronize()
    gone = perm.view(-1)[[0, 7]].long().cuda()
    keep = torch.ones(len(perm), dtype=torch.bool, device="cuda")
    keep[gone] = False
    assert torch.equal(left[keep], got[keep]) and (left[gone] == 0).all()
    assert rsq.gqe_read_status() == rsq.GQE_ERR_DEVICE_CHECK


def test_axis_outside_is_recorded(rsq):
    case = (1, 4, 1, 1, 32, 32, False, False, False, 2, 30, 1.0)
    d, _, _, _, pos, inv, axis = make(case)
    cfg = rsq.GQEConfig(1, 4, 64, 1, 1, 1, 32, 0)
    bad, zero = axis.clone(), axis.clone()
    bad[3], zero[3] = 2, 0
    bad[5], zero[5] = -1, 0
    K, a, b = d["K"].cuda(), d["K"].cuda(), d["K"].cuda()
    rsq.gqe_qk_rope(cfg, description(rsq, case, None, None, pos, inv, bad), None, None, K, None, None, None, a)
    torch.cuda.synchronize()
    assert rsq.gqe_read_status() == rsq.GQE_ERR_DEVICE_CHECK
    rsq.gqe_qk_rope(cfg, description(rsq, case, None, None, pos, inv, zero), None, None, K, None, None, None, b)
    assert torch.equal(a, b) and rsq.gqe_read_status() == 0


def test_rows_of_zeros_and_of_large_values(rsq):
    # Zero rows norm to zero (eps > 0); a NaN stays in its row.
    cfg = rsq.GQEConfig(1, 4, 64, 1, 1, 1, 64, 0)
    K = torch.randn(1, 1, 4, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    K[0, 0, 1] = 0
    K[0, 0, 2] *= 2.0 ** 60
    K[0, 0, 3, 5] = float("nan")
    inv = 10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)
    rope = rsq.GQERope.of(64, inv.cuda(), eps=1e-6, flags=rsq.GQE_ROPE_NORM)
    y = torch.empty_like(K, device="cuda")
    rsq.gqe_qk_rope(cfg, rope, None, None, K.cuda(), None, None, None, y)
    y = y.cpu()[0, 0].double()
    assert (y[1] == 0).all() and torch.isnan(y[3]).all() and torch.isfinite(y[:3]).all()
    assert abs(float((y[2] ** 2).mean()) - 1) < 2 ** -6


def test_eps_of_zero_and_a_partial_tile(rsq):
    # Tokens behind the last one add nothing to the weights' gradients, although
    # a row of zeros has no norm with eps = 0.
    cfg = rsq.GQEConfig(1, 5, 64, 2, 1, 1, 64, 0)
    gen = torch.Generator().manual_seed(6)
    K, g = torch.randn(1, 2, 5, 64, generator=gen).to(torch.bfloat16), torch.randn(1, 2, 5, 64, generator=gen)
    rope = rsq.GQERope.of(0, torch.empty(0, dtype=torch.float64, device="cuda"), eps=0.0, flags=rsq.GQE_ROPE_NORM)
    ws = torch.empty(rsq.gqe_workspace_bytes(cfg, rsq.GQE_WS_QK_ROPE), dtype=torch.uint8, device="cuda")
    dk, dw = torch.empty(1, 2, 5, 64, device="cuda"), torch.empty(64, device="cuda")
    rsq.gqe_qk_rope_bwd(cfg, rope, None, None, K.cuda(), None, None, None, g.cuda(), None, None, dk, None, dw, ws)
    dx, dwr = op.rope_backward(f64(K), f64(g), np.zeros((5, 0)), norm=True)
    assert np.abs(dk.cpu().double().numpy() - dx).max() <= 2.0 ** -16 * np.abs(dx).max()
    size = np.abs(f64(g) * op.rope_norm(f64(K), 1.0, 0.0)).reshape(-1, 64).sum(0)
    assert (np.abs(dw.cpu().double().numpy() - dwr) <= 2.0 ** -16 * size).all()


def test_passed_elements_do_not_meet_their_neighbours(rsq):
    # Without the norm an infinity stays in its element (or its rotated pair).
    cfg = rsq.GQEConfig(1, 3, 64, 1, 1, 1, 64, 0)
    K = torch.randn(1, 1, 3, 64, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16)
    K[..., 40] = float("inf")
    K[..., 63] = float("nan")
    for flags in (0, rsq.GQE_ROPE_ADJACENT):
        rope = rsq.GQERope.of(16, torch.ones(8, dtype=torch.float64, device="cuda"), flags=flags)
        y = torch.empty_like(K, device="cuda")
        rsq.gqe_qk_rope(cfg, rope, None, None, K.cuda(), None, None, None, y)
        y = y.cpu()
        keep = [i for i in range(16, 64) if i != 63]
        assert torch.equal(y[..., keep], K[..., keep]) and torch.isfinite(y[..., :16].float()).all()


def test_streams_and_graph_capture(rsq):
    case = CASES["odd_dh32"]
    B, T, G, k, dh = case[:5]
    data = make(case)
    d, g = {n: t.cuda() for n, t in data[0].items()}, {n: t.cuda() for n, t in data[1].items()}
    rope = description(rsq, case, *data[2:])
    cfg = rsq.GQEConfig(B, T, 64, G, 2, k, dh, 0)
    ws = torch.empty(rsq.gqe_workspace_bytes(cfg, rsq.GQE_WS_QK_ROPE), dtype=torch.uint8, device="cuda")

    def outputs():
        return ([torch.empty_like(d[n]) for n in d], [torch.empty_like(g[n]) for n in g],
                [torch.empty(dh, device="cuda") for _ in range(2)])

    def both(o, stream=None):
        rsq.gqe_qk_rope(cfg, rope, *d.values(), None, *o[0], stream=stream)
        rsq.gqe_qk_rope_bwd(cfg, rope, *d.values(), None, *g.values(), *o[1], *o[2], ws, stream=stream)

    want, other, captured = outputs(), outputs(), outputs()
    both(want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    both(other, side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(captured)
    for n in d:
        d[n].neg_()  # the replay sees the inputs' present values
    graph.replay()
    for n in d:
        d[n].neg_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, other, captured):
        assert all(torch.equal(x, y) and torch.equal(x, z) for x, y, z in zip(a, b, c))


def test_binding_checks_arguments(rsq):
    inv = torch.ones(16, dtype=torch.float64, device="cuda")
    cfg = rsq.GQEConfig(1, 4, 64, 1, 1, 1, 32, 0)
    K = torch.zeros(1, 1, 4, 32, dtype=torch.bfloat16, device="cuda")
    rope = rsq.GQERope.of(32, inv)
    for bad in (K.float(), K[:, :, :3].contiguous(), K.transpose(2, 3)):
        with pytest.raises(ValueError):
            rsq.gqe_qk_rope(cfg, rope, None, None, bad, None, None, None, K)
    with pytest.raises(ValueError):
        rsq.GQERope.of(32, inv.float())
    with pytest.raises(ValueError):
        rsq.gqe_qk_rope(cfg, rsq.GQERope.of(32, inv, pos=torch.zeros(5, dtype=torch.int32, device="cuda")), None, None, K,
                        None, None, None, K)
    with pytest.raises(rsq.GQEError):
        rsq.gqe_qk_rope(cfg, rope, None, None, None, None, None, None, None)
