"""The layer's calls with positions, balance loss and 4-bit cache: bit for bit
the run of their steps, and against an fp64 layer (torch, CPU, automatic
differentiation) with the GPU's selection.

Tolerances: those of the layer's other tests -- y within 2e-2 max and 2e-3 mean of
the fp64 layer (scaled by 2 rms(y) where that passes 1: a token that sees few keys
has outputs of order 1), gradients within 3e-2 of the largest and 1e-2 of the mean
magnitude: the bf16 roundings on the path (Q, K, V, P, slots, y, and the operand
copies of the backward) are the layer's, with one more of the rotated Q and K
(2^-8).

The bias gradient is a sum over the rows of dz with signs of its own, and may come
out small against its terms' errors, which it inherits: db_r[e] = sum_r sum_q
J[e, q] dw[r, q] with |J[e, q]| <= 2 p_e / sum(selected p) (quotient rule, then the
group's softmax Jacobian) and dw[r, q] = sum_{c, d} o[r, q, c] dy[r, d] W_o[c, d].
Each term carries up to 4 independent bf16 roundings (of the slot, of dy, and of P
and of Q, K, V inside o), each uniform within half a step of 2^-8: a standard
deviation of at most 2^-8/sqrt(3) of the term, so that of the sum is at most
sqrt(4) 2^-8/sqrt(3) sqrt(sum of squared terms). Six of those bound db_r."""
import math

import numpy as np
import pytest
import torch

import synth
from synth import LayerShape
from gpu_common import bf16_dev, device_inputs, n_slots, run_steps

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rsq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import routed_sparse_query_b200 as m
    return m


def close(got, want, what, max_abs=2e-2, mean_abs=2e-3):
    want = want.detach()
    s = max(1.0, 2.0 * float(want.square().mean().sqrt()))
    e = (got.double().cpu().reshape(want.shape) - want).abs()
    assert e.max() <= max_abs * s and e.mean() <= mean_abs * s, f"{what}: {e.max():.2e} max, {e.mean():.2e} mean"


def close_grad(got, want, what):
    e = (got.double().cpu().reshape(want.shape) - want).abs()
    assert e.max() <= 3e-2 * want.abs().max(), f"{what}: max {e.max():.3e} of {want.abs().max():.3e}"
    assert e.mean() <= 1e-2 * want.abs().mean(), f"{what}: mean {e.mean():.3e} of {want.abs().mean():.3e}"


class Positions:
    """One description on both sides."""

    def __init__(self, rsq, shape, tokens, axes=1, adjacent=False, norm=True, far=0, seed=3):
        gen = torch.Generator().manual_seed(seed)
        dh = shape.d_head
        self.norm, self.adjacent, self.dh = norm, adjacent, dh
        self.inv = 10000.0 ** (-2.0 * torch.arange(dh // 2, dtype=torch.float64) / dh)
        self.w_q, self.w_k = (1 + 0.2 * torch.randn(dh, generator=gen) for _ in range(2))
        self.pos = torch.randint(0, far, (axes, tokens), generator=gen, dtype=torch.int32) if far else None
        self.axis = torch.randint(0, axes, (dh // 2,), generator=gen, dtype=torch.int32) if axes > 1 else None
        c = lambda t: None if t is None else t.cuda()  # noqa: E731
        self.rope = rsq.GQERope.of(dh, self.inv.cuda(), pos=c(self.pos), axis=c(self.axis),
                                   w_q=self.w_q.cuda() if norm else None, w_k=self.w_k.cuda() if norm else None, eps=1e-5,
                                   flags=(rsq.GQE_ROPE_NORM if norm else 0) | (rsq.GQE_ROPE_ADJACENT if adjacent else 0))

    def apply(self, x, w, default_pos):
        """x [tokens, heads, dh] fp64 (tensors with gradients), w fp64 [dh]."""
        p = default_pos[None] if self.pos is None else self.pos
        a = torch.zeros(self.dh // 2, dtype=torch.long) if self.axis is None else self.axis.long()
        th = (p[a].T.double() * self.inv)[:, None]
        if self.norm:
            x = w * x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-5)
        h = self.dh // 2
        u, v = (x[..., 0::2], x[..., 1::2]) if self.adjacent else (x[..., :h], x[..., h:])
        y = (u * th.cos() - v * th.sin(), u * th.sin() + v * th.cos())
        return torch.stack(y, -1).flatten(-2) if self.adjacent else torch.cat(y, -1)


def leaves(inp):
    f = lambda a: torch.from_numpy(synth.bf16_to_f64(a))  # noqa: E731
    p = {"x": f(inp.x), "W_r": torch.from_numpy(inp.W_r).double(), "W_q": f(inp.W_q), "W_qs": f(inp.W_qs),
         "W_k": f(inp.W_k), "W_v": f(inp.W_v), "W_o": f(inp.W_o)}
    p["b_r"] = torch.zeros(p["W_r"].shape[1], dtype=torch.float64) if inp.b_r is None else torch.from_numpy(inp.b_r).double()
    return {n: t.reshape(inp.x.shape) if n == "x" else t for n, t in p.items()}


def plain_layer(s, p, idx, pos, w_qn, w_kn):
    """y and logits of the fp64 layer with the selection idx [R, G, k]."""
    B, T, G, M, k, dh = s.B, s.T, s.G, s.M, s.k, s.d_head
    R = B * T
    x = p["x"].reshape(R, -1)
    z = x @ p["W_r"] + p["b_r"]
    prob = torch.softmax(z.view(R, G, M), -1)
    psel = prob.gather(-1, idx)
    w = psel / psel.sum((1, 2), keepdim=True)
    t = torch.arange(T, dtype=torch.int32).repeat(B)
    e = (torch.arange(G)[None, :, None] * M + idx).reshape(R, G * k)
    q = (x @ p["W_q"]).view(R, G * M, dh).gather(1, e[..., None].expand(-1, -1, dh))
    qs, K, V = (x @ p["W_qs"]).view(R, 1, dh), (x @ p["W_k"]).view(R, G, dh), (x @ p["W_v"]).view(R, G, dh)
    if pos is not None:
        q, qs, K = pos.apply(q, w_qn, t), pos.apply(qs, w_qn, t), pos.apply(K, w_kn, t)
    heads = torch.cat([q, qs], 1).view(B, T, G * k + 1, dh).transpose(1, 2)
    group = torch.tensor([g for g in range(G) for _ in range(k)] + [0])
    Kh, Vh = (u.view(B, T, G, dh).transpose(1, 2)[:, group] for u in (K, V))
    sc = heads @ Kh.transpose(2, 3) / math.sqrt(dh)
    sc = sc.masked_fill(torch.ones(T, T).triu(1).bool(), -math.inf)
    o = (torch.softmax(sc, -1) @ Vh).transpose(1, 2).reshape(R, G * k + 1, dh)
    weighted = (w.reshape(R, G * k, 1) * o[:, : G * k]).sum(1, keepdim=True)
    return torch.cat([o, weighted], 1).reshape(R, -1) @ p["W_o"], z, o, prob.reshape(R, -1), psel.sum((1, 2))


def bias_tolerance(s, p, dy, o, prob, total):
    with torch.no_grad():
        gk, dh = s.G * s.k, s.d_head
        Ww = p["W_o"][(gk + 1) * dh:]                                    # the weighted slot's rows
        t2 = (o[:, :gk].square() * (dy.double().square() @ Ww.T.square())[:, None]).sum((1, 2))  # [R]
        j = 2 * prob / total[:, None]
        return 6 * 2 * 2.0 ** -8 / math.sqrt(3) * (j.square() * t2[:, None]).sum(0).sqrt()


def plain_balance(s, z, idx, mask, cb, cz):
    G, M, k = s.G, s.M, s.k
    rows = torch.arange(z.shape[0]) if mask is None else mask.nonzero().view(-1)
    zz = z[rows].view(-1, G, M)
    f = torch.nn.functional.one_hot(idx[rows], M).sum((0, 2)).double() / (k * len(rows))
    return cb * M / G * (f * torch.softmax(zz, -1).mean(0)).sum() + cz * torch.logsumexp(zz, -1).square().mean()


SHAPES = {
    "b2_t70": LayerShape(B=2, T=70, d_model=128, G=2, M=2, k=1, d_head=64),
    "m3_k2_dh32": LayerShape(B=1, T=130, d_model=128, G=2, M=3, k=2, d_head=32),
    "one_token": LayerShape(B=3, T=1, d_model=64, G=2, M=2, k=1, d_head=64),
    "g4_t300": LayerShape(B=1, T=300, d_model=256, G=4, M=2, k=1, d_head=64),
}
KINDS = {"plain": {}, "axes_adjacent_far": dict(axes=3, adjacent=True, far=40000), "no_norm": dict(norm=False)}


def weights(d):
    return [d[n] for n in ("W_r", "b_r", "W_q", "W_qs", "W_k", "W_v", "W_o")]


def ws_of(rsq, cfg, kind):
    return torch.full((rsq.gqe_workspace_bytes(cfg, kind),), 255, dtype=torch.uint8, device="cuda")


def layer_fwd(rsq, s, d, rope, flags=0):
    cfg = rsq.GQEConfig.of(s, flags)
    ws, y = ws_of(rsq, cfg, rsq.GQE_WS_LAYER), torch.empty(s.R, s.d_model, dtype=torch.bfloat16, device="cuda")
    rsq.gqe_layer_fwd_rope(cfg, rope, d["x"], *weights(d), y, ws)
    return y, ws, cfg


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("name", list(SHAPES))
def test_layer_with_positions(rsq, name, kind):
    s = SHAPES[name]
    inp = synth.make_layer_inputs(s, seed=8)
    d = device_inputs(inp)
    pos = Positions(rsq, s, s.R, **KINDS[kind])
    y, ws, cfg = layer_fwd(rsq, s, d, pos.rope)
    idx = rsq.workspace_view(ws, cfg, rsq.GQE_WS_LAYER, "idx", torch.int32, (s.R, s.G, s.k)).cpu().long()
    want = plain_layer(s, leaves(inp), idx, pos, pos.w_q.double(), pos.w_k.double())[0]
    close(y, want, "y")
    # The steps: the same bits; token-list order: the same values up to the attention's tiling.
    B, T, G, k, dh = s.B, s.T, s.G, s.k, s.d_head
    view = lambda n, *shape: rsq.workspace_view(ws, cfg, rsq.GQE_WS_LAYER, n, torch.bfloat16, shape)  # noqa: E731
    o = run_steps(rsq, s, d)
    rsq.gqe_qk_rope(cfg, pos.rope, o["Qv"], o["Qs"], o["K"], None, o["Qv"], o["Qs"], o["K"])
    assert torch.equal(o["Qv"], view("Qv", B, G, k, T, dh)) and torch.equal(o["K"], view("K", B, G, T, dh))
    assert torch.equal(o["Qs"], view("Qs", B, T, dh))
    slots = torch.zeros(s.R, n_slots(s) * dh, dtype=torch.bfloat16, device="cuda")
    rsq.gqe_attention_fwd(cfg, o["Qv"], o["Qs"], o["K"], o["V"], slots, ws_of(rsq, cfg, rsq.GQE_WS_ATTENTION))
    y2 = torch.empty_like(y)
    rsq.gqe_output_proj(cfg, slots, o["omega"], d["W_o"], y2)
    assert torch.equal(y, y2)
    ye, _, _ = layer_fwd(rsq, s, d, pos.rope, rsq.GQE_FLAG_EXPERT_MAJOR)
    close(ye, want, "y, token-list order")
    assert rsq.gqe_read_status() == 0


def test_output_constructions_with_positions(rsq):
    # The constructions without a shared head rotate what is there.
    s = SHAPES["b2_t70"]
    inp = synth.make_layer_inputs(s, seed=8)
    d = device_inputs(inp)
    pos = Positions(rsq, s, s.R)
    cfg = rsq.GQEConfig.of(s, rsq.GQE_FLAG_OUT_HARD)
    d["W_o"] = d["W_o"][: s.k * s.G * s.d_head].contiguous()
    ws, y = ws_of(rsq, cfg, rsq.GQE_WS_LAYER), torch.empty(s.R, s.d_model, dtype=torch.bfloat16, device="cuda")
    rsq.gqe_layer_fwd_rope(cfg, pos.rope, d["x"], *weights(d), y, ws)
    _, ws0, c0 = layer_fwd(rsq, s, device_inputs(inp), pos.rope)
    gk = s.G * s.k * s.d_head
    a = rsq.workspace_view(ws, cfg, rsq.GQE_WS_LAYER, "slots", torch.bfloat16, (s.R, gk))
    b = rsq.workspace_view(ws0, c0, rsq.GQE_WS_LAYER, "slots", torch.bfloat16, (s.R, gk + 2 * s.d_head))
    assert torch.equal(a, b[:, :gk])


@pytest.mark.parametrize("kind", ["none", "plain", "axes_adjacent_far", "no_norm"])
@pytest.mark.parametrize("bal", [None, "all", "masked"])
@pytest.mark.parametrize("name", ["b2_t70", "m3_k2_dh32", "g4_t300"])
def test_backward_with_positions_and_balance(rsq, name, kind, bal):
    s = SHAPES[name]
    inp = synth.make_layer_inputs(s, seed=31)
    d = device_inputs(inp)
    pos = None if kind == "none" else Positions(rsq, s, s.R, **KINDS[kind])
    cfg, R, dh, dm, N = rsq.GQEConfig.of(s), s.R, s.d_head, s.d_model, s.N
    dy = torch.randn(R, dm, generator=torch.Generator().manual_seed(5))
    # The balance loss alone is far smaller than the sum of dy * y: weigh it up.
    cb, cz = 300.0, 30.0
    mask = (torch.arange(R) % 3 != 1).to(torch.uint8) if bal == "masked" else None
    f = lambda *shape: torch.full(shape, float("nan"), device="cuda")  # noqa: E731
    out = {"x": f(R, dm), "W_r": f(dm, N), "b_r": f(N), "W_q": f(dm, N * dh), "W_qs": f(dm, dh), "W_k": f(dm, s.G * dh),
           "W_v": f(dm, s.G * dh), "W_o": f((s.k * s.G + 2) * dh, dm)}
    norm = pos is not None and pos.norm
    dwn = [f(dh) if norm else None for _ in range(2)]
    counts, sums, loss = torch.empty(N + 1, dtype=torch.int32, device="cuda"), f(N + 1), f(3)
    balance = None if bal is None else rsq.GQEBalance.of(counts, sums, loss, None if mask is None else mask.cuda(), cb, cz)
    ws = ws_of(rsq, cfg, rsq.GQE_WS_BACKWARD_AUX)

    def call():
        rsq.gqe_layer_bwd_aux(cfg, None if pos is None else pos.rope, balance, d["x"], *weights(d), dy.cuda(),
                              *out.values(), *dwn, ws)

    call()
    idx = rsq.workspace_view(ws, cfg, rsq.GQE_WS_LAYER, "idx", torch.int32, (R, s.G, s.k)).cpu().long()
    p = {n: t.requires_grad_(True) for n, t in leaves(inp).items()}
    wn = [pos.w_q.double().requires_grad_(True), pos.w_k.double().requires_grad_(True)] if norm else [None, None]
    y, z, o, prob, psel = plain_layer(s, p, idx, pos, *wn)
    total = (y * dy.double()).sum()
    if bal is not None:
        lb = plain_balance(s, z, idx, mask, cb, cz)
        total = total + lb
        assert abs(float(loss[0]) - float(lb)) <= 1e-3 * abs(float(lb))  # the GPU's logits are fp32 sums
    want = torch.autograd.grad(total, list(p.values()) + [w for w in wn if w is not None])
    for n, g in zip(p, want):
        if n == "b_r":
            assert ((out[n].double().cpu() - g).abs() <= bias_tolerance(s, p, dy, o, prob, psel)).all(), n
        else:
            close_grad(out[n], g, n)
    for n, got, g in zip(("w_q", "w_k"), dwn if norm else [], want[len(p):]):
        close_grad(got, g, n)
    first = [t.clone() for t in out.values()]
    call()
    assert all(torch.equal(a, b) for a, b in zip(first, out.values()))
    assert rsq.gqe_read_status() == 0
    if pos is None and bal is None:  # nothing added: the plain backward's bits
        ref = [torch.empty_like(t) for t in out.values()]
        rsq.gqe_layer_bwd(cfg, d["x"], *weights(d), dy.cuda(), *ref, ws_of(rsq, cfg, rsq.GQE_WS_BACKWARD))
        assert all(torch.equal(a, b) for a, b in zip(first, ref))


def test_decode_with_positions_continues_a_prefill(rsq):
    # The last token's row of a prefill with positions, decoded against the
    # prefill's rotated keys.
    for s in (SHAPES["b2_t70"], SHAPES["one_token"], LayerShape(B=2, T=257, d_model=128, G=2, M=3, k=2, d_head=32)):
        inp = synth.make_layer_inputs(s, seed=8)
        d = device_inputs(inp)
        pos = Positions(rsq, s, s.R)
        y, ws, cfg = layer_fwd(rsq, s, d, pos.rope)
        B, T, G, dh = s.B, s.T, s.G, s.d_head
        cap = T + 5
        caches = []
        for n in ("K", "V"):
            full = rsq.workspace_view(ws, cfg, rsq.GQE_WS_LAYER, n, torch.bfloat16, (B, G, T, dh))
            c = torch.zeros(B, G, cap, dh, dtype=torch.bfloat16, device="cuda")
            c[:, :, : T - 1] = full[:, :, : T - 1]
            caches.append((c, full))
        x = d["x"].view(B, T, -1)[:, T - 1].contiguous()
        yd = torch.empty(B, s.d_model, dtype=torch.bfloat16, device="cuda")
        wd = ws_of(rsq, cfg, rsq.GQE_WS_DECODE)
        rsq.gqe_decode_step_rope(cfg, pos.rope, x, *weights(d), caches[0][0], caches[1][0], yd, wd)
        for c, full in caches:
            e = (c[:, :, T - 1].float() - full[:, :, T - 1].float()).abs()
            assert (e <= 2.0 ** -6 * full[:, :, T - 1].float().abs() + 2.0 ** -6).all()
            assert (c[:, :, T:] == 0).all() and torch.equal(c[:, :, : T - 1], full[:, :, : T - 1])
        close(yd, y.double().cpu().view(B, T, -1)[:, T - 1], "decoded y")
        assert rsq.gqe_read_status() == 0


def kv4(rsq, B, G, cap, dh):
    t = [torch.zeros(B, G, cap, dh // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
    t.append(torch.zeros(B, G, cap, 4, dtype=torch.bfloat16, device="cuda"))
    return t, rsq.GQEKv4.of(*t)


@pytest.mark.parametrize("with_rope", [True, False])
def test_serving_over_the_4_bit_cache(rsq, with_rope):
    """Prefill with positions, its keys and values into the 4-bit cache, then
    captured decode steps of a ragged batch with an idle sequence: each the
    same bits as its steps, and y against the stored values in fp64."""
    s = LayerShape(B=4, T=40, d_model=128, G=2, M=3, k=2, d_head=64)
    inp = synth.make_layer_inputs(s, seed=8)
    d = device_inputs(inp)
    B, T, G, M, k, dh = s.B, s.T, s.G, s.M, s.k, s.d_head
    most = 64
    pos = Positions(rsq, s, s.R)
    if with_rope:
        _, ws, cfg = layer_fwd(rsq, s, d, pos.rope)
        Kp, Vp = (rsq.workspace_view(ws, cfg, rsq.GQE_WS_LAYER, n, torch.bfloat16, (B, G, T, dh)) for n in ("K", "V"))
    else:
        cfg = rsq.GQEConfig.of(s)
        Kp, Vp = (torch.empty(B, G, T, dh, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        rsq.gqe_kv_proj(cfg, d["x"], d["W_k"], d["W_v"], Kp, Vp)
    n0 = torch.tensor([40, 7, -1, 0], dtype=torch.int32, device="cuda")
    t, cache = kv4(rsq, B, G, most, dh)
    rsq.gqe_kv4_append(cfg, Kp, Vp, None, n0, cache)
    shadow, c2 = kv4(rsq, B, G, most, dh)
    for a, b in zip(shadow, t):
        a.copy_(b)
    step_cfg, one = rsq.GQEConfig(B, most, s.d_model, G, M, k, dh, 0), rsq.GQEConfig(B, 1, s.d_model, G, M, k, dh, 0)
    lens = n0.clone()
    xn = torch.empty(B, s.d_model, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(xn)
    wd = ws_of(rsq, step_cfg, rsq.GQE_WS_DECODE_KV4)
    rope = pos.rope if with_rope else None

    def step():
        rsq.gqe_decode_step_kv4(step_cfg, rope, xn, *weights(d), cache, lens, y, wd)

    gen = torch.Generator().manual_seed(3)
    xs = [torch.randn(B, s.d_model, generator=gen).to(torch.bfloat16).cuda() for _ in range(5)]
    xn.copy_(xs[0])
    before = [a.clone() for a in t]
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for a, b in zip(t, before):
        a.copy_(b)
    wsd, wsk = ws_of(rsq, one, rsq.GQE_WS_DISPATCH), ws_of(rsq, step_cfg, rsq.GQE_WS_KV4)
    p = leaves(inp)
    for x in xs:
        xn.copy_(x)
        graph.replay()
        # The steps, on the shadow cache.
        e = lambda *shape, dt=torch.bfloat16: torch.empty(*shape, dtype=dt, device="cuda")  # noqa: E731
        i32 = dict(dt=torch.int32)
        idx, r, om = e(B, G, k, **i32), e(B, G, k, dt=torch.float32), e(B, G, k, dt=torch.float32)
        rsq.gqe_router_topk(one, x, d["W_r"], d["b_r"], idx, r, om)
        Q, Qs, K, V = e(B, G, k, 1, dh), e(B, 1, dh), e(B, G, 1, dh), e(B, G, 1, dh)
        rsq.gqe_dispatch(one, idx, x, d["W_q"], d["W_qs"], e(G * M * B, **i32), e(G * M * B + 1, **i32), e(k * G * B, **i32),
                         e(B, G, k, **i32), Q, Qs, wsd)
        rsq.gqe_kv_proj(one, x, d["W_k"], d["W_v"], K, V)
        if with_rope:
            at = rsq.GQERope.of(dh, pos.inv.cuda(), pos=lens.clamp(min=0).view(1, B).contiguous(), w_q=pos.w_q.cuda(),
                                w_k=pos.w_k.cuda(), eps=1e-5, flags=rsq.GQE_ROPE_NORM)
            rsq.gqe_qk_rope(one, at, Q, Qs, K, None, Q, Qs, K)
        rsq.gqe_kv4_append(one, K, V, lens, None, c2)
        slots = e(B, (G * k + 2) * dh)
        rsq.gqe_kv4_attention(step_cfg, Q, Qs, c2, lens + 1, slots, wsk)
        y2 = e(B, s.d_model)
        rsq.gqe_output_proj(one, slots, om, d["W_o"], y2)
        assert torch.equal(y, y2)
        assert all(torch.equal(a, b) for a, b in zip(t, shadow))
        # fp64 on the stored keys and values.
        Kd, Vd = e(B, G, most, dh), e(B, G, most, dh)
        rsq.gqe_kv4_read(rsq.GQEConfig(B, most, s.d_model, G, M, k, dh, 0), cache, None, None, Kd, Vd)
        Kd, Vd, xd, ix = Kd.double().cpu(), Vd.double().cpu(), x.double().cpu(), idx.cpu().long()
        prob = torch.softmax((xd @ p["W_r"] + p["b_r"]).view(B, G, M), -1).gather(-1, ix)
        w = prob / prob.sum((1, 2), keepdim=True)
        ex = (torch.arange(G)[None, :, None] * M + ix).reshape(B, G * k)
        q = (xd @ p["W_q"]).view(B, G * M, dh).gather(1, ex[..., None].expand(-1, -1, dh))
        q = torch.cat([q, (xd @ p["W_qs"]).view(B, 1, dh)], 1)
        if with_rope:
            q = pos_at(pos, q, lens.cpu().clamp(min=0))
        want = torch.zeros(B, s.d_model, dtype=torch.float64)
        for b in range(B):
            n = int(lens[b]) + 1
            if n == 0:
                continue
            o = []
            for h in range(G * k + 1):
                g = h // k if h < G * k else 0
                pr = torch.softmax(Kd[b, g, :n] @ q[b, h] / math.sqrt(dh), 0)
                o.append(pr @ Vd[b, g, :n])
            o.append(sum(w[b].view(-1)[h] * o[h] for h in range(G * k)))
            want[b] = torch.cat(o) @ p["W_o"]
        close(y, want, "y over the 4-bit cache")
        assert (y[2] == 0).all()
        lens.add_((lens >= 0).to(torch.int32))
    assert rsq.gqe_read_status() == 0


def pos_at(pos, x, at):
    th = (at.double()[:, None] * pos.inv)[:, None]
    x = pos.w_q.double() * x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-5)
    h = pos.dh // 2
    u, v = x[..., :h], x[..., h:]
    return torch.cat([u * th.cos() - v * th.sin(), u * th.sin() + v * th.cos()], -1)


def test_captured_training_step(rsq):
    # Forward with positions and backward with both extras, captured on another
    # stream (the layer's side stream joins the capture) and replayed on new
    # inputs, with a workspace declared clean.
    s = SHAPES["b2_t70"]
    d = device_inputs(synth.make_layer_inputs(s, seed=8))
    pos = Positions(rsq, s, s.R, axes=3, far=500)
    cfg = rsq.GQEConfig.of(s, rsq.GQE_FLAG_WS_CLEAN)
    R, N, dh, dm = s.R, s.N, s.d_head, s.d_model
    f = lambda *shape: torch.zeros(shape, device="cuda")  # noqa: E731
    grads = [f(R, dm), f(dm, N), f(N), f(dm, N * dh), f(dm, dh), f(dm, s.G * dh), f(dm, s.G * dh),
             f((s.k * s.G + 2) * dh, dm), f(dh), f(dh)]
    counts, sums, loss = torch.zeros(N + 1, dtype=torch.int32, device="cuda"), f(N + 1), f(3)
    balance = rsq.GQEBalance.of(counts, sums, loss, None, 0.1, 0.01)
    dy, y = torch.randn(R, dm, generator=torch.Generator().manual_seed(5)).cuda(), torch.empty(R, dm, dtype=torch.bfloat16, device="cuda")
    wf, wb = (torch.zeros(rsq.gqe_workspace_bytes(cfg, k), dtype=torch.uint8, device="cuda")
              for k in (rsq.GQE_WS_LAYER, rsq.GQE_WS_BACKWARD_AUX))

    def step():
        rsq.gqe_layer_fwd_rope(cfg, pos.rope, d["x"], *weights(d), y, wf)
        rsq.gqe_layer_bwd_aux(cfg, pos.rope, balance, d["x"], *weights(d), dy, *grads, wb)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    d["x"].copy_(d["x"].flip(0))
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (y, loss, counts, *grads)]
    step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, (y, loss, counts, *grads)))
    assert int(counts[-1]) == R and int(counts[:-1].sum()) == R * s.G * s.k
    assert rsq.gqe_read_status() == 0


def test_lengths_default_to_the_bound(rsq):
    s = LayerShape(B=2, T=33, d_model=64, G=2, M=2, k=1, d_head=64)
    d = device_inputs(synth.make_layer_inputs(s, seed=8))
    pos = Positions(rsq, s, s.B)
    cfg = rsq.GQEConfig.of(s)
    ws = ws_of(rsq, cfg, rsq.GQE_WS_DECODE_KV4)
    x = d["x"][: s.B].contiguous()
    res = []
    for lens in (None, torch.full((2,), 32, dtype=torch.int32, device="cuda")):
        t, cache = kv4(rsq, 2, 2, 48, 64)
        y = torch.empty(2, 64, dtype=torch.bfloat16, device="cuda")
        rsq.gqe_decode_step_kv4(cfg, pos.rope, x, *weights(d), cache, lens, y, ws)
        res.append((y, *t))
    assert all(torch.equal(a, b) for a, b in zip(*res))
    assert res[0][3][:, :, 32].ne(0).any() and not res[0][3][:, :, :32].ne(0).any()


def test_bf16_dev_helper_is_the_recipe(rsq):
    # The inputs above and the fp64 leaves hold the same numbers.
    inp = synth.make_layer_inputs(SHAPES["one_token"], seed=8)
    assert np.array_equal(bf16_dev(inp.W_k).double().cpu().numpy(), synth.bf16_to_f64(inp.W_k))
