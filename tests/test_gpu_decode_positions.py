"""The decode steps with positions given (rope->pos [axes, B], one row per
sequence), on several axes, with adjacent pairs, without the norm. Tolerances: those
of tests/test_gpu_operators_layer.py."""
import pytest
import torch

import synth
from gpu_common import device_inputs
from test_gpu_operators_layer import KINDS, SHAPES, Positions, close, kv4, layer_fwd, rsq, weights, ws_of  # noqa: F401

pytestmark = pytest.mark.gpu

GIVEN = {"far": dict(far=70000), "axes": dict(axes=2, far=900), **{n: dict(KINDS[n]) for n in ("axes_adjacent_far", "no_norm")}}
GIVEN["no_norm"]["far"] = 5000


def rope_with(rsq, pos, at):  # noqa: F811
    """pos's description with the positions `at` [axes, B]."""
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    return rsq.GQERope.of(pos.dh, pos.inv.cuda(), pos=at.to(torch.int32).contiguous().cuda(), axis=cuda(pos.axis),
                          w_q=pos.w_q.cuda() if pos.norm else None, w_k=pos.w_k.cuda() if pos.norm else None, eps=1e-5,
                          flags=(rsq.GQE_ROPE_NORM if pos.norm else 0) | (rsq.GQE_ROPE_ADJACENT if pos.adjacent else 0))


@pytest.mark.parametrize("kind", list(GIVEN))
@pytest.mark.parametrize("name", ["b2_t70", "m3_k2_dh32", "one_token"])
def test_decode_continues_a_prefill(rsq, name, kind):  # noqa: F811
    # The last token's row of a prefill, decoded at that token's own positions.
    s = SHAPES[name]
    d = device_inputs(synth.make_layer_inputs(s, seed=8))
    pos = Positions(rsq, s, s.R, **GIVEN[kind])
    y, ws, cfg = layer_fwd(rsq, s, d, pos.rope)
    B, T, G, dh = s.B, s.T, s.G, s.d_head
    cap = T + 5
    K, V = (rsq.workspace_view(ws, cfg, rsq.GQE_WS_LAYER, n, torch.bfloat16, (B, G, T, dh)) for n in ("K", "V"))
    caches = [torch.zeros(B, G, cap, dh, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for c, full in zip(caches, (K, V)):
        c[:, :, : T - 1] = full[:, :, : T - 1]
    x = d["x"].view(B, T, -1)[:, T - 1].contiguous()
    at = pos.pos.view(-1, B, T)[:, :, T - 1]
    yd, wd = torch.empty(B, s.d_model, dtype=torch.bfloat16, device="cuda"), ws_of(rsq, cfg, rsq.GQE_WS_DECODE)
    rsq.gqe_decode_step_rope(cfg, rope_with(rsq, pos, at), x, *weights(d), *caches, yd, wd)
    for c, full in zip(caches, (K, V)):
        want = full[:, :, T - 1].float()
        assert ((c[:, :, T - 1].float() - want).abs() <= 2.0 ** -6 * want.abs() + 2.0 ** -6).all()
        assert (c[:, :, T:] == 0).all() and torch.equal(c[:, :, : T - 1], full[:, :, : T - 1])
    close(yd, y.double().cpu().view(B, T, -1)[:, T - 1], "decoded y")
    assert rsq.gqe_read_status() == 0


@pytest.mark.parametrize("kind", list(GIVEN))
@pytest.mark.parametrize("B,dh", [(1, 64), (5, 64), (3, 32)])
def test_decode_over_the_4_bit_cache(rsq, B, dh, kind):  # noqa: F811
    # Positions that have nothing to do with the sequences' lengths: bit for bit
    # the step's parts, with the positions on the queries and keys of one token.
    s = synth.LayerShape(B=B, T=40, d_model=128, G=2, M=3, k=2, d_head=dh)
    d = device_inputs(synth.make_layer_inputs(s, seed=8))
    G, M, k, most = s.G, s.M, s.k, 48
    pos = Positions(rsq, s, B, **GIVEN[kind])
    rope = rope_with(rsq, pos, pos.pos)
    lens = torch.tensor([40, 7, -1, 0, 13][:B], dtype=torch.int32, device="cuda")
    gen = torch.Generator().manual_seed(3)
    Kp, Vp = (torch.randn(B, G, 40, dh, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    caches = []
    for _ in range(2):
        caches.append(kv4(rsq, B, G, most, dh))
        rsq.gqe_kv4_append(rsq.GQEConfig.of(s), Kp, Vp, None, lens.clamp(min=0), caches[-1][1])
    cfg, one = rsq.GQEConfig(B, most, 128, G, M, k, dh, 0), rsq.GQEConfig(B, 1, 128, G, M, k, dh, 0)
    x = d["x"].view(B, 40, -1)[:, 39].contiguous()
    e = lambda *shape, dt=torch.bfloat16: torch.empty(*shape, dtype=dt, device="cuda")  # noqa: E731
    y, y2 = e(B, 128), e(B, 128)
    rsq.gqe_decode_step_kv4(cfg, rope, x, *weights(d), caches[0][1], lens, y, ws_of(rsq, cfg, rsq.GQE_WS_DECODE_KV4))
    i32 = dict(dt=torch.int32)
    idx, r, om = e(B, G, k, **i32), e(B, G, k, dt=torch.float32), e(B, G, k, dt=torch.float32)
    rsq.gqe_router_topk(one, x, d["W_r"], d["b_r"], idx, r, om)
    Q, Qs, K, V = e(B, G, k, 1, dh), e(B, 1, dh), e(B, G, 1, dh), e(B, G, 1, dh)
    rsq.gqe_dispatch(one, idx, x, d["W_q"], d["W_qs"], e(G * M * B, **i32), e(G * M * B + 1, **i32), e(k * G * B, **i32),
                     e(B, G, k, **i32), Q, Qs, ws_of(rsq, one, rsq.GQE_WS_DISPATCH))
    rsq.gqe_kv_proj(one, x, d["W_k"], d["W_v"], K, V)
    # In fp64, from the unrotated keys: half a step of bf16, and 2^-16 for fp32.
    heads = K[:, :, 0].double().cpu()
    want = pos.apply(heads, pos.w_k.double(), None)
    rsq.gqe_qk_rope(one, rope, Q, Qs, K, None, Q, Qs, K)
    size = want.abs() + 2.0 ** -8 * want.abs().amax(-1, keepdim=True)
    assert ((K[:, :, 0].double().cpu() - want).abs() <= (2.0 ** -8 + 2.0 ** -16) * size).all()
    rsq.gqe_kv4_append(one, K, V, lens, None, caches[1][1])
    slots = e(B, (G * k + 2) * dh)
    rsq.gqe_kv4_attention(cfg, Q, Qs, caches[1][1], lens + 1, slots, ws_of(rsq, cfg, rsq.GQE_WS_KV4))
    rsq.gqe_output_proj(one, slots, om, d["W_o"], y2)
    assert torch.equal(y, y2)
    assert all(torch.equal(a, b) for a, b in zip(caches[0][0], caches[1][0]))
    assert rsq.gqe_read_status() == 0
