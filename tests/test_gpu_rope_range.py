"""Norm and rotation of rows near the ends of the stated range, 2^-60 <= |x| <=
2^60: the norm's sum of squares is an fp32 and neither overflows nor, with eps = 0,
is lost. Tolerances: those of tests/test_gpu_rope.py, relative to the result."""
import numpy as np
import pytest
import torch

from oracle import operators as op
from test_gpu_rope import rsq  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dh", [32, 64])
@pytest.mark.parametrize("size", [-57, 57])
def test_rows_near_the_ends_of_the_range(rsq, size, dh):  # noqa: F811
    # Elements of 2^(size - 3) to 2^(size + 3).
    B, T, G = 1, 40, 2
    rng = np.random.default_rng(3)
    x = rng.choice([-1, 1], (B, G, T, dh)) * np.exp2(size + rng.uniform(-3, 3, (B, G, T, dh)))
    K = torch.from_numpy(x).to(torch.bfloat16)
    g = torch.from_numpy(rng.standard_normal((B, G, T, dh))).float()
    w = torch.from_numpy(1 + 0.2 * rng.standard_normal(dh)).float()
    inv = 10000.0 ** (-2.0 * torch.arange(dh // 2, dtype=torch.float64) / dh)
    rope = rsq.GQERope.of(dh, inv.cuda(), w_k=w.cuda(), eps=0.0, flags=rsq.GQE_ROPE_NORM)
    cfg = rsq.GQEConfig(B, T, 64, G, 1, 1, dh, 0)
    y, dk, dw = torch.empty_like(K, device="cuda"), torch.empty(B, G, T, dh, device="cuda"), torch.empty(dh, device="cuda")
    ws = torch.empty(rsq.gqe_workspace_bytes(cfg, rsq.GQE_WS_QK_ROPE), dtype=torch.uint8, device="cuda")
    rsq.gqe_qk_rope(cfg, rope, None, None, K.cuda(), None, None, None, y)
    rsq.gqe_qk_rope_bwd(cfg, rope, None, None, K.cuda(), None, None, None, g.cuda(), None, None, dk, None, dw, ws)
    ang = op.rope_angles(np.arange(T)[None], inv.numpy(), None)
    x, gd, wd = K.double().numpy(), g.double().numpy(), w.double().numpy()
    want = op.rope(x, ang, norm=True, w=wd)
    n = op.rope_norm(x, wd, 0.0)
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -17 * np.abs(n).max(-1, keepdims=True)
    assert (np.abs(y.double().cpu().numpy() - want) <= tol).all()
    dx, dwr = op.rope_backward(x, gd, ang, norm=True, w=wd)
    rstd = 1 / np.sqrt((x * x).mean(-1, keepdims=True))
    gmax = 2 * np.abs(gd).max(-1, keepdims=True) * np.abs(wd).max()
    btol = 2.0 ** -16 * rstd * gmax * (1 + np.abs(x * rstd).max(-1, keepdims=True)) + np.zeros_like(x)
    assert (np.abs(dk.double().cpu().numpy() - dx) <= btol).all()
    size = (2 * np.abs(gd).max(-1, keepdims=True) * np.abs(x * rstd)).reshape(-1, dh).sum(0)
    assert (np.abs(dw.double().cpu().numpy() - dwr) <= 2.0 ** -16 * size).all()
    assert rsq.gqe_read_status() == 0
