"""The 4-bit attention at the ends of the queries' range.

A query may be any finite bf16: what is formed of it on the way (its factor, the
sum of its elements, its product with a row's codes) stays finite where the scores
are. Tolerances are those of tests/test_gpu_kv4.py."""
import numpy as np
import pytest
import torch

from test_gpu_kv4 import attention_reference, host, new_cache, rsq, run_attention  # noqa: F401

pytestmark = pytest.mark.gpu

# B, G, k, shared, dh, T: one to four heads, up to eight and sixteen; a cluster per
# unit, then equal shares with a join.
CASES = {
    "k1": (2, 2, 1, False, 64, 330),
    "k1_shared_dh32": (2, 2, 1, True, 32, 130),
    "k4": (1, 2, 4, False, 64, 200),
    "k8": (1, 1, 8, False, 64, 200),
    "k15_shared_dh32": (1, 1, 15, True, 32, 70),
    "shares_k1": (300, 1, 1, False, 64, 130),
    "shares_k4_dh32": (300, 1, 4, False, 32, 70),
    "shares_long": (1, 1, 2, True, 64, 33001),
}


@pytest.mark.parametrize("name", list(CASES))
def test_queries_near_the_largest(rsq, name):  # noqa: F811
    # Queries up to the largest bf16 on keys so small that the scores are of
    # order one; rows whose codes are all 0 or all 15 among them.
    B, G, k, shared, dh, T = CASES[name]
    t, cache = new_cache(rsq, B, G, (T + 15) // 16 * 16, dh, seed=2)
    t[2][..., :2] *= 2.0 ** -124
    t[0][:, :, 3] = 0
    t[0][:, :, 4] = 255
    gen = torch.Generator().manual_seed(1)
    q = (torch.randn(B, G, k, dh, generator=gen).clamp(-7, 7) * 2.0 ** 122).to(torch.bfloat16)
    q[:, :, 0, 0] = torch.finfo(torch.bfloat16).max
    q[:, -1, -1] = 2.0 ** 126  # one sign: their sum passes fp32's range
    qs = (torch.randn(B, dh, generator=gen).clamp(-7, 7) * 2.0 ** 122).to(torch.bfloat16) if shared else None
    cfg = rsq.GQEConfig(B, T, 64, G, k, k, dh, 0)
    got = run_attention(rsq, cfg, q, qs, cache, None)
    want, tol = attention_reference(q, qs, host(t), [T] * B, T, k)
    err = np.abs(got.double().numpy() - want)
    assert (err <= tol).all(), f"{int(np.isnan(err).sum())} NaN, worst {np.nanmax(err / tol):.3f} of the tolerance"


def test_ordinary_queries_beside_tiny_ones(rsq):  # noqa: F811
    # Heads of one group with queries of 2^-110 and 0 (all scores even), 1 and
    # 2^-4 side by side: each head has its own factor.
    B, G, k, dh, T = 1, 1, 4, 64, 500
    t, cache = new_cache(rsq, B, G, 512, dh, seed=2)
    q = torch.randn(B, G, k, dh, generator=torch.Generator().manual_seed(1))
    q = (q * torch.tensor([2.0 ** -110, 1.0, 0.0, 2.0 ** -4]).view(1, 1, k, 1)).to(torch.bfloat16)
    cfg = rsq.GQEConfig(B, T, 64, G, k, k, dh, 0)
    got = run_attention(rsq, cfg, q, None, cache, None)
    want, tol = attention_reference(q, None, host(t), [T], T, k)
    assert (np.abs(got.double().numpy() - want) <= tol).all()
