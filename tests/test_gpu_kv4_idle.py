"""The 4-bit attention over batches that are mostly idle (a server's padded batch):
runs of sequences without keys in front, between and behind the live ones."""
import numpy as np
import pytest
import torch

from test_gpu_kv4 import attention_reference, host, new_cache, rsq, run_attention  # noqa: F401

pytestmark = pytest.mark.gpu

# Live sequences of a batch of 400 and their keys: runs of idle ones of 31 to 33,
# 63 to 65 and more, at either end, one live sequence only.
LIVE = {
    "runs_of_31_to_65": {0: 65, 32: 64, 64: 1, 98: 200, 130: 63, 194: 130, 259: 7, 325: 64, 399: 128},
    "last_only": {399: 200},
    "first_only": {0: 200},
    "behind_255": {255: 70, 256: 70, 300: 200},
    "idle_ends": {33: 200, 34: 1, 367: 65},
}


@pytest.mark.parametrize("G,k", [(1, 1), (2, 2), (3, 5)])
@pytest.mark.parametrize("name", list(LIVE))
def test_idle_runs(rsq, name, G, k):  # noqa: F811
    B, T, dh = 400, 200, 64
    lens = [LIVE[name].get(b, -1 if b % 3 else 0) for b in range(B)]
    t, cache = new_cache(rsq, B, G, 208, dh, seed=5)
    q = torch.randn(B, G, k, dh, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16)
    cfg = rsq.GQEConfig(B, T, 64, G, k, k, dh, 0)
    got = run_attention(rsq, cfg, q, None, cache, lens)
    want, tol = attention_reference(q, None, host(t), lens, T, k)
    assert (np.abs(got.double().numpy() - want) <= tol).all()
    assert rsq.gqe_read_status() == 0


def test_idle_sequences_cost_less_than_live_ones(rsq):  # noqa: F811
    # 4096 sequences of up to 256 keys, all of them live against one: a batch
    # with less to read is not slower.
    B, G, k, dh, T = 4096, 8, 1, 64, 256
    codes = [torch.zeros(B, G, T, dh // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache = rsq.GQEKv4.of(*codes, torch.ones(B, G, T, 4, dtype=torch.bfloat16, device="cuda"))
    q = torch.ones(B, G, k, dh, dtype=torch.bfloat16, device="cuda")
    cfg = rsq.GQEConfig(B, T, 64, G, k, k, dh, 0)
    ws = torch.empty(rsq.gqe_workspace_bytes(cfg, rsq.GQE_WS_KV4), dtype=torch.uint8, device="cuda")
    out = torch.empty(B, G * k * dh, dtype=torch.bfloat16, device="cuda")

    def time_of(lens):
        best = float("inf")
        for _ in range(20):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            rsq.gqe_kv4_attention(cfg, q, None, cache, lens, out, ws)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    one = torch.zeros(B, dtype=torch.int32, device="cuda")
    one[0] = T
    assert time_of(one) < time_of(None)
