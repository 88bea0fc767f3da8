"""The operators where offsets pass 32 bits (up to 26 GB on the device)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rsq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import routed_sparse_query_b200 as m
    yield m
    torch.cuda.empty_cache()


def test_kv4_rows_past_4_gb(rsq):
    # 2^27 + 32 keys of 32 bytes: the last rows' codes lie past 2^32 bytes. All
    # other keys are zero, so that the last, far larger score takes everything.
    cap, dh = (1 << 27) + 32, 64
    codes = [torch.zeros(1, 1, cap, dh // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
    meta = torch.zeros(1, 1, cap, 4, dtype=torch.bfloat16, device="cuda")
    cache = rsq.GQEKv4.of(*codes, meta)
    gen = torch.Generator().manual_seed(1)
    K, V = (torch.randn(1, 1, 5, dh, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    K[0, 0, 4] = 20.0 * K[0, 0, 4].sign()
    cfg = rsq.GQEConfig(1, 5, 64, 1, 1, 1, dh, 0)
    start = torch.tensor([cap - 5], dtype=torch.int32, device="cuda")
    rsq.gqe_kv4_append(cfg, K, V, start, None, cache)
    near = [torch.zeros(1, 1, 16, *t.shape[3:], dtype=t.dtype, device="cuda") for t in (*codes, meta)]
    rsq.gqe_kv4_append(cfg, K, V, None, None, rsq.GQEKv4.of(*near))
    for far, n in zip((*codes, meta), near):
        assert torch.equal(far[:, :, -5:], n[:, :, :5]) and not far[:, :, -100:-5].ne(0).any()
        assert not far[:, :, :100].ne(0).any()
    Ko, Vo = torch.empty_like(K), torch.empty_like(V)
    rsq.gqe_kv4_read(cfg, cache, start, None, Ko, Vo)
    assert (Ko - K).abs().max() <= 1.5 and (Vo - V).abs().max() <= 0.5
    q = K[:, :, 4:5].sign().contiguous()
    big = rsq.GQEConfig(1, cap, 64, 1, 1, 1, dh, 0)
    ws = torch.empty(rsq.gqe_workspace_bytes(big, rsq.GQE_WS_KV4), dtype=torch.uint8, device="cuda")
    out = torch.empty(1, dh, dtype=torch.bfloat16, device="cuda")
    rsq.gqe_kv4_attention(big, q, None, cache, None, out, ws)
    # The score is 160 against 0 and less: e^-120 times 2^27 keys is nothing.
    assert torch.equal(out[0], Vo[0, 0, 4])
    assert rsq.gqe_read_status() == 0


def test_rope_past_2_31_elements(rsq):
    # Keys [1, 8, T, 64] of 2.2e9 elements: the last head's last tokens.
    T, dh = 4300000, 64
    K = torch.zeros(1, 8, T, dh, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator().manual_seed(1)
    tail = torch.randn(1, 8, 40, dh, generator=gen).to(torch.bfloat16).cuda()
    K[:, :, -40:] = tail
    inv = (10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).cuda()
    rope = rsq.GQERope.of(64, inv, eps=1e-6, flags=rsq.GQE_ROPE_NORM)
    rsq.gqe_qk_rope(rsq.GQEConfig(1, T, 64, 8, 1, 1, dh, 0), rope, None, None, K, None, None, None, K)
    pos = torch.arange(T - 40, T, dtype=torch.int32, device="cuda").view(1, -1)
    small = rsq.GQERope.of(64, inv, pos=pos, eps=1e-6, flags=rsq.GQE_ROPE_NORM)
    want = torch.empty_like(tail)
    rsq.gqe_qk_rope(rsq.GQEConfig(1, 40, 64, 8, 1, 1, dh, 0), small, None, None, tail, None, None, None, want)
    assert torch.equal(K[:, :, -40:], want) and not K[:, :, -80:-40].ne(0).any()


def test_balance_past_2_31_logits(rsq):
    # 2^27 rows of 32 logits, equal but in the last row.
    R, G, M = 1 << 27, 16, 2
    z = torch.zeros(R, G * M, device="cuda")
    z[-1, 0] = 2.0
    idx = torch.zeros(R, G, 1, dtype=torch.int32, device="cuda")
    cfg = rsq.GQEConfig(1, R, 64, G, M, 1, 64, 0)
    assert rsq.gqe_workspace_bytes(cfg, rsq.GQE_WS_BALANCE) == 0  # more than 2^31 selections are refused
    R //= 2
    z, idx = z[R:], idx[R:]
    cfg = rsq.GQEConfig(1, R, 64, G, M, 1, 64, 0)
    counts, sums = torch.empty(G * M + 1, dtype=torch.int32, device="cuda"), torch.empty(G * M + 1, device="cuda")
    ws = torch.empty(rsq.gqe_workspace_bytes(cfg, rsq.GQE_WS_BALANCE), dtype=torch.uint8, device="cuda")
    loss, dz = torch.empty(3, device="cuda"), torch.empty(R, G * M, device="cuda")
    rsq.gqe_balance_stats(cfg, z, idx, None, counts, sums, ws)
    rsq.gqe_balance_loss(cfg, z, None, counts, sums, 1.0, 0.0, loss, dz)
    assert counts.tolist() == [R, 0] * G + [R]
    # f - 1/M = +-1/2, p = 1/2: dz = M/(G n) p (f - sum p f) = 2/(16 R) / 4 * +-1
    w = 1.0 / (32 * R)
    assert torch.allclose(dz[:-1].abs(), torch.full((), w, device="cuda"), rtol=1e-5, atol=0)
    p = torch.softmax(torch.tensor([2.0, 0.0], dtype=torch.float64), 0)
    f = torch.tensor([1.0, 0.0], dtype=torch.float64)
    want = 2 / (16 * R) * p * (f - (p * f).sum())
    assert torch.allclose(dz[-1, :2].cpu().double(), want, rtol=1e-5, atol=0)
    assert abs(float(loss[1]) - 1.0) < 1e-5
