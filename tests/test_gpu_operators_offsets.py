"""Rows whose offsets from the pointers of the call pass 2^31 elements (up to 40 GB
on the device): balance loss, backward of the rotation, token lists, rows stored
in the 4-bit cache. The rows at the end against a small call on the same rows."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def rsq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import routed_sparse_query_b200 as m
    yield m
    torch.cuda.empty_cache()


@pytest.fixture(autouse=True)
def room():
    yield
    torch.cuda.empty_cache()


def positions(rsq, T, first, dh=64):
    """GQERope of T tokens, positions from `first` on."""
    gen = torch.Generator().manual_seed(2)
    inv = (10000.0 ** (-torch.arange(dh // 2, dtype=torch.float64) / (dh // 2))).cuda()
    w = (1 + 0.2 * torch.randn(2, dh, generator=gen)).cuda()
    pos = torch.arange(first, first + T, dtype=torch.int32, device="cuda").view(1, -1)
    return rsq.GQERope.of(dh, inv, pos=pos, w_q=w[0], w_k=w[1], eps=1e-6, flags=rsq.GQE_ROPE_NORM)


def test_balance(rsq):
    # 2^26 + 300 rows of 32 logits, equal but in the last row: its logits and
    # their gradient lie past 2^31 elements.
    R, G, M = (1 << 26) + 300, 8, 4
    N = G * M
    assert R * N > 1 << 31
    z = torch.zeros(R, N, device="cuda")
    z[-1, 0] = 2.0
    idx = torch.zeros(R, G, 1, dtype=torch.int32, device="cuda")
    idx[-1] = 1
    cfg = rsq.GQEConfig(1, R, 64, G, M, 1, 64, 0)
    counts, sums = torch.empty(N + 1, dtype=torch.int32, device="cuda"), torch.empty(N + 1, device="cuda")
    ws = torch.empty(rsq.gqe_workspace_bytes(cfg, rsq.GQE_WS_BALANCE), dtype=torch.uint8, device="cuda")
    loss, dz = torch.empty(3, device="cuda"), torch.full((R, N), float("nan"), device="cuda")
    rsq.gqe_balance_stats(cfg, z, idx, None, counts, sums, ws)
    rsq.gqe_balance_loss(cfg, z, None, counts, sums, 1.0, 0.0, loss, dz)
    assert counts.tolist() == [R - 1, 1, 0, 0] * G + [R]
    f = torch.tensor([(R - 1) / R, 1 / R, 0, 0], dtype=torch.float64)
    even = (M / (G * R) * 0.25 * (f - f.mean())).float().cuda()
    del z, idx
    for rows in dz[:-1].split(1 << 24):  # 2^-15 of the terms, as at other sizes
        assert ((rows.view(-1, G, M) - even).abs() <= 2.0 ** -15 * M / (G * R) * 0.25).all()
    p = torch.softmax(torch.tensor([2.0, 0, 0, 0], dtype=torch.float64), 0)
    want = M / (G * R) * p * (f - (p * f).sum())
    assert ((dz[-1, :M].double().cpu() - want).abs() <= 2.0 ** -15 * M / (G * R) * p).all()
    assert rsq.gqe_read_status() == 0


def test_rotation_backward(rsq):
    # dK [1, 8, T, 64] of 2.2e9 elements, all zero but for the last tokens.
    T, G, dh, n = 4300000, 8, 64, 70
    gen = torch.Generator().manual_seed(1)
    tail = torch.randn(1, G, n, dh, generator=gen).to(BF16).cuda()
    gtail = torch.randn(1, G, n, dh, generator=gen).cuda()
    K, dKo = torch.zeros(1, G, T, dh, dtype=BF16, device="cuda"), torch.zeros(1, G, T, dh, device="cuda")
    dK = torch.full((1, G, T, dh), float("nan"), device="cuda")
    K[:, :, -n:], dKo[:, :, -n:] = tail, gtail
    ws = torch.empty(rsq.gqe_workspace_bytes(rsq.GQEConfig(1, T, 64, G, 1, 1, dh, 0), rsq.GQE_WS_QK_ROPE),
                     dtype=torch.uint8, device="cuda")

    def call(T, K, dKo, dK, rope):
        dw = [torch.empty(dh, device="cuda") for _ in range(2)]
        rsq.gqe_qk_rope_bwd(rsq.GQEConfig(1, T, 64, G, 1, 1, dh, 0), rope, None, None, K, None, None, None, dKo, None, None,
                            dK, *dw, ws)
        return dw

    dw = call(T, K, dKo, dK, positions(rsq, T, 0))
    want = torch.empty_like(gtail)
    dw_small = call(n, tail, gtail, want, positions(rsq, n, T - n))
    assert torch.equal(dK[:, :, -n:], want)
    for rows in dK[0, :, :-n].split(1 << 20, 1):
        assert not rows.ne(0).any()  # nothing else: zeros, and every row written
    assert (dw[0] == 0).all()
    # The same 560 terms in two orders, each in at most 64 additions one after the
    # other: 2^-17 of the sum of their sizes.
    pair = gtail.square().unflatten(-1, (2, dh // 2)).sum(-2).sqrt().repeat(1, 1, 1, 2)
    x = tail.float()
    size = (pair * x.abs() * x.square().mean(-1, keepdim=True).rsqrt()).sum((0, 1, 2))
    assert ((dw[1] - dw_small[1]).abs() <= 2.0 ** -17 * size).all() and dw[1].abs().max() > 1
    del K, dKo, dK
    assert rsq.gqe_read_status() == 0


def test_rotation_in_token_list_order(rsq):
    # Queries [8 T, 64] of 2.2e9 elements; the list names a token's rows in
    # reverse, so that the last rows belong to the first token and the reverse.
    T, G, dh = 4300000, 8, 64
    Q = torch.zeros(G * T, dh, dtype=BF16, device="cuda")
    gen = torch.Generator().manual_seed(1)
    ends = torch.randn(2, 40, dh, generator=gen).to(BF16).cuda()
    Q[:40], Q[-40:] = ends[0], ends[1]
    slot = (G * T - 1 - torch.arange(G * T, dtype=torch.int32, device="cuda")).view(T, G, 1).contiguous()
    rsq.gqe_qk_rope(rsq.GQEConfig(1, T, 64, G, 1, 1, dh, 0), positions(rsq, T, 0), Q, None, None, slot, Q, None, None)
    # Row e belongs to token (G T - 1 - e) / G: 5 tokens' rows at either end.
    small_slot = (39 - torch.arange(40, dtype=torch.int32, device="cuda")).view(5, G, 1).contiguous()
    for rows, x, first in ((Q[-40:], ends[1], 0), (Q[:40], ends[0], T - 5)):
        want = torch.empty_like(x)
        rsq.gqe_qk_rope(rsq.GQEConfig(1, 5, 64, G, 1, 1, dh, 0), positions(rsq, 5, first), x, None, None, small_slot, want,
                        None, None)
        assert torch.equal(rows, want) and not torch.equal(rows, x)
    for rows in Q[40:-40].split(1 << 22):
        assert not rows.ne(0).any()
    assert rsq.gqe_read_status() == 0


def test_kv4_rows(rsq):
    # K, V [1, 8, T, 64] of 2.2e9 elements stored and read back.
    T, G, dh, n = 4300000, 8, 64, 33
    cap = T + 16
    gen = torch.Generator().manual_seed(1)
    tails = [torch.randn(1, G, n, dh, generator=gen).to(BF16).cuda() for _ in range(2)]
    K, V = (torch.zeros(1, G, T, dh, dtype=BF16, device="cuda") for _ in range(2))
    K[:, :, -n:], V[:, :, -n:] = tails

    def cache(cap):
        t = [torch.zeros(1, G, cap, dh // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
        t.append(torch.zeros(1, G, cap, 4, dtype=BF16, device="cuda"))
        return t, rsq.GQEKv4.of(*t)

    big, small = cache(cap), cache(48)
    cfg, c2 = rsq.GQEConfig(1, T, 64, G, 1, 1, dh, 0), rsq.GQEConfig(1, n, 64, G, 1, 1, dh, 0)
    start = torch.tensor([3], dtype=torch.int32, device="cuda")
    rsq.gqe_kv4_append(cfg, K, V, start, None, big[1])
    rsq.gqe_kv4_append(c2, *tails, None, None, small[1])
    for far, near in zip(big[0], small[0]):
        assert torch.equal(far[:, :, T + 3 - n:T + 3], near[:, :, :n])
        assert not far[:, :, T + 3:].ne(0).any() and not far[:, :, :T + 3 - n].ne(0).any()
    K.fill_(7.0)
    V.fill_(7.0)
    rsq.gqe_kv4_read(cfg, big[1], start, None, K, V)
    out = [torch.empty_like(t) for t in tails]
    rsq.gqe_kv4_read(c2, small[1], None, None, *out)
    for far, near in zip((K, V), out):
        assert torch.equal(far[:, :, -n:], near)
        for rows in far[0, :, :-n].split(1 << 20, 1):
            assert not rows.ne(0).any()
    assert rsq.gqe_read_status() == 0
