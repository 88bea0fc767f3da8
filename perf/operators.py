"""Workloads of the layer's position, balance and 4-bit cache operators.

Every case is one operator on the shapes that the layer meets: 8 KV groups of 2 or 4 query-head experts,
head dim 64, sequences of one token to 256k, a decode batch of 64 sequences over a 32k cache. `run` computes it
in plain torch operations, or through the library's entry points where `own` is true.
"""
import math

import torch

own = False

_BF16 = torch.bfloat16


def listed():
    return [
        # One decode step of 64 sequences: their new queries and keys, each at its own far position.
        {"name": "rope-decode-b64", "op": "rope", "B": 64, "T": 1, "G": 8, "M": 2, "k": 1, "dh": 64, "rot": 64,
         "norm": True, "axes": 1, "pairs": "half", "far": 32768, "grad": False},
        # Prefill of the batch-4 8k layer.
        {"name": "rope-4x8k", "op": "rope", "B": 4, "T": 8192, "G": 8, "M": 2, "k": 1, "dh": 64, "rot": 64,
         "norm": True, "axes": 1, "pairs": "half", "far": 0, "grad": False},
        # Long-context prefill with image and video tokens: time, height and width positions.
        {"name": "rope-256k-3axes", "op": "rope", "B": 1, "T": 262144, "G": 8, "M": 2, "k": 1, "dh": 64, "rot": 64,
         "norm": True, "axes": 3, "pairs": "half", "far": 0, "grad": False},
        # The backward pass of the headline 2k layer, and of the batch-4 8k expert pool.
        {"name": "rope-bwd-2k", "op": "rope", "B": 1, "T": 2048, "G": 8, "M": 2, "k": 1, "dh": 64, "rot": 64,
         "norm": True, "axes": 1, "pairs": "half", "far": 0, "grad": True},
        {"name": "rope-bwd-4x8k-pool", "op": "rope", "B": 4, "T": 8192, "G": 8, "M": 4, "k": 2, "dh": 64, "rot": 64,
         "norm": True, "axes": 1, "pairs": "half", "far": 0, "grad": True},
        # The router's balance loss, counts and logit gradient in a training step: the 2k layer ...
        {"name": "balance-2k", "op": "balance", "B": 1, "T": 2048, "G": 8, "M": 2, "k": 1, "skew": 0.0, "masked": False},
        # ... and a 256k batch of the expert pool with one favoured expert per group and padded rows.
        {"name": "balance-256k-pool", "op": "balance", "B": 1, "T": 262144, "G": 8, "M": 4, "k": 2, "skew": 2.0,
         "masked": True},
        # The new keys and values of a decode step into the 4-bit cache and back ...
        {"name": "kv4-store-decode-b64", "op": "store", "B": 64, "T": 1, "G": 8, "dh": 64, "cap": 32768},
        # ... and a whole prefill's.
        {"name": "kv4-store-4x8k", "op": "store", "B": 4, "T": 8192, "G": 8, "dh": 64, "cap": 8192},
        # Decode attention over the 4-bit cache: one 2k sequence (latency), a ragged batch with empty sequences and
        # all heads of the pool, the full 64 x 32k cache.
        {"name": "kv4-attn-b1-2k", "op": "attn", "B": 1, "T": 2048, "G": 8, "M": 2, "k": 1, "dh": 64, "dense": False,
         "ragged": False},
        {"name": "kv4-attn-b33-5k-ragged", "op": "attn", "B": 33, "T": 5003, "G": 8, "M": 4, "k": 2, "dh": 64,
         "dense": True, "ragged": True},
        {"name": "kv4-attn-b64-32k", "op": "attn", "B": 64, "T": 32768, "G": 8, "M": 2, "k": 1, "dh": 64,
         "dense": False, "ragged": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "balance", "store", "attn", "attn"])
    G, M = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4])
    k = rng.randint(1, M)
    dh = rng.choice([32, 64, 64])
    if op == "rope":
        B = _log_int(rng, 1, 64)
        T = _log_int(rng, 1, max(1, 32768 // B))
        return {"op": op, "B": B, "T": T, "G": G, "M": M, "k": min(k, 2), "dh": dh,
                "rot": rng.choice([dh, dh, dh // 2, 8, 0]), "norm": rng.random() < 0.75, "axes": rng.choice([1, 1, 2, 3]),
                "pairs": rng.choice(["half", "adjacent"]), "far": rng.choice([0, 32768, 1048576]),
                "grad": rng.random() < 0.5}
    if op == "balance":
        M = rng.choice([1, 2, 3, 4, 8])
        B = _log_int(rng, 1, 16)
        return {"op": op, "B": B, "T": _log_int(rng, 1, 262144 // B), "G": min(G, 64 // M), "M": M,
                "k": rng.randint(1, min(M, 2)), "skew": rng.choice([0.0, 2.0]), "masked": rng.random() < 0.5}
    if op == "store":
        B = _log_int(rng, 1, 64)
        T = _log_int(rng, 1, max(1, 32768 // B))
        return {"op": op, "B": B, "T": T, "G": G, "dh": dh, "cap": (T + rng.randint(0, 64) + 15) // 16 * 16}
    B = _log_int(rng, 1, 64)
    return {"op": op, "B": B, "T": _log_int(rng, 1, 32768), "G": G, "M": M, "k": k, "dh": dh,
            "dense": rng.random() < 0.4, "ragged": rng.random() < 0.6}


def _heads(case):
    """(query streams, the shared head's) of a case: k routed streams per group and the shared head, or every head."""
    return (case["G"] * case["M"], 0) if case.get("dense") else (case["G"] * case["k"], 1)


def _lens(case):
    """Keys per sequence: T, or ragged from nothing to T (a padded batch, with idle sequences)."""
    B, T = case["B"], case["T"]
    if not case["ragged"]:
        return [T] * B
    return [T if b == 0 else 0 if b % 8 == 5 else 1 + (b * 7919) % T for b in range(B)]


def work(case):
    B, T, G = case["B"], case["T"], case["G"]
    R = B * T
    if case["op"] == "rope":
        n = R * (G * case["k"] + 1 + G) * case["dh"]
        pos = 4 * R * case["axes"]
        return {"bytes": n * (10 if case["grad"] else 4) + pos, "flops": n * (14 if case["grad"] else 8)}
    if case["op"] == "balance":
        n = R * G * case["M"]
        return {"bytes": 8 * n + 4 * R * G * case["k"] + (R if case["masked"] else 0), "flops": 12 * n}
    if case["op"] == "store":
        n = 2 * R * G * case["dh"]  # read, stored as 4 bits with scale and zero, and given back
        return {"bytes": n * 4 + n // 2 + n // case["dh"] * 4, "flops": 6 * n}
    keys = sum(_lens(case)) * G
    hq, hs = _heads(case)
    return {"bytes": keys * (case["dh"] + 8) + 4 * B * (hq + hs) * case["dh"],
            "flops": sum(_lens(case)) * (hq + hs) * 4 * case["dh"]}


def _rand(gen, *shape, dtype=_BF16, mul=1.0):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).mul_(mul).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    B, T, G = case["B"], case["T"], case["G"]
    R = B * T
    s = {"case": case}
    if case["op"] == "rope":
        k, dh, rot = case["k"], case["dh"], case["rot"]
        # Projections of rms ~1 with a few large channels, as trained keys and queries have them.
        gain = 1.0 + 3.0 * (torch.arange(dh, device="cuda") % 16 == 3).float()
        shapes = {"Q": (B, G, k, T, dh), "Qs": (B, T, dh), "K": (B, G, T, dh)}
        for name, shape in shapes.items():
            s[name] = (_rand(gen, *shape, dtype=torch.float32) * gain).to(_BF16)
            if case["grad"]:
                s["g" + name] = _rand(gen, *shape, dtype=torch.float32, mul=0.1)
            s["o" + name] = torch.empty(shape, dtype=torch.float32 if case["grad"] else _BF16, device="cuda")
        s["w_q"] = 1.0 + _rand(gen, dh, dtype=torch.float32, mul=0.1) if case["norm"] else None
        s["w_k"] = 1.0 + _rand(gen, dh, dtype=torch.float32, mul=0.1) if case["norm"] else None
        s["dw_q"], s["dw_k"] = torch.empty(dh, device="cuda"), torch.empty(dh, device="cuda")
        i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
        s["inv_freq"] = 500000.0 ** (-2.0 * i / max(rot, 1))
        s["axis"] = (torch.arange(rot // 2, device="cuda") % case["axes"]).to(torch.int32) if case["axes"] > 1 else None
        t = torch.arange(T, device="cuda").repeat(B)
        if case["far"]:  # each sequence at its own place of a long context
            t = t + torch.randint(0, case["far"], (B,), generator=gen, device="cuda").repeat_interleave(T)
        # Time, then height and width in 24 x 24 patches.
        axes = [t] if case["axes"] == 1 else [t // 576, t // 24 % 24, t % 24][: case["axes"]]
        s["pos"] = torch.stack(axes).to(torch.int32).contiguous()
        s["eps"] = 1e-6
    elif case["op"] == "balance":
        M, k = case["M"], case["k"]
        z = _rand(gen, R, G, M, dtype=torch.float32)
        z[:, :, 0] += case["skew"]
        top = z.topk(k, dim=2).indices
        s["idx"] = top.sort(dim=2).values.to(torch.int32).contiguous()
        s["z"] = z.reshape(R, G * M)
        # Padded rows at each sequence's end.
        s["mask"] = ((torch.arange(T, device="cuda") < T - T // 5).repeat(B).to(torch.uint8)
                     if case["masked"] else None)
        s["c_balance"], s["c_z"] = 0.01, 0.001
        s["counts"] = torch.empty(G * M + 1, dtype=torch.int32, device="cuda")
        s["sums"] = torch.empty(G * M + 1, dtype=torch.float32, device="cuda")
        s["loss"] = torch.empty(3, dtype=torch.float32, device="cuda")
        s["dz"] = torch.empty(R, G * M, dtype=torch.float32, device="cuda")
    elif case["op"] == "store":
        dh, cap = case["dh"], case["cap"]
        s["K"] = _rand(gen, B, G, T, dh) * (1.0 + 3.0 * (torch.arange(dh, device="cuda") % 16 == 3)).to(_BF16)
        s["V"] = _rand(gen, B, G, T, dh)
        s["start"] = torch.randint(0, cap - T + 1, (B,), generator=gen, device="cuda").to(torch.int32)
        s["k_codes"] = torch.zeros(B, G, cap, dh // 2, dtype=torch.uint8, device="cuda")
        s["v_codes"] = torch.zeros(B, G, cap, dh // 2, dtype=torch.uint8, device="cuda")
        s["meta"] = torch.zeros(B, G, cap, 4, dtype=_BF16, device="cuda")
        s["oK"], s["oV"] = torch.empty_like(s["K"]), torch.empty_like(s["V"])
    else:
        k, dh, M = case["k"], case["dh"], case["M"]
        cap = (T + 15) // 16 * 16
        hq, hs = _heads(case)
        s["Q"] = _rand(gen, B, G, hq // G, dh)
        s["Qs"] = _rand(gen, B, dh) if hs else None
        # Codes of rows of rms ~1: the range of dh normal values in 15 steps.
        for name in ("k_codes", "v_codes"):
            s[name] = torch.randint(0, 256, (B, G, cap, dh // 2), generator=gen, device="cuda", dtype=torch.uint8)
        step = 0.2 + 0.1 * torch.rand(B, G, cap, 2, generator=gen, device="cuda")
        s["meta"] = torch.stack([step[..., 0], -7.5 * step[..., 0], step[..., 1], -7.5 * step[..., 1]], -1).to(_BF16)
        s["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
        s["out"] = torch.empty(B, (hq + hs) * dh, dtype=_BF16, device="cuda")
    return s


# ------------------------------------------------------------------ the library's calls


def _handle(s):
    """What a program sets up once: the configuration, the operator's description and its workspace."""
    if "cfg" in s:
        return s
    import routed_sparse_query_b200 as rsq
    c = s["case"]
    op = c["op"]
    M = c.get("M", 2)
    heads = M if c.get("dense") else c.get("k", 1)
    s["cfg"] = rsq.GQEConfig(c["B"], c["T"], 1024, c["G"], M, heads, c.get("dh", 64), 0)
    kind = None
    if op == "rope":
        flags = (rsq.GQE_ROPE_NORM if c["norm"] else 0) | (rsq.GQE_ROPE_ADJACENT if c["pairs"] == "adjacent" else 0)
        s["rope"] = rsq.GQERope.of(c["rot"], s["inv_freq"], pos=s["pos"], axis=s["axis"], w_q=s["w_q"], w_k=s["w_k"],
                                   eps=s["eps"], flags=flags)
        kind = rsq.GQE_WS_QK_ROPE if c["grad"] else None
    elif op == "balance":
        kind = rsq.GQE_WS_BALANCE
    else:
        s["cache"] = rsq.GQEKv4.of(s["k_codes"], s["v_codes"], s["meta"])
        kind = rsq.GQE_WS_KV4 if op == "attn" else None
    if kind is not None:
        s["ws"] = torch.empty(rsq.gqe_workspace_bytes(s["cfg"], kind), dtype=torch.uint8, device="cuda")
    s["rsq"] = rsq
    return s


def _run_own(s):
    c = s["case"]
    _handle(s)
    rsq, cfg = s["rsq"], s["cfg"]
    if c["op"] == "rope":
        if c["grad"]:
            dw = (s["dw_q"], s["dw_k"]) if c["norm"] else (None, None)
            rsq.gqe_qk_rope_bwd(cfg, s["rope"], s["Q"], s["Qs"], s["K"], None, s["gQ"], s["gQs"], s["gK"], s["oQ"],
                                s["oQs"], s["oK"], *dw, s["ws"])
            return [s["oQ"], s["oQs"], s["oK"]] + [x for x in dw if x is not None]
        rsq.gqe_qk_rope(cfg, s["rope"], s["Q"], s["Qs"], s["K"], None, s["oQ"], s["oQs"], s["oK"])
        return [s["oQ"], s["oQs"], s["oK"]]
    if c["op"] == "balance":
        rsq.gqe_balance_stats(cfg, s["z"], s["idx"], s["mask"], s["counts"], s["sums"], s["ws"])
        rsq.gqe_balance_loss(cfg, s["z"], s["mask"], s["counts"], s["sums"], s["c_balance"], s["c_z"], s["loss"], s["dz"])
        return {"counts": s["counts"], "loss": s["loss"], "dz": s["dz"]}
    if c["op"] == "store":
        rsq.gqe_kv4_append(cfg, s["K"], s["V"], s["start"], None, s["cache"])
        rsq.gqe_kv4_read(cfg, s["cache"], s["start"], None, s["oK"], s["oV"])
        return [s["oK"], s["oV"]]
    rsq.gqe_kv4_attention(cfg, s["Q"], s["Qs"], s["cache"], s["lens"], s["out"], s["ws"])
    return s["out"]


# ------------------------------------------------------------------ the plain forms


def _plain_angles(s):
    """cos, sin [R, d_rot/2]: angles of far positions need 64 bits."""
    c = s["case"]
    pos = s["pos"].double()
    p = pos[s["axis"].long()].T if s["axis"] is not None else pos[0].unsqueeze(1)
    th = p * s["inv_freq"]
    return torch.cos(th).float(), torch.sin(th).float()


def _plain_split(n, rot, pairs):
    if pairs == "half":
        return n[..., : rot // 2], n[..., rot // 2: rot]
    return n[..., 0:rot:2], n[..., 1:rot:2]


def _plain_join(a, b, rest, pairs):
    r = torch.cat([a, b], -1) if pairs == "half" else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([r, rest], -1)


def _plain_rope(s):
    c = s["case"]
    B, T, rot = c["B"], c["T"], c["rot"]
    cos, sin = _plain_angles(s)
    out, dws = [], {}
    for name in ("Q", "Qs", "K"):
        x = s[name].float()
        lead = (B,) + (1,) * (x.dim() - 3) + (T, -1)
        cs, sn = cos.view(lead), sin.view(lead)
        w = s["w_k"] if name == "K" else s["w_q"]
        if c["norm"]:
            rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"])
            xh = x * rstd
        if not c["grad"]:
            n = xh * w if c["norm"] else x
            a, b = _plain_split(n, rot, c["pairs"])
            out.append(_plain_join(a * cs - b * sn, a * sn + b * cs, n[..., rot:], c["pairs"]).to(_BF16))
            continue
        g = s["g" + name]
        a, b = _plain_split(g, rot, c["pairs"])
        gn = _plain_join(a * cs + b * sn, b * cs - a * sn, g[..., rot:], c["pairs"])
        if not c["norm"]:
            out.append(gn)
            continue
        gw = gn * w
        out.append(rstd * (gw - xh * (gw * xh).mean(-1, keepdim=True)))
        dw = (gn * xh).flatten(0, -2).sum(0)
        key = "k" if name == "K" else "q"
        dws[key] = dws[key] + dw if key in dws else dw
    return out + ([dws["q"], dws["k"]] if dws else [])


def _plain_balance(s):
    c = s["case"]
    G, M, k = c["G"], c["M"], c["k"]
    z = s["z"].view(-1, G, M)
    on = s["mask"].bool() if s["mask"] is not None else torch.ones(z.shape[0], dtype=torch.bool, device="cuda")
    onf = on.float().view(-1, 1, 1)
    n = on.sum()
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z - m)
    tot = e.sum(-1, keepdim=True)
    p = e / tot
    lse = m + torch.log(tot)
    hot = (s["idx"].unsqueeze(-1) == torch.arange(M, device="cuda", dtype=torch.int32)).any(2) & on.view(-1, 1, 1)
    counts = hot.sum(0)
    nd = n.double().clamp(min=1)
    # The loads around their mean: the softmax's gradient does not see the mean, and 32 bits would lose the rest in it.
    f = ((counts * M - k * n).double() / (M * k * nd)).float()
    P = (p * onf).double().sum(0) / nd
    load = counts.double() / (k * nd)
    bal = (M / G) * (load * P).sum()
    zl = (lse.double().square() * onf).sum() / (G * nd)
    cb, cz = s["c_balance"], s["c_z"]
    a = (cb * M / (G * nd)).float()
    b = (2 * cz / (G * nd)).float()
    dz = p * (a * (f - (p * f).sum(-1, keepdim=True)) + b * lse) * onf
    loss = torch.stack([cb * bal + cz * zl, bal, zl]).float()
    return {"counts": torch.cat([counts.flatten(), n.view(1)]).to(torch.int32), "loss": loss, "dz": dz.view(-1, G * M)}


def _plain_store(s):
    B, T = s["case"]["B"], s["case"]["T"]
    b = torch.arange(B, device="cuda").view(B, 1)
    t = s["start"].view(B, 1) + torch.arange(T, device="cuda")
    out = []
    for name, codes, at in (("K", s["k_codes"], 0), ("V", s["v_codes"], 2)):
        x = s[name].float()
        lo, hi = x.amin(-1), x.amax(-1)
        step = ((hi - lo) / 15).to(_BF16)
        zero = lo.to(_BF16)
        q = torch.round((x - zero.float().unsqueeze(-1)) / step.float().unsqueeze(-1)).clamp(0, 15)
        q = torch.where(step.unsqueeze(-1) == 0, torch.zeros_like(q), q).to(torch.uint8)
        packed = q[..., 0::2] | (q[..., 1::2] << 4)
        codes[b, :, t] = packed.transpose(1, 2)
        s["meta"][b, :, t, at] = step.transpose(1, 2)
        s["meta"][b, :, t, at + 1] = zero.transpose(1, 2)
        out.append(_plain_decode(codes[b, :, t], s["meta"][b, :, t, at], s["meta"][b, :, t, at + 1])
                   .transpose(1, 2).to(_BF16).contiguous())
    return out


def _plain_decode(codes, step, zero):
    q = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    return q * step.float().unsqueeze(-1) + zero.float().unsqueeze(-1)


def _plain_attn(s):
    c = s["case"]
    B, T, G, dh = c["B"], c["T"], c["G"], c["dh"]
    K = _plain_decode(s["k_codes"][:, :, :T], s["meta"][:, :, :T, 0], s["meta"][:, :, :T, 1])
    V = _plain_decode(s["v_codes"][:, :, :T], s["meta"][:, :, :T, 2], s["meta"][:, :, :T, 3])
    dead = (torch.arange(T, device="cuda") >= s["lens"].view(B, 1)).view(B, 1, 1, T)
    out = []
    for q, g in ((s["Q"].float(), G), (None if s["Qs"] is None else s["Qs"].float().view(B, 1, 1, dh), 1)):
        if q is None:
            continue
        sc = (torch.matmul(q, K[:, :g].transpose(2, 3)) / math.sqrt(dh)).masked_fill(dead, -math.inf)
        m = sc.amax(-1, keepdim=True)
        e = torch.exp(sc - torch.where(m == -math.inf, torch.zeros_like(m), m))
        tot = e.sum(-1, keepdim=True)
        p = e / torch.where(tot == 0, torch.ones_like(tot), tot)
        out.append(torch.matmul(p, V[:, :g]).reshape(B, -1))
    return torch.cat(out, -1).to(_BF16)


def run(state):
    if own:
        return _run_own(state)
    return {"rope": _plain_rope, "balance": _plain_balance, "store": _plain_store, "attn": _plain_attn}[state["case"]["op"]](state)


# ------------------------------------------------------------------ the definition in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "balance": _exact_balance, "store": _exact_store, "attn": _exact_attn}[case["op"]](s)


def _exact_rope(s):
    """The rotation as one complex product per pair; gradients by automatic differentiation of that."""
    c = s["case"]
    B, T, rot, h = c["B"], c["T"], c["rot"], c["rot"] // 2
    pos = s["pos"].to(torch.float64)
    axis = s["axis"].long() if s["axis"] is not None else torch.zeros(h, dtype=torch.long, device="cuda")
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos[axis].T * s["inv_freq"]).view(B, T, h)
    order = torch.arange(rot, device="cuda")
    order = order.view(2, h).T.reshape(-1) if c["pairs"] == "half" else order  # the dims of the pairs, pair by pair
    weights = [s[n].double().requires_grad_(c["grad"]) if c["norm"] else None for n in ("w_q", "w_k")]
    outs, dws = [], [None, None]
    for name, wi in (("Q", 0), ("Qs", 0), ("K", 1)):
        heads = s[name].reshape(B, -1, T, c["dh"])
        parts = []
        for j in range(heads.shape[1]):  # a head at a time: 64 bits take room
            x = heads[:, j].double().requires_grad_(c["grad"])
            y = x
            if c["norm"]:
                y = x / torch.sqrt(torch.sum(x ** 2, -1, keepdim=True) / c["dh"] + s["eps"]) * weights[wi]
            if rot:
                pair = torch.view_as_complex(y[..., order].reshape(B, T, h, 2).contiguous())
                turned = torch.view_as_real(pair * turn).reshape(B, T, rot)
                y = torch.cat([turned[..., torch.argsort(order)], y[..., rot:]], -1)
            if c["grad"]:
                g = s["g" + name].reshape(B, -1, T, c["dh"])[:, j].double()
                want = [x] + ([weights[wi]] if c["norm"] else [])
                got = torch.autograd.grad(y, want, g) if (c["norm"] or rot) else [g]
                parts.append(got[0])
                if c["norm"]:
                    dws[wi] = got[1] if dws[wi] is None else dws[wi] + got[1]
            else:
                parts.append(y)
        outs.append(torch.stack(parts, 1).view(s[name].shape).detach())
    return outs + ([d.detach() for d in dws] if c["grad"] and c["norm"] else [])


def _exact_balance(s):
    c = s["case"]
    G, M, k = c["G"], c["M"], c["k"]
    rows = torch.nonzero(s["mask"]).view(-1) if s["mask"] is not None else torch.arange(s["z"].shape[0], device="cuda")
    z = s["z"].double().requires_grad_(True)
    n = rows.numel()
    counts = torch.stack([torch.bincount(s["idx"][rows][:, g].reshape(-1).long(), minlength=M) for g in range(G)])
    if n == 0:
        zero = torch.zeros(3, dtype=torch.float64, device="cuda")
        return {"counts": torch.cat([counts.view(-1), counts.new_zeros(1)]).to(torch.int32), "loss": zero,
                "dz": torch.zeros_like(z)}
    zr = z[rows].view(n, G, M)
    bal = M / G * ((counts.double() / (k * n)) * torch.softmax(zr, -1).mean(0)).sum()
    zl = torch.logsumexp(zr, -1).pow(2).mean()
    total = s["c_balance"] * bal + s["c_z"] * zl
    dz, = torch.autograd.grad(total, z)
    return {"counts": torch.cat([counts.view(-1), counts.new_full((1,), n)]).to(torch.int32),
            "loss": torch.stack([total, bal, zl]).detach(), "dz": dz}


def _exact_store(s):
    """The stored values: whole steps over the row's least value, the step rounded to bf16 (part of the format)."""
    got = []
    for x in (s["K"], s["V"]):
        x = x.double()
        low = x.min(-1, keepdim=True).values
        step = ((x.max(-1, keepdim=True).values - low) / 15).float().to(_BF16).double()
        whole = torch.clamp(torch.round((x - low) / torch.where(step > 0, step, torch.ones_like(step))), 0, 15)
        got.append(low + step * whole)
    return got


def _exact_attn(s):
    c = s["case"]
    B, G, dh = c["B"], c["G"], c["dh"]
    out = torch.zeros(B, s["out"].shape[1] // dh, dh, dtype=torch.float64, device="cuda")
    per = s["Q"].shape[2]
    shifts = torch.tensor([0, 4], device="cuda")
    for b, n in enumerate(_lens(c)):
        if n == 0:
            continue
        meta = s["meta"][b, :, :n].double()
        K, V = (((codes[b, :, :n].int().unsqueeze(-1) >> shifts) & 15).reshape(G, n, dh).double() * meta[..., i: i + 1]
                + meta[..., i + 1: i + 2] for codes, i in ((s["k_codes"], 0), (s["v_codes"], 2)))
        for g in range(G):
            q = s["Q"][b, g].double()
            shared = g == 0 and s["Qs"] is not None
            if shared:
                q = torch.cat([q, s["Qs"][b: b + 1].double()])
            o = torch.softmax(q @ K[g].T * dh ** -0.5, -1) @ V[g]
            out[b, g * per: (g + 1) * per] = o[:per]
            if shared:
                out[b, G * per] = o[per]
    return out.view(B, -1)
