"""Plain definitions, in fp64 numpy, of the operators around the layer: the
norm and rotation of queries and keys, the router's balance loss, and the
4-bit K/V cache.

TEST INFRASTRUCTURE, under the same rules as the rest of ``oracle``: only the
tests may call it, the CUDA library never does, and it shares no code with it.
The pages have no counterpart (their layer has no positions, their balancing
loss comes without a formula, their cache is bf16); the definitions are the
ones ``include/gqe.h`` states.
"""
from __future__ import annotations

import math

import numpy as np


# ---------------------------------------------------------------- norm and rotation

def rope_angles(pos: np.ndarray, inv_freq: np.ndarray, axis: np.ndarray | None) -> np.ndarray:
    """[tokens, d_rot/2] angles; pos [axes, tokens]."""
    a = np.zeros(len(inv_freq), dtype=np.int64) if axis is None else np.asarray(axis, dtype=np.int64)
    return pos[a].T.astype(np.float64) * inv_freq


def _pairs(d_rot: int, adjacent: bool):
    i = np.arange(d_rot // 2)
    return (2 * i, 2 * i + 1) if adjacent else (i, i + d_rot // 2)


def rope_norm(x, w, eps):
    """w * x / sqrt(mean(x^2) + eps) over the last axis."""
    return w * x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)


def rope(x: np.ndarray, angles: np.ndarray, *, norm: bool, w=1.0, eps=0.0, scale=1.0, adjacent=False) -> np.ndarray:
    """x [..., tokens, dh] (fp64), angles [tokens, d_rot/2]."""
    y = rope_norm(x, w, eps) if norm else x.copy()
    ia, ib = _pairs(2 * angles.shape[1], adjacent)
    a, b = y[..., ia].copy(), y[..., ib].copy()
    c, s = np.cos(angles) * scale, np.sin(angles) * scale
    y[..., ia] = a * c - b * s
    y[..., ib] = a * s + b * c
    return y


def rope_backward(x, g, angles, *, norm: bool, w=1.0, eps=0.0, scale=1.0, adjacent=False):
    """(dx, dw): dw [dh] summed over every row, None without the norm."""
    g = g.copy()
    ia, ib = _pairs(2 * angles.shape[1], adjacent)
    a, b = g[..., ia].copy(), g[..., ib].copy()
    c, s = np.cos(angles) * scale, np.sin(angles) * scale
    g[..., ia] = a * c + b * s
    g[..., ib] = -a * s + b * c
    if not norm:
        return g, None
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    # n_i = w_i x_i r, dr/dx_j = -r^3 x_j / dh
    dw = (g * x * r).reshape(-1, x.shape[-1]).sum(axis=0)
    inner = np.sum(g * w * x, axis=-1, keepdims=True)
    return g * w * r - x * r ** 3 * inner / x.shape[-1], dw


# ---------------------------------------------------------------- balance loss

def balance(z: np.ndarray, idx: np.ndarray, mask, G: int, M: int, c_balance: float, c_z: float) -> dict:
    """z [R, G*M] fp64, idx [R, G, k], mask [R] or None."""
    R, k = z.shape[0], idx.shape[2]
    on = np.ones(R, dtype=bool) if mask is None else np.asarray(mask) != 0
    counts = np.zeros((G, M), dtype=np.int64)
    psum = np.zeros((G, M))
    zsum = 0.0
    dz = np.zeros((R, G, M))
    n = int(on.sum())
    out = {"counts": counts, "psum": psum, "n": n}
    rows = np.nonzero(on)[0]
    zz = z.reshape(R, G, M)[rows]
    m = zz.max(axis=-1, keepdims=True) if n else zz
    e = np.exp(zz - m)
    p = e / e.sum(axis=-1, keepdims=True)
    lse = (m + np.log(e.sum(axis=-1, keepdims=True)))[..., 0]
    for g in range(G):
        for j in range(M):
            counts[g, j] = int(np.sum(idx[rows, g] == j))
    if n:
        psum += p.sum(axis=0)
        zsum = float((lse ** 2).sum())
        f = counts / (k * n)
        bal = M / G * float((f * psum / n).sum())
        zl = zsum / (n * G)
        d = c_balance * M / (G * n) * p * (f - (p * f).sum(axis=-1, keepdims=True))
        d += c_z * 2.0 / (n * G) * lse[..., None] * p
        dz[rows] = d
    else:
        bal = zl = 0.0
    out.update(zsum=zsum, loss=np.array([c_balance * bal + c_z * zl, bal, zl]), dz=dz.reshape(R, G * M), p=p, lse=lse)
    return out


# ---------------------------------------------------------------- 4-bit cache

def bf16_round(a: np.ndarray) -> np.ndarray:
    """fp32 -> nearest bf16 (ties to even), as fp32 values."""
    b = np.ascontiguousarray(a, dtype=np.float32).view(np.uint32)
    r = (b + np.uint32(0x7FFF) + ((b >> np.uint32(16)) & np.uint32(1))) & np.uint32(0xFFFF0000)
    return r.view(np.float32)


def kv4_quantise(x: np.ndarray):
    """(codes, scale, zero) of rows x [..., dh] of bf16 values; the format's
    arithmetic is single IEEE fp32 operations. Rows with an infinity or NaN:
    NaN scale and zero, codes 0."""
    x = x.astype(np.float32)
    bad = ~np.isfinite(x).all(axis=-1)
    xs = np.where(bad[..., None], np.float32(0), x)
    lo, hi = xs.min(axis=-1), xs.max(axis=-1)
    half = np.float32(0.5)
    scale = bf16_round((half * hi - half * lo) / np.float32(7.5))
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.rint((half * xs - half * lo[..., None]) / (half * scale[..., None]))
    codes = np.where(scale[..., None] > 0, np.clip(q, 0, 15), 0)
    nan = np.float32(np.nan)
    return codes.astype(np.uint8), np.where(bad, nan, scale), np.where(bad, nan, lo)


def kv4_values(codes, scale, zero) -> np.ndarray:
    return zero.astype(np.float64)[..., None] + scale.astype(np.float64)[..., None] * codes


def kv4_pack(codes: np.ndarray) -> np.ndarray:
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def kv4_unpack(packed: np.ndarray) -> np.ndarray:
    return np.stack([packed & 15, packed >> 4], axis=-1).reshape(*packed.shape[:-1], -1)


def decode_attention(q: np.ndarray, K: np.ndarray, V: np.ndarray) -> np.ndarray:
    """softmax(q K^T / sqrt(dh)) V for heads q [h, dh] over n >= 0 keys."""
    if K.shape[0] == 0:
        return np.zeros_like(q)
    s = q @ K.T / math.sqrt(q.shape[-1])
    e = np.exp(s - s.max(axis=-1, keepdims=True))
    return (e / e.sum(axis=-1, keepdims=True)) @ V
