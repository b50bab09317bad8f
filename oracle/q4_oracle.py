"""Plain fp64 definitions of the 4-bit cache, of attention over it and of the vocabulary scoring.

TEST INFRASTRUCTURE, like kv_oracle: it shares no code with the CUDA library.  The pages hold
caches in 16 or 32 bits and pick tokens greedily; the quantiser and the scoring below are the
definitions that include/kv_attn.h states.
"""
from __future__ import annotations

import math

import numpy as np

from .kv_oracle import F64, bf16_round

GROUP = 64


def bf16_up(x) -> np.ndarray:
    """Smallest bfloat16 value not below x (finite x)."""
    x = np.asarray(x, F64)
    m, e = np.frexp(x)
    return np.where(x == 0, 0.0, np.ldexp(np.ceil(m * 256.0), e - 8))


def q4_quantise(x):
    """x [.., D] -> codes u [.., D/64, 64] (0..15), scale [.., D/64], mid [.., D/64]."""
    g = np.asarray(x, F64)
    g = g.reshape(*g.shape[:-1], -1, GROUP)
    bad = ~np.all(np.isfinite(g), -1)
    g = np.where(bad[..., None], 0.0, g)
    lo, hi = g.min(-1), g.max(-1)
    scale = bf16_up((hi - lo) / 15.0)
    scale = np.where(scale < 2.0 ** -126, 0.0, scale)
    mid = bf16_round(lo + 8.0 * scale)
    q = (g - mid[..., None]) / np.where(scale > 0, scale, 1.0)[..., None]
    u = np.where((scale > 0)[..., None], np.clip(np.round(q), -8, 7), 0.0) + 8
    scale, mid = np.where(bad, np.nan, scale), np.where(bad, np.nan, mid)
    return u.astype(np.int64), scale, mid


def q4_values(u, scale, mid):
    """[.., D] values of codes [.., G, 64]."""
    v = np.asarray(scale, F64)[..., None] * (np.asarray(u, F64) - 8.0) + np.asarray(mid, F64)[..., None]
    return v.reshape(*v.shape[:-2], -1)


def q4_pack(u) -> np.ndarray:
    """Codes [.., G, 64] -> bytes [.., 32 G]: 32-bit little-endian words, word w = dims
    64 * (w % G) + 8 * (w // G) + 0..7, lowest dim in the lowest 4 bits."""
    u = np.asarray(u)
    G = u.shape[-2]
    out = np.zeros(u.shape[:-2] + (8 * G,), np.uint32)
    for w in range(8 * G):
        for i in range(8):
            out[..., w] |= u[..., w % G, 8 * (w // G) + i].astype(np.uint32) << np.uint32(4 * i)
    return out.astype("<u4").view(np.uint8)


def q4_unpack(b) -> np.ndarray:
    """Inverse of q4_pack."""
    w = np.ascontiguousarray(b).view("<u4")
    G = w.shape[-1] // 8
    u = np.zeros(w.shape[:-1] + (G, GROUP), np.int64)
    for j in range(8 * G):
        for i in range(8):
            u[..., j % G, 8 * (j // G) + i] = (w[..., j] >> np.uint32(4 * i)) & np.uint32(15)
    return u


def attend_block(q, k, v, length: int, scale=None) -> np.ndarray:
    """q [T,Hq,Dk] over k [Hkv,W,Dk], v [Hkv,W,Dv]: token i sees slots 0 .. length-T+i; a token that
    sees none gives zeros."""
    q, k, v = (np.asarray(t, F64) for t in (q, k, v))
    T, Hq, Dk = q.shape
    G = Hq // k.shape[0]
    scale = 1.0 / math.sqrt(Dk) if scale is None else scale
    out = np.zeros((T, Hq, v.shape[-1]))
    for i in range(T):
        n = length - T + i + 1
        if n <= 0:
            continue
        for h in range(Hq):
            x = k[h // G, :n] @ q[i, h] * scale
            p = np.exp(x - x.max())
            out[i, h] = (p / p.sum()) @ v[h // G, :n]
    return out


def logprobs(h, W, V: int, targets=None, norm_w=None, eps=1e-6, top_k=0):
    """(logprob [B] or None, entropy [B], lse [B], top ids [B,k], top logprobs [B,k])."""
    h, W = np.asarray(h, F64), np.asarray(W, F64)[:V]
    if norm_w is not None:
        h = h / np.sqrt(np.mean(h * h, -1, keepdims=True) + eps) * np.asarray(norm_w, F64)
    z = h @ W.T
    m = z.max(-1, keepdims=True)
    e = np.exp(z - m)
    lse = m[:, 0] + np.log(e.sum(-1))
    p = e / e.sum(-1, keepdims=True)
    entropy = lse - (p * z).sum(-1)
    lp = None
    if targets is not None:
        lp = np.array([0.0 if t < 0 else (np.nan if t >= V else z[b, t] - lse[b]) for b, t in enumerate(targets)])
    order = np.argsort(-z, axis=-1, kind="stable")[:, :top_k]             # equal logits: lower id first
    return lp, entropy, lse, order, np.take_along_axis(z, order, -1) - lse[:, None]
