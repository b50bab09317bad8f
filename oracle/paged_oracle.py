"""Plain fp64 definitions of the paged cache, of attention over it, and of beam search's steps.

TEST INFRASTRUCTURE, like kv_oracle: it shares no code with the CUDA library.  The pages that the
library goes by keep fixed windows and pick tokens greedily; these are the definitions that
include/kv_attn.h states.
"""
from __future__ import annotations

import math

import numpy as np

from .kv_oracle import F64, Rope, inv_freq, rms_norm, rope_apply, rotate_half_apply, store


def scaled_inv(inv, factor: float, orig_len: float, low: float, high: float):
    """Frequencies for longer contexts: slow ones divided by `factor`, fast ones kept, a ramp between."""
    out = []
    for w in np.asarray(inv, F64):
        keep = 0.0
        if orig_len > 0:
            turns = orig_len * w / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - low) / (high - low)))
        out.append(w * keep + w / factor * (1 - keep))
    return np.array(out, F64)


def rope_scaled(x, pos, rope: Rope, scale=None):
    """rope_apply with scaled frequencies; scale = (factor, orig_len, low, high, magnitude) or None."""
    if scale is None or rope.kind == "none":
        return rope_apply(x, pos, rope)
    x, pos = np.asarray(x, F64), np.asarray(pos, F64)
    factor, orig, low, high, mag = scale
    out = x.copy()
    o = rope.rot_offset
    w = rope.rot_dim or x.shape[-1]
    part = x[..., o:o + w]
    if rope.kind == "interleaved":
        part = np.concatenate([part[..., 0::2], part[..., 1::2]], -1)
    blocks = 2 if rope.kind == "2d" else 1
    wb = w // blocks
    inv = scaled_inv(inv_freq(rope.base, wb), factor, orig, low, high)
    for b in range(blocks):
        if rope.kind == "sections":
            axis = np.repeat(np.arange(len(rope.sections)), rope.sections)
        else:
            axis = np.full(wb // 2, b)
        ang = pos[:, axis] * inv
        out[..., o + b * wb:o + (b + 1) * wb] = mag * rotate_half_apply(part[..., b * wb:(b + 1) * wb], ang[:, None, :])
    return out


def qk_step(x, pos, w, eps, rope, scale, after):
    """QK-Norm and (scaled) RoPE of x [T, H, D] in either order; w None: no norm."""
    x = np.asarray(x, F64)
    if w is not None and not after:
        x = rms_norm(x, w, eps)
    x = rope_scaled(x, pos, rope, scale)
    return rms_norm(x, w, eps) if w is not None and after else x


def paged_append(k, v, pool_k, pool_v, table, lengths, start, dtype):
    """Writes transformed keys k [T, Hkv, Dk] and values v into pools [pages, Hkv, page, D], in place."""
    page = pool_k.shape[2]
    for b in range(len(lengths)):
        n = start[b + 1] - start[b]
        for i in range(n):
            slot = lengths[b] - n + i
            if slot >= 0:
                p, r = table[b][slot // page], slot % page
                pool_k[p, :, r] = store(k[start[b] + i], dtype)
                pool_v[p, :, r] = store(v[start[b] + i], dtype)


def paged_rows(pool, table_row, L):
    """[Hkv, L, D] rows of a sequence's slots."""
    page = pool.shape[2]
    if L == 0:
        return np.zeros((pool.shape[1], 0, pool.shape[3]))
    return np.stack([pool[table_row[s // page], :, s % page] for s in range(L)], 1)


def paged_attention(q, pool_k, pool_v, table, lengths, start, scale=None):
    """o [T, Hq, Dv] and the sums of weight * |value|, the scale of a weight's rounding."""
    q, T, Hq = np.asarray(q, F64), len(q), q.shape[1]
    Hkv, Dk, Dv = pool_k.shape[1], pool_k.shape[3], pool_v.shape[3]
    scale = 1 / math.sqrt(Dk) if scale is None else scale
    out, size = np.zeros((T, Hq, Dv)), np.zeros((T, Hq, Dv))
    for b in range(len(lengths)):
        n, L = start[b + 1] - start[b], max(0, lengths[b])
        if n == 0:
            continue
        K, V = paged_rows(pool_k, table[b], L), paged_rows(pool_v, table[b], L)
        for i in range(n):
            sees = L - n + i + 1
            if sees <= 0:
                continue
            for h in range(Hq):
                g = h // (Hq // Hkv)
                x = K[g, :sees] @ q[start[b] + i, h] * scale
                e = np.exp(x - x.max())
                out[start[b] + i, h] = e @ V[g, :sees] / e.sum()
                size[start[b] + i, h] = e @ np.abs(V[g, :sees]) / e.sum()
    return out, size


def beam_step(logits, scores, n, finished=None, end_id=0):
    """The n best (beam, token, total) of each group, equal totals toward the lower beam, then the lower token."""
    B, K, V = logits.shape
    res = []
    for b in range(B):
        offers = []
        for k in range(K):
            s = float(scores[b, k])
            if finished is not None and finished[b, k]:
                if math.isfinite(s):
                    offers.append((-s, k, end_id))
                continue
            z = np.asarray(logits[b, k], F64)
            if not math.isfinite(s) or np.isnan(z).any() or (z == math.inf).any() or not (z > -math.inf).any():
                continue
            m = z.max()
            total = s + (z - m - math.log(np.exp(z - m).sum()))
            best = np.lexsort((np.arange(V), -total))[:n]
            offers += [(-total[t], k, int(t)) for t in best if total[t] > -math.inf]
        offers = sorted(offers)[:n]
        res.append([(k, t, -u) for u, k, t in offers] + [(-1, -1, -math.inf)] * (n - len(offers)))
    return res


def reorder(parent, table, lengths, spare, pools, n_pages):
    """Beams go on from their parents.  table [B, K, W], pools: arrays [layers, pages, Hkv, page, D] changed in place.
    Returns rows (lists of page ids), lengths and spares."""
    B, K, page = len(parent), len(parent[0]), pools[0].shape[3]
    rows_out, len_out, spare_out = [], [], []
    for b in range(B):
        tails = [table[b][j][lengths[b][j] // page] if lengths[b][j] % page else None for j in range(K)]
        carried, used = set(), []
        rows, lens, spares = [], [], list(spare[b])
        before = [p.copy() for p in pools]
        for k in range(K):
            p = parent[b][k]
            if not 0 <= p < K:
                rows.append([])
                lens.append(0)
                continue
            L = lengths[b][p]
            row = [int(x) for x in table[b][p][:-(-L // page)]]
            if tails[p] is not None:
                if tails[p] in carried:
                    if not (0 <= spare[b][k] < n_pages and 0 <= tails[p] < n_pages):
                        rows.append([])
                        lens.append(-1)
                        used.append((k, False))
                        continue
                    for pool, old in zip(pools, before):
                        pool[:, spare[b][k], :, :L % page] = old[:, tails[p], :, :L % page]
                    row[-1] = int(spare[b][k])
                    used.append((k, True))
                carried.add(tails[p])
            rows.append(row)
            lens.append(L)
        freed = []
        for t in tails:
            if t is not None and t not in carried and t not in freed:
                freed.append(t)
        for i, (k, done) in enumerate(used):
            if done:
                spares[k] = freed[i] if i < len(freed) else -1
        rows_out.append(rows)
        len_out.append(lens)
        spare_out.append(spares)
    return rows_out, len_out, spare_out
