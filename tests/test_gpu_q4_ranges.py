"""The 4-bit cache calls over the rest of the range that they accept: shapes that change on one
workspace, long blocks, long appends, far positions, values of very different sizes.  Against the
float64 definitions in oracle/q4_oracle.py; attention in plain float64 products."""
import math
import zlib

import numpy as np
import pytest

import oracle as O
from helpers import dev, host, row_rel_err
from oracle import q4_oracle as Q
from test_gpu_q4_cache import ROW_REL, dt, filled, random_q4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from kv_cache_gqa_gb300 import build
    build.build_library(verbose=False)
    import kv_cache_gqa_gb300 as K
    return K


def _torch():
    import torch
    return torch


def seeded(*key):
    return np.random.default_rng(zlib.crc32(repr(key).encode()))


def attend(q, k, v, L):
    """q [T,Hq,Dk] over k [Hkv,W,Dk], v [Hkv,W,Dv] (float64, on the GPU): token i sees slots 0 .. L-T+i."""
    torch = _torch()
    T, Hq, Dk = q.shape
    Hkv = k.shape[0]
    G = Hq // Hkv
    rows = q.view(T, Hkv, G, Dk).permute(1, 0, 2, 3).reshape(Hkv, T * G, Dk)
    s = rows @ k[:, :L].transpose(1, 2) / math.sqrt(Dk)
    seen = L - T + 1 + torch.arange(T, device=s.device).repeat_interleave(G)
    s = s.masked_fill(torch.arange(L, device=s.device)[None, None, :] >= seen[None, :, None], -math.inf)
    p = torch.softmax(s, -1).nan_to_num(0.0)                   # rows that see nothing: zeros
    o = p @ v[:, :L]
    return o.view(Hkv, T, G, -1).permute(1, 0, 2, 3).reshape(T, Hq, -1)


# ---------------------------------------------------------------------------------------------
# one workspace, several shapes
# ---------------------------------------------------------------------------------------------
def test_tokens_and_draft_blocks_share_a_workspace(K):
    """A workspace sized for the longest block and zeroed once, then single tokens and blocks of 16 and 40 in
    turn, over 8 sequences and over one: units are joined over CTAs in every call."""
    torch = _torch()
    rng = seeded("share")
    B, Hkv, G, D, W = 8, 8, 2, 128, 1200
    Hq = Hkv * G
    pk, pv = random_q4(rng, B, Hkv, W, D), random_q4(rng, B, Hkv, W, D)
    cache = filled(K, *pk, *pv)
    vk, vv = dev(Q.q4_values(*pk)), dev(Q.q4_values(*pv))
    lengths = np.array([1200, 1000, 1111, 800, 77, 1200, 950, 1199], np.int32)
    zero = K.lib().kva_decode_q4_workspace_zero_bytes(B, Hkv, Hq, 40)
    ws = torch.zeros(K.decode_q4_workspace_bytes(B, Hkv, Hq, 40, W, D), dtype=torch.uint8, device="cuda")
    for n, T in ((8, 1), (8, 16), (8, 1), (1, 40), (8, 40), (1, 1), (8, 16)):
        q = dev(rng.standard_normal((n, T, Hq, D)).astype(np.float32), torch.bfloat16)
        out = torch.full((n, T, Hq, D), float("nan"), device="cuda")
        K.kv_attn_decode_q4(q, cache, dev(lengths[:n]), lengths[:n], out, ws)
        torch.cuda.synchronize()
        assert int(ws[:zero].sum()) == 0
        for b in range(n):
            ref = attend(q[b].double(), vk[b], vv[b], int(lengths[b]))
            assert row_rel_err(host(out[b]), host(ref)) <= ROW_REL, f"n={n} T={T} b={b}"


# ---------------------------------------------------------------------------------------------
# append and read-back
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("in_dt", ["f32", "bf16"])
def test_groups_of_huge_values_whose_spread_is_finite(K, in_dt):
    """Values up to 1.6e38 of either sign: their sums overflow, their spread does not.  The elements are
    their groups' ends, far from a tie between codes, so a value read back is the definition's rounded to float32."""
    torch = _torch()
    T, D = 6, 128
    x = np.zeros((1, T, 1, D), np.float64)
    big = float(O.bf16_round(np.float64(1.6e38)))
    sign = np.where(np.arange(D) % 2 == 0, 1.0, -1.0)
    x[0, 0, 0] = big * sign                                    # a lane's even elements positive, its odd ones negative
    x[0, 1, 0] = big * np.where(np.arange(D) % 8 < 4, 1.0, -1.0)
    x[0, 2, 0] = 1.0e38 * sign
    x[0, 3, 0, :64] = 0.9e38 * sign[:64]                       # huge beside small
    x[0, 3, 0, 64:] = sign[64:]
    x[0, 4, 0] = 2.0e38                                        # equal values whose sum overflows
    x[0, 5, 0, :] = -1.6e38
    x[0, 5, 0, ::2] = 0.0
    x = O.store(x, in_dt)
    slot = np.arange(T, dtype=np.int32)
    cache = K.KVCacheQ4.zeros(1, 1, 8, D)
    xd = dev(x.astype(np.float32), dt(in_dt))
    K.kv_cache_append_q4(None, xd, xd, None, dev(slot), slot, cache, None, K.Rope("none"))
    out = K.KVCache(*(torch.zeros((1, 1, T, D), device="cuda") for _ in range(2)))
    K.kv_cache_expand_q4(cache, dev(slot), slot, out)
    torch.cuda.synchronize()
    u, scale, mid = Q.q4_quantise(x[0, :, 0])
    assert np.all(np.isfinite(scale))
    want = Q.q4_values(u, scale, mid)
    for t in (out.k, out.v):
        got = host(t)[0, 0]
        assert np.all(np.isfinite(got))
        assert np.max(np.abs(got - want)) <= 2.0 ** -24 * np.abs(want).max()
