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
