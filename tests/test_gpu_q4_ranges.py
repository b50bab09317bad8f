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


# ---------------------------------------------------------------------------------------------
# attention over values of very different sizes
# ---------------------------------------------------------------------------------------------
# A weight is off by at most 2^-22 of itself, and by 2^-34 of the largest scale of V among the 16 keys beside it in
# its group of 64 dims (2^-45 of the 32 keys with at most 4 query rows a KV head), where the largest probability is at
# least 1.  The first is within ROW_REL.  The second moves each dim of the output by at most
# 8 (the largest |u - 8|) x the tile's keys x 2^-34 S / Z, Z = sum exp(s - max s): slack() below, 8 = sqrt(64) times that
# for the 64 dims of a group together.
ROWS = [(2, 1, "bf16"), (4, 1, "f32"), (8, 1, "bf16"), (2, 8, "f32"), (16, 1, "bf16")]


def run_decode(K, k, v, q, q_dt, L):
    """kv_attn_decode_q4 over the quantised k, v [1,1,W,D] and the float64 result, both [T,Hq,D] on the host, and
    Z of each row [T,Hq]."""
    torch = _torch()
    pk, pv = Q.q4_quantise(k), Q.q4_quantise(v)
    T, Hq, D = q.shape
    lengths = np.array([L], np.int32)
    qd = dev(q.astype(np.float32), dt(q_dt))[None]
    out = torch.full((1, T, Hq, v.shape[-1]), float("nan"), device="cuda")
    ws = torch.zeros(K.decode_q4_workspace_bytes(1, k.shape[1], Hq, T, L, v.shape[-1]), dtype=torch.uint8, device="cuda")
    K.kv_attn_decode_q4(qd, filled(K, *pk, *pv), dev(lengths), lengths, out, ws)
    torch.cuda.synchronize()
    ref = attend(qd[0].double(), dev(Q.q4_values(*pk)[0]), dev(Q.q4_values(*pv)[0]), L)
    s = np.einsum("thd,jd->thj", host(qd[0]), Q.q4_values(*pk)[0, 0, :L]) / math.sqrt(D)
    s = np.where(np.arange(L) < (L - T + 1 + np.arange(T))[:, None, None], s, -np.inf)
    return host(out[0]), host(ref), np.exp(s - s.max(-1, keepdims=True)).sum(-1)


def grouped(x):
    return x.reshape(*x.shape[:-1], -1, 64)


def slack(v, at, z):
    """What the scales of slot `at` of v [1,1,W,D] may move the groups of the rows by, [T,Hq,groups]."""
    few = z.size <= 4
    S = Q.q4_quantise(v[0, 0, at])[1]
    return 8.0 * 8.0 * (32 if few else 16) * 2.0 ** (-45 if few else -34) * S / z[..., None]


def assert_groups_close(got, ref, more=0.0):
    err = np.linalg.norm(grouped(got) - grouped(ref), axis=-1)
    assert np.all(err <= ROW_REL * np.linalg.norm(grouped(ref), axis=-1) + more), np.max(err / np.linalg.norm(grouped(ref), axis=-1))


@pytest.mark.parametrize("power", [-20, 20, 60])
@pytest.mark.parametrize("G,T,q_dt", ROWS)
def test_decode_groups_of_different_sizes(K, G, T, q_dt, power):
    """The second 64 dims of V are 2^power times the first: each group is as precise as it would be alone."""
    rng = seeded("groups", G, T, power)
    L, W, D = 1203, 1204, 128
    k, v = rng.standard_normal((1, 1, W, D)), rng.standard_normal((1, 1, W, D))
    v[..., 64:] *= 2.0 ** power
    got, ref, _ = run_decode(K, k, v, rng.standard_normal((T, G, D)), q_dt, L)
    assert_groups_close(got, ref)


@pytest.mark.parametrize("at", [0, 600, 1202])
@pytest.mark.parametrize("G,T,q_dt", ROWS)
def test_decode_a_huge_value_that_no_token_attends(K, G, T, q_dt, at):
    """One slot's V is 2^20 times the others' and its score, below -45, so low that its weight
    vanishes: e^-45 2^20 is 2^-45 of one value, 2^-35 of the sum of 1200."""
    rng = seeded("outlier", G, T, at)
    L, W, D = 1203, 1204, 128
    k, v = rng.standard_normal((1, 1, W, D)), rng.standard_normal((1, 1, W, D))
    v[0, 0, at] *= 2.0 ** 20
    k[0, 0, at] = -8.0
    q = np.abs(rng.standard_normal((T, G, D)))                 # the slot's score is -8 sum(q) / sqrt(D), about -72
    assert q.sum(-1).min() * 8 / math.sqrt(D) > 45
    got, ref, z = run_decode(K, k, v, q, q_dt, L)
    assert_groups_close(got, ref, slack(v, at, z))


@pytest.mark.parametrize("G,T,q_dt", [(1, 3, "f32"), (2, 8, "bf16"), (1, 16, "f32")])
def test_decode_a_huge_value_that_earlier_tokens_do_not_see(K, G, T, q_dt):
    """The last token of a block has a V 2^20 times the others': the tokens before it keep their precision."""
    rng = seeded("hidden", G, T)
    L, W, D = 1203, 1204, 128
    k, v = rng.standard_normal((1, 1, W, D)), rng.standard_normal((1, 1, W, D))
    v[0, 0, L - 1] *= 2.0 ** 20
    got, ref, z = run_decode(K, k, v, rng.standard_normal((T, G, D)), q_dt, L)
    assert_groups_close(got, ref, slack(v, L - 1, z))


@pytest.mark.parametrize("G,T,q_dt,lead", [(2, 1, "bf16", 13.0), (4, 1, "f32", 13.0), (8, 1, "bf16", 8.0), (2, 8, "f32", 8.0)])
def test_decode_a_leading_key_with_a_tiny_value(K, G, T, q_dt, lead):
    """One key takes nearly all the weight and its V is 2^-20 of the others': the output is the others', whose
    weights are about e^-lead.  At lead 8 (2^-12) the floor 2^-34 is 2^-22 of such a weight; at 13 (2^-19), with
    at most 4 rows, 2^-45 is 2^-26 of it."""
    rng = seeded("sink", G, T)
    L, W, D = 1203, 1204, 128
    k, v = 0.3 * rng.standard_normal((1, 1, W, D)), rng.standard_normal((1, 1, W, D))
    v[0, 0, 3] *= 2.0 ** -20
    q = np.abs(rng.standard_normal((T, G, D)))
    q *= 100.0 / q.sum(-1, keepdims=True)                      # every row's elements sum to 100 (before rounding)
    k[0, 0, 3] = lead * math.sqrt(D) / 100.0
    got, ref, _ = run_decode(K, k, v, q, q_dt, L)
    assert_groups_close(got, ref)


@pytest.mark.parametrize("G,T,q_dt", ROWS)
def test_decode_tiles_of_huge_values_that_no_token_attends(K, G, T, q_dt):
    """The first 128 slots, a tile of each warp, are such slots: the tiles after them keep their precision.  1300
    copies of the sequence, so that one CTA walks all of it."""
    torch = _torch()
    rng = seeded("tiles", G, T)
    L, W, D, copies = 515, 516, 128, 1300
    k, v = rng.standard_normal((1, 1, W, D)), rng.standard_normal((1, 1, W, D))
    v[0, 0, :128] *= 2.0 ** 20
    k[0, 0, :128] = -8.0
    q = np.abs(rng.standard_normal((T, G, D)))
    assert q.sum(-1).min() * 8 / math.sqrt(D) > 45             # 128 e^-45 2^20 is 2^-27 of the sum of 387
    pk, pv = Q.q4_quantise(k), Q.q4_quantise(v)
    one = filled(K, *pk, *pv)
    cache = K.KVCacheQ4(*(t.expand(copies, *t.shape[1:]).contiguous() for t in (one.k, one.v, one.k_scale, one.v_scale)))
    lengths = np.full(copies, L, np.int32)
    qd = dev(q.astype(np.float32), dt(q_dt)).expand(copies, T, G, D).contiguous()
    out = torch.full((copies, T, G, D), float("nan"), device="cuda")
    ws = torch.zeros(K.decode_q4_workspace_bytes(copies, 1, G, T, L, D), dtype=torch.uint8, device="cuda")
    K.kv_attn_decode_q4(qd, cache, dev(lengths), lengths, out, ws)
    torch.cuda.synchronize()
    assert bool((out == out[:1]).all())
    ref = attend(qd[0].double(), dev(Q.q4_values(*pk)[0]), dev(Q.q4_values(*pv)[0]), L)
    assert_groups_close(host(out[0]), host(ref))
