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


@pytest.mark.parametrize("G,T,q_dt", ROWS)
def test_decode_negative_scales(K, G, T, q_dt):
    """A cache that another program wrote: a value is scale * (u - 8) + mid whatever the scale's sign."""
    torch = _torch()
    rng = seeded("negative", G, T)
    L, W, D = 203, 204, 128
    pk, pv = (Q.q4_quantise(rng.standard_normal((1, 1, W, D))) for _ in range(2))
    q = dev(rng.standard_normal((1, T, G, D)).astype(np.float32), dt(q_dt))
    lengths = np.array([L], np.int32)
    ws = torch.zeros(K.decode_q4_workspace_bytes(1, 1, G, T, L, D), dtype=torch.uint8, device="cuda")
    for sign in (-np.ones((1, 1, W, 2)), np.where(rng.random((1, 1, W, 2)) < 0.5, -1.0, 1.0)):
        k, v = (pk[0], sign * pk[1], pk[2]), (pv[0], sign * pv[1], pv[2])
        out = torch.full((1, T, G, D), float("nan"), device="cuda")
        K.kv_attn_decode_q4(q, filled(K, *k, *v), dev(lengths), lengths, out, ws)
        torch.cuda.synchronize()
        ref = attend(q[0].double(), dev(Q.q4_values(*k)[0]), dev(Q.q4_values(*v)[0]), L)
        assert_groups_close(host(out[0]), host(ref))


# ---------------------------------------------------------------------------------------------
# long blocks and contexts
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("G,T,q_dt,Dk,Dv", [(2, 17, "bf16", 128, 128), (1, 33, "f32", 64, 64), (2, 64, "f32", 128, 128),
                                            (4, 64, "bf16", 192, 128), (3, 63, "f32", 64, 64), (16, 64, "bf16", 128, 128),
                                            (1, 64, "bf16", 192, 128)])
def test_decode_blocks_up_to_the_longest(K, G, T, q_dt, Dk, Dv):
    """Blocks of 17 to 64 tokens: of sequences longer and shorter than the block, empty and exactly as long."""
    torch = _torch()
    rng = seeded("blocks", G, T, q_dt, Dk)
    Hkv, W = 2, 804
    lengths = np.array([801, 5, 0, T, T + 1, 97], np.int32)
    B, Hq = len(lengths), Hkv * G
    pk, pv = random_q4(rng, B, Hkv, W, Dk), random_q4(rng, B, Hkv, W, Dv)
    q = dev(rng.standard_normal((B, T, Hq, Dk)).astype(np.float32), dt(q_dt))
    out = torch.full((B, T, Hq, Dv), float("nan"), device="cuda")
    ws = torch.zeros(K.decode_q4_workspace_bytes(B, Hkv, Hq, T, W, Dv), dtype=torch.uint8, device="cuda")
    K.kv_attn_decode_q4(q, filled(K, *pk, *pv), dev(lengths), lengths, out, ws)
    torch.cuda.synchronize()
    vk, vv = dev(Q.q4_values(*pk)), dev(Q.q4_values(*pv))
    for b, L in enumerate(lengths):
        empty = max(0, T - int(L))
        got = host(out[b])
        assert np.all(got[:empty] == 0), f"L={L}: rows that see nothing"
        if empty < T:
            ref = host(attend(q[b].double(), vk[b], vv[b], int(L)))
            assert row_rel_err(got[empty:], ref[empty:]) <= ROW_REL, f"L={L}"


@pytest.mark.parametrize("G,T", [(2, 1), (8, 2)])
def test_decode_one_unit_of_very_many_parts(K, G, T):
    """600001 slots of one KV head: more parts than the last CTA joins in one pass (256)."""
    rng = seeded("parts", G, T)
    L, W, D = 600001, 600004, 64
    k, v = rng.standard_normal((1, 1, W, D)), rng.standard_normal((1, 1, W, D))
    torch = _torch()
    pk, pv = Q.q4_quantise(k), Q.q4_quantise(v)
    lengths = np.array([L], np.int32)
    q = dev(rng.standard_normal((1, T, G, D)).astype(np.float32), torch.bfloat16)
    out = torch.full((1, T, G, D), float("nan"), device="cuda")
    ws = torch.zeros(K.decode_q4_workspace_bytes(1, 1, G, T, L, D), dtype=torch.uint8, device="cuda")
    K.kv_attn_decode_q4(q, filled(K, *pk, *pv), dev(lengths), lengths, out, ws)
    torch.cuda.synchronize()
    ref = attend(q[0].double(), dev(Q.q4_values(*pk)[0]), dev(Q.q4_values(*pv)[0]), L)
    assert row_rel_err(host(out[0]), host(ref)) <= ROW_REL


# ---------------------------------------------------------------------------------------------
# long appends and far positions
# ---------------------------------------------------------------------------------------------
def append_and_check(K, rng, N, T, Hkv, G, Dk, Dv, in_dt, q_dt, rope, pos, norm, after, with_q):
    """kv_cache_append_q4 of random rows against the float64 transform and quantiser's bounds.  bf16 has 8
    significant bits: a rounding is off by at most 2^-8 of the value (half its eps of 2^-7)."""
    torch = _torch()
    W, first = (T + 5 + 3) // 4 * 4, 2
    Hq = Hkv * G
    q, k, v = (O.store(rng.standard_normal(s), in_dt) for s in ((N, T, Hq, Dk), (N, T, Hkv, Dk), (N, T, Hkv, Dv)))
    qw, kw = ((1 + 0.2 * rng.standard_normal((N, Dk))).astype(np.float32) for _ in range(2))
    slot = np.arange(first, first + T, dtype=np.int32)
    cache = K.KVCacheQ4.zeros(N, Hkv, W, Dk, Dv)
    for t in (cache.k, cache.v):
        t.fill_(0xA5)
    q_out = torch.full((N, T, Hq, Dk), float("nan"), dtype=dt(q_dt), device="cuda") if with_q else None
    f = lambda x: dev(x.astype(np.float32), dt(in_dt))   # noqa: E731
    K.kv_cache_append_q4(f(q) if with_q else None, f(k), f(v), dev(pos) if pos is not None else None, dev(slot), slot, cache,
                         q_out, K.Rope(**rope), q_norm_w=dev(qw) if norm else None, k_norm_w=dev(kw) if norm else None,
                         norm_after_rope=after, norm_inst_stride=Dk if norm else 0)
    torch.cuda.synchronize()
    kinds = dict(rope)
    if "rot_dim" not in kinds:
        kinds["rot_dim"] = None
    r = O.Rope(**kinds)
    uk, sk, mk = Q.q4_unpack(cache.k.cpu().numpy()), host(cache.k_scale)[..., 0], host(cache.k_scale)[..., 1]
    uv, sv, mv = Q.q4_unpack(cache.v.cpu().numpy()), host(cache.v_scale)[..., 0], host(cache.v_scale)[..., 1]
    rest = np.ones(W, bool)
    rest[slot] = False
    assert bool((cache.k[:, :, rest] == 0xA5).all()) and bool((cache.v[:, :, rest] == 0xA5).all())
    for n in range(N):
        p = pos[n] if pos is not None else None
        if with_q:
            want = O.qk_transform(q[n], p, qw[n] if norm else None, 1e-6, r, after)
            off = np.abs(host(q_out[n]) - want)
            assert np.all(off <= np.abs(want) * (2.0 ** -8 if q_dt == "bf16" else 0) + 4e-6 * np.abs(want).max(-1, keepdims=True))
        for x, u, scale, mid, exact in ((O.qk_transform(k[n], p, kw[n] if norm else None, 1e-6, r, after), uk[n], sk[n], mk[n], False),
                                        (v[n], uv[n], sv[n], mv[n], True)):
            x = x.transpose(1, 0, 2)                           # [Hkv, T, D]
            u, scale, mid = u[:, slot], scale[:, slot], mid[:, slot]
            g = x.reshape(*x.shape[:-1], -1, 64)
            # float32 steps before the quantiser (4e-6, as in the transforms' test); none for V
            slack = (0.0 if exact else 4e-6) * np.abs(x).max(-1)[..., None] + 2.0 ** -22 * np.abs(mid)
            off = np.abs(Q.q4_values(u, scale, mid).reshape(g.shape) - g)
            assert np.all(off <= (scale / 2 + np.abs(mid) * 2.0 ** -8 + slack)[..., None])
            spread = g.max(-1) - g.min(-1)
            assert np.all(15 * scale <= (spread + 2 * slack) * (1 + 2.0 ** -7)) and np.all(15 * scale >= spread - 2 * slack)


@pytest.mark.parametrize("N,T,Hkv,G,Dk,Dv,in_dt,q_dt,rope,axes,norm,after,with_q", [
    (28, 181, 2, 2, 128, 128, "bf16", "bf16", dict(kind="1d", base=1e6), 1, True, False, True),
    (1, 4999, 1, 3, 64, 64, "f32", "f32", dict(kind="1d", base=1e4, rot_offset=5, rot_dim=22), 1, True, False, True),
    (2, 2501, 3, 1, 192, 128, "f32", "bf16", dict(kind="interleaved", base=1e6, rot_offset=128, rot_dim=64), 1, False, False, False),
    (7, 701, 2, 2, 256, 64, "bf16", "f32", dict(kind="2d", base=1e4), 2, True, True, True),
    (1, 4867, 4, 1, 128, 192, "f32", "f32", dict(kind="sections", base=1.11588e7, sections=(16, 16, 16, 16)), 4, True, True, False),
    (3, 1627, 5, 1, 64, 256, "bf16", "bf16", dict(kind="none"), 0, True, False, True),
])
def test_long_appends(K, N, T, Hkv, G, Dk, Dv, in_dt, q_dt, rope, axes, norm, after, with_q):
    """Enough tokens that a warp takes one each and a CTA eight; the last CTA of an instance is partly filled."""
    assert N * T >= 4864 and T % 8 != 0
    rng = seeded("long append", N, T, Dk, Dv)
    pos = rng.integers(-2000, 130000, (N, T, axes)).astype(np.int32) if axes else None
    append_and_check(K, rng, N, T, Hkv, G, Dk, Dv, in_dt, q_dt, rope, pos, norm, after, with_q)


@pytest.mark.parametrize("rope,axes,Dk", [(dict(kind="1d", base=1e6), 1, 128), (dict(kind="interleaved", base=1e4), 1, 64),
                                          (dict(kind="sections", base=1.11588e7, sections=(16, 16, 16, 16)), 4, 128),
                                          (dict(kind="2d", base=1e4), 2, 64)])
def test_far_and_negative_positions(K, rope, axes, Dk):
    """Positions on both sides of +-2^20, where the angle passes from pairs of floats to float64, up to the ends of
    32 bits.  There float64 rounds an angle near 2^31 by up to 1.2e-7, in the definition as in the kernel."""
    rng = seeded("far positions", rope["kind"])
    at = np.array([0, -1, 1, (1 << 20) - 1, 1 << 20, (1 << 20) + 1, -(1 << 20) + 1, -(1 << 20), -(1 << 20) - 1, 12345678, -98765432,
                   (1 << 31) - 1, -(1 << 31), 999999999], np.int64)
    T = len(at)
    pos = np.stack([np.roll(at, a) for a in range(axes)], -1)[None].astype(np.int32)
    append_and_check(K, rng, 1, T, 2, 2, Dk, 64, "f32", "f32", rope, pos, False, False, True)
