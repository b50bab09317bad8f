"""GPU parity of the 4-bit cache (kv_cache_append_q4, kv_cache_expand_q4, kv_attn_decode_q4) against
the float64 definitions in oracle/q4_oracle.py.

Tolerances.  Codes and scales of inputs whose quotients are exact are equal bit for bit.  Transformed
inputs (norm, rotation) carry a float32 error of at most 4e-6 of the row's largest value, so a value
read back is off by that plus scale / 2 plus half a bf16 step of mid (2^-9 |mid|).  Attention: the
bounds allow for weights of 17 significant bits or more (two bf16 halves; the kernel's float16 halves hold
22), i.e. a weight is off by at most 2^-18 of itself, and for a float32 q likewise (bf16 q is exact),
which moves a score s by up to 2^-18 sum |q k| and its weight by as much, relatively.  With |sum| terms of the inputs below
(sum |q k| scale <= 12) a row is off by at most (2^-18 + 2 * 12 * 2^-18) < 1e-4 of sum p |v| when every
rounding conspires; independent roundings leave the root of that, below 2e-5 of the row's norm,
which is the bound used; float32 sums add less than 1e-6 to it.
"""
import ctypes as C
import zlib

import numpy as np
import pytest

import oracle as O
from helpers import dev, host, row_rel_err
from oracle import q4_oracle as Q

pytestmark = pytest.mark.gpu

ROW_REL = 2e-5


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


def dt(name):
    torch = _torch()
    return torch.float32 if name == "f32" else torch.bfloat16


def filled(K, u_k, s_k, m_k, u_v, s_v, m_v):
    """KVCacheQ4 of codes [N,H,W,G,64] and their scale/mid."""
    torch = _torch()
    pair = lambda s, m: dev(np.stack([s, m], -1).astype(np.float32)).to(torch.bfloat16)  # noqa: E731
    return K.KVCacheQ4(dev(Q.q4_pack(u_k)), dev(Q.q4_pack(u_v)), pair(s_k, m_k), pair(s_v, m_v))


def random_q4(rng, N, H, W, D, offset=0.0, width=1.0):
    return Q.q4_quantise(rng.standard_normal((N, H, W, D)) * width + offset)


def parts(codes, pairs):
    """(u, scale, mid) of cache tensors on the device."""
    p = host(pairs)
    return Q.q4_unpack(codes.cpu().numpy()), p[..., 0], p[..., 1]


# ---------------------------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("Dk,Dv,Hkv,G,N,T", [(64, 64, 1, 1, 1, 1), (128, 128, 8, 2, 3, 5), (192, 128, 3, 1, 2, 4),
                                             (256, 256, 2, 4, 1, 3), (64, 256, 2, 3, 2, 7), (256, 64, 1, 1, 1, 2),
                                             (128, 128, 1, 40, 2, 9)])
@pytest.mark.parametrize("in_dt", ["bf16", "f32"])
def test_append_exact_inputs_bit_for_bit(K, Dk, Dv, Hkv, G, N, T, in_dt):
    torch = _torch()
    rng = seeded("exact", Dk, Dv, Hkv, G, N, T)
    Hq, W = Hkv * G, T + 5 + (-(T + 5)) % 4
    grid = lambda *s: rng.integers(-96, 97, s) / 32.0    # noqa: E731  (bf16 values; every quotient's operands exact)
    q, k, v = grid(N, T, Hq, Dk), grid(N, T, Hkv, Dk), grid(N, T, Hkv, Dv)
    slot = np.stack([rng.permutation(W)[:T] for _ in range(N)]).astype(np.int32)
    cache = K.KVCacheQ4.zeros(N, Hkv, W, Dk, Dv)
    for t in (cache.k, cache.v):
        t.fill_(0xA5)
    for t in (cache.k_scale, cache.v_scale):
        t.fill_(77.0)
    q_out = torch.full((N, T, Hq, Dk), float("nan"), device="cuda")
    K.kv_cache_append_q4(dev(q.astype(np.float32), dt(in_dt)), dev(k.astype(np.float32), dt(in_dt)),
                         dev(v.astype(np.float32), dt(in_dt)), None, dev(slot), slot, cache, q_out, K.Rope("none"))
    torch.cuda.synchronize()
    assert np.array_equal(host(q_out), q)
    for x, codes, pairs in ((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale)):
        u, scale, mid = parts(codes, pairs)
        want_u, want_s, want_m = Q.q4_quantise(x.transpose(0, 2, 1, 3))
        untouched = np.ones((N, Hkv, W), bool)
        for n in range(N):
            untouched[n][:, slot[n]] = False
            assert np.array_equal(u[n][:, slot[n]], want_u[n])
            assert np.array_equal(scale[n][:, slot[n]], want_s[n]) and np.array_equal(mid[n][:, slot[n]], want_m[n])
        assert np.all(codes.cpu().numpy()[untouched] == 0xA5) and np.all(host(pairs)[untouched] == 77.0)


ROPES = {
    "1d": (dict(kind="1d", base=1e6), 1), "sections": (dict(kind="sections", base=1.11588e7, sections=(16, 16, 16, 16)), 4),
    "2d": (dict(kind="2d", base=1e4), 2), "interleaved": (dict(kind="interleaved", base=1e6), 1),
    "tail64": (dict(kind="interleaved", base=1e6, rot_offset=128, rot_dim=64), 1),
    "odd_range": (dict(kind="1d", base=1e4, rot_offset=5, rot_dim=22), 1), "none": (dict(kind="none"), 0),
}


@pytest.mark.parametrize("rope,Dk,Dv", [("1d", 128, 128), ("sections", 128, 128), ("2d", 64, 64), ("interleaved", 256, 128),
                                        ("tail64", 192, 128), ("odd_range", 64, 128), ("none", 192, 64)])
@pytest.mark.parametrize("in_dt,q_dt,norm,after", [("f32", "f32", True, False), ("bf16", "bf16", True, True),
                                                   ("f32", "bf16", False, False)])
def test_append_transforms(K, rope, Dk, Dv, in_dt, q_dt, norm, after):
    torch = _torch()
    rng = seeded("transform", rope, in_dt, norm, after)
    N, T, Hkv, Hq, W = 2, 6, 2, 6, 12
    kw, axes = ROPES[rope]
    q, k, v = (O.store(rng.standard_normal(s), in_dt) for s in ((N, T, Hq, Dk), (N, T, Hkv, Dk), (N, T, Hkv, Dv)))
    pos = rng.integers(0, 130000, (N, T, max(axes, 1))).astype(np.int32)
    qw, kwt = ((1 + 0.2 * rng.standard_normal((N, Dk))).astype(np.float32) for _ in range(2))
    slot = np.arange(2, 2 + T, dtype=np.int32)
    cache = K.KVCacheQ4.zeros(N, Hkv, W, Dk, Dv)
    q_out = torch.empty((N, T, Hq, Dk), dtype=dt(q_dt), device="cuda")
    f = lambda x: dev(x.astype(np.float32), dt(in_dt))   # noqa: E731
    K.kv_cache_append_q4(f(q), f(k), f(v), dev(pos) if axes else None, dev(slot), slot, cache, q_out, K.Rope(**kw),
                         q_norm_w=dev(qw) if norm else None, k_norm_w=dev(kwt) if norm else None,
                         norm_after_rope=after, norm_inst_stride=Dk if norm else 0)
    kc = torch.zeros((N, Hkv, W, Dk), device="cuda")
    vc = torch.zeros((N, Hkv, W, Dv), device="cuda")
    # the unquantised append of the same rows is the transformed value (checked on its own elsewhere)
    q_ref = torch.empty((N, T, Hq, Dk), device="cuda")
    K.kv_cache_append_rope_qknorm(f(q), f(k), f(v), dev(pos) if axes else None, dev(slot), slot, K.KVCache(kc, vc), q_ref,
                                  K.Rope(**kw), q_norm_w=dev(qw) if norm else None, k_norm_w=dev(kwt) if norm else None,
                                  norm_after_rope=after, norm_inst_stride=Dk if norm else 0)
    torch.cuda.synchronize()
    got_q, want_q = host(q_out), host(q_ref)
    assert np.all(np.abs(got_q - want_q) <= np.abs(want_q) * (2.0 ** -8 if q_dt == "bf16" else 0) + 4e-6 * np.abs(want_q).max())
    for want, codes, pairs in ((host(kc), cache.k, cache.k_scale), (host(vc), cache.v, cache.v_scale)):
        u, scale, mid = parts(codes, pairs)
        x = want[:, :, 2:2 + T]
        u, scale, mid = u[:, :, 2:2 + T], scale[:, :, 2:2 + T], mid[:, :, 2:2 + T]
        g = x.reshape(*x.shape[:-1], -1, 64)
        slack = 4e-6 * np.abs(x).max(-1)[..., None]
        off = np.abs(Q.q4_values(u, scale, mid).reshape(g.shape) - g)
        assert np.all(off <= (scale / 2 + np.abs(mid) * 2.0 ** -9 + slack)[..., None])
        spread = g.max(-1) - g.min(-1)
        assert np.all(15 * scale <= (spread + 2 * slack) * (1 + 2.0 ** -7)) and np.all(15 * scale >= spread - 2 * slack)


def test_append_special_groups(K):
    """NaN, infinities, a spread beyond float32, equal values, a spread below bf16's normal range."""
    torch = _torch()
    x = np.zeros((1, 8, 1, 128), np.float32)
    x[0, 0, 0, 5] = np.nan
    x[0, 1, 0, 70] = np.inf
    x[0, 2, 0, 0], x[0, 2, 0, 1] = 3e38, -3e38
    x[0, 3, 0, :64] = 0.1
    x[0, 4, 0, 3] = 1e-41
    x[0, 5, 0, :] = -np.arange(128) / 4
    x[0, 6, 0, 64:] = 3.4e38                       # beyond bf16's largest value
    x[0, 7, 0, 1] = 1e30
    slot = np.arange(8, dtype=np.int32)
    cache = K.KVCacheQ4.zeros(1, 1, 8, 128)
    K.kv_cache_append_q4(None, dev(x), dev(x), None, dev(slot), slot, cache, None, K.Rope("none"))
    out = K.KVCache(torch.zeros((1, 1, 8, 128), device="cuda"), torch.zeros((1, 1, 8, 128), device="cuda"))
    K.kv_cache_expand_q4(cache, dev(slot), slot, out)
    torch.cuda.synchronize()
    for t in (out.k, out.v):
        r = host(t)[0, 0]
        assert np.all(np.isnan(r[0, :64])) and np.all(r[0, 64:] == 0)
        assert np.all(np.isnan(r[1, 64:])) and np.all(r[1, :64] == 0)
        assert np.all(np.isnan(r[2, :64]))
        assert np.all(r[3, :64] == O.bf16_round(np.float64(np.float32(0.1))))
        assert np.all(np.abs(r[4]) <= 1e-41)
        assert np.array_equal(r[5], Q.q4_values(*Q.q4_quantise(x[0, 5, 0])))
        assert np.all(np.isnan(r[6, 64:])) and np.all(r[6, :64] == 0)
        assert np.array_equal(r[7], Q.q4_values(*Q.q4_quantise(x[0, 7, 0].astype(np.float64))))


@pytest.mark.parametrize("dst", ["f32", "bf16"])
@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128), (192, 128), (256, 64)])
def test_expand(K, Dk, Dv, dst):
    torch = _torch()
    rng = seeded("expand", Dk, Dv)
    N, H, W, T, first = 2, 3, 20, 9, 4
    pk, pv = random_q4(rng, N, H, W, Dk), random_q4(rng, N, H, W, Dv, offset=2.0)
    cache = filled(K, *pk, *pv)
    slot = rng.integers(0, W, (N, T)).astype(np.int32)         # repeats allowed
    out = K.KVCache(torch.full((N, H, 16, Dk), 7.0, dtype=dt(dst), device="cuda"),
                    torch.full((N, H, 16, Dv), 7.0, dtype=dt(dst), device="cuda"))
    K.kv_cache_expand_q4(cache, dev(slot), slot, out, dst_first=first)
    torch.cuda.synchronize()
    for p, t in ((pk, out.k), (pv, out.v)):
        want = O.store(Q.q4_values(*p).astype(np.float32), dst)
        got = host(t)
        for n in range(N):
            assert np.array_equal(got[n][:, first:first + T], want[n][:, slot[n]])
        assert np.all(got[:, :, :first] == 7.0) and np.all(got[:, :, first + T:] == 7.0)


# ---------------------------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------------------------
def check_decode(K, rng, B, T, Hkv, G, Dk, Dv, lengths, W, q_dt, q_width=1.0, offset=0.0, width=1.0, scale=0.0, tol=ROW_REL,
                 bound=None):
    torch = _torch()
    Hq = Hkv * G
    lengths = np.asarray(lengths, np.int32)
    pk, pv = random_q4(rng, B, Hkv, W, Dk), random_q4(rng, B, Hkv, W, Dv, offset, width)
    q = O.store(q_width * rng.standard_normal((B, T, Hq, Dk)), q_dt)
    cache = filled(K, *pk, *pv)
    for b, L in enumerate(lengths):                            # canaries past the valid slots
        cache.k_scale[b, :, L:] = float("nan")
        cache.v_scale[b, :, L:] = float("inf")
        cache.k[b, :, L:] = 0xFF
    ws = torch.zeros(K.decode_q4_workspace_bytes(B, Hkv, Hq, T, max(1, int(lengths.max())), Dv), dtype=torch.uint8,
                     device="cuda")
    outs = []
    for _ in range(2):                                         # the second call reuses the workspace
        out = torch.full((B, T, Hq, Dv), float("nan"), device="cuda")
        K.kv_attn_decode_q4(dev(q.astype(np.float32), dt(q_dt)), cache, dev(lengths), lengths, out, ws, scale=scale)
        torch.cuda.synchronize()
        outs.append(host(out))
        zero = K.lib().kva_decode_q4_workspace_zero_bytes(B, Hkv, Hq, T)
        assert int(ws[:zero].sum()) == 0
    assert np.array_equal(outs[0], outs[1])
    got, vk, vv = outs[0], Q.q4_values(*pk), Q.q4_values(*pv)
    for b, L in enumerate(lengths):
        ref = Q.attend_block(q[b], vk[b], vv[b], int(L), scale if scale > 0 else None)
        empty = max(0, T - int(L))
        assert np.all(got[b, :empty] == 0), f"b={b} L={L}: rows that see nothing"
        if empty < T:
            if bound is not None:
                assert np.max(np.abs(got[b, empty:] - ref[empty:])) <= bound, f"b={b} L={L}"
            else:
                assert row_rel_err(got[b, empty:], ref[empty:]) <= tol, f"b={b} L={L}"


EDGES = [0, 1, 2, 3, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 200]


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("G,T,q_dt", [(1, 1, "bf16"), (2, 1, "f32"), (3, 1, "bf16"), (4, 1, "f32"), (5, 1, "f32"),
                                      (8, 1, "bf16"), (9, 1, "f32"), (2, 2, "bf16"), (2, 5, "f32"), (1, 16, "bf16"),
                                      (4, 5, "f32"), (16, 1, "bf16"), (3, 11, "bf16")])
def test_decode_parity(K, Dk, Dv, G, T, q_dt):
    check_decode(K, seeded("decode", Dk, Dv, G, T, q_dt), len(EDGES), T, 2, G, Dk, Dv, EDGES, 204, q_dt)


@pytest.mark.parametrize("G,T,q_dt,Dk,Dv", [(2, 1, "bf16", 128, 128), (4, 1, "f32", 128, 128), (8, 1, "bf16", 64, 64),
                                            (1, 1, "f32", 192, 128), (2, 16, "bf16", 128, 128), (1, 3, "f32", 192, 128)])
def test_decode_long_and_ragged(K, G, T, q_dt, Dk, Dv):
    """Chunks of several lengths, joined over CTAs."""
    check_decode(K, seeded("long", G, T, q_dt), 5, T, 1, G, Dk, Dv, [1, 4097, 9001, 0, 3333], 9004, q_dt)


def test_decode_extreme_scores_and_values(K):
    # scores up to a few hundred: one key takes the row, the weights of the rest underflow
    check_decode(K, seeded("peaked"), 3, 1, 2, 2, 128, 128, [77, 900, 5], 900, "bf16", q_width=60.0, tol=1e-4)
    # large and tiny values
    check_decode(K, seeded("wide"), 2, 1, 1, 2, 128, 128, [300, 64], 300, "bf16", width=1e5)
    check_decode(K, seeded("tiny"), 2, 1, 1, 2, 128, 128, [300, 64], 300, "bf16", width=1e-6)
    # a common offset: the row's norm is the offset's
    check_decode(K, seeded("offset"), 2, 1, 1, 4, 64, 64, [300, 63], 300, "f32", offset=50.0)
    # a scale given by the caller; scale 1e-3 makes the weights flat
    check_decode(K, seeded("flat"), 2, 1, 1, 4, 128, 128, [500, 63], 500, "f32", scale=1e-3)


def test_decode_flat_long_context_keeps_its_precision(K):
    """Flat weights over a long context: the output is the small mean of 30000 values, far below one
    value's size.  The weights' rounding (2^-18 each, independent) and the float32 sums leave an
    error below 2e-5 of the row's norm."""
    check_decode(K, seeded("flat-long"), 1, 1, 1, 2, 128, 128, [30001], 30004, "bf16", q_width=0.1)


@pytest.mark.parametrize("G,D,L", [(8, 128, 100001), (2, 128, 100001), (16, 64, 50003)])
def test_decode_long_sums_are_not_cut_off(K, G, D, L):
    """Thousands of values a sum.  A score of at most 8 (base 2) takes up to 6 roundings of 2^-24, 2.9e-6 of
    its weight, exp and the weight's halves 2^-22 + 2^-23: 3.3e-6 when all conspire.  Values of either
    sign: errors and output are both root sums of p^2 v^2, so the row is off by less than that."""
    check_decode(K, seeded("sums", G, D), 1, 1, 1, G, D, D, [L], (L + 3) // 4 * 4, "bf16", tol=3.3e-6)


@pytest.mark.parametrize("G,T,D,Hkv,q_dt", [(2, 1, 64, 4, "bf16"), (3, 2, 64, 4, "f32"), (2, 8, 128, 4, "bf16")])
def test_decode_many_short_instances(K, G, T, D, Hkv, q_dt):
    """More units than the GPU holds at once, each of one or two stages, empty ones among them."""
    lengths = [(0, 1, 31, 64, 33, 63, 2, 32, 64, 50)[b % 10] for b in range(800)]
    check_decode(K, seeded("many", G, T, D), len(lengths), T, Hkv, G, D, D, lengths, 64, q_dt)


@pytest.mark.parametrize("G,T", [(2, 1), (2, 4)])
def test_decode_many_instances_and_a_long_one(K, G, T):
    """More instances than a CTA has threads, a long one among short and empty ones."""
    lengths = [(0, 1, 31, 64, 33)[b % 5] for b in range(300)]
    lengths[137] = 1001
    check_decode(K, seeded("mixed", G, T), len(lengths), T, 1, G, 64, 64, lengths, 1004, "bf16")


def test_decode_lengths_on_the_device_rule(K):
    """The host lengths are an upper bound: the device's decide, also when a captured call is replayed."""
    torch = _torch()
    rng = seeded("graph")
    B, Hkv, G, D, W = 3, 2, 2, 128, 1000
    pk, pv = random_q4(rng, B, Hkv, W, D), random_q4(rng, B, Hkv, W, D)
    cache = filled(K, *pk, *pv)
    q = O.store(rng.standard_normal((B, 1, Hkv * G, D)), "bf16")
    qd = dev(q.astype(np.float32), torch.bfloat16)
    upper = np.full(B, W, np.int32)
    lengths = dev(np.array([1000, 3, 0], np.int32))
    ws = torch.zeros(K.decode_q4_workspace_bytes(B, Hkv, Hkv * G, 1, W, D), dtype=torch.uint8, device="cuda")
    out = torch.empty((B, 1, Hkv * G, D), device="cuda")
    call = lambda: K.kv_attn_decode_q4(qd, cache, lengths, upper, out, ws)   # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    vk, vv = Q.q4_values(*pk), Q.q4_values(*pv)
    for now in ([1000, 3, 0], [17, 999, 64], [0, 0, 1]):
        lengths.copy_(torch.tensor(now, dtype=torch.int32))
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        for b, L in enumerate(now):
            ref = Q.attend_block(q[b], vk[b], vv[b], L)
            got = host(out[b])
            assert np.all(got == 0) if L == 0 else row_rel_err(got, ref) <= ROW_REL
    # a device length beyond the cache is cut to it
    lengths.fill_(1 << 30)
    call()
    torch.cuda.synchronize()
    assert row_rel_err(host(out[1]), Q.attend_block(q[1], vk[1], vv[1], W)) <= ROW_REL


def test_decode_instances_apart_in_memory(K):
    """inst_rows larger than an instance's rows, on a stream of its own."""
    torch = _torch()
    rng = seeded("strided")
    B, Hkv, G, D, W = 2, 2, 2, 128, 40
    pk, pv = random_q4(rng, 2 * B, Hkv, W, D), random_q4(rng, 2 * B, Hkv, W, D)
    c = filled(K, *pk, *pv)                                    # every second instance belongs to the call
    st = c.struct
    st = type(st)(st.k, st.v, st.k_scale, st.v_scale, Hkv, D, W, 0, 2 * Hkv * W)
    q = O.store(rng.standard_normal((B, 1, Hkv * G, D)), "f32")
    lengths = np.array([40, 23], np.int32)
    side = torch.cuda.Stream()
    qd, ld = dev(q.astype(np.float32)), dev(lengths)
    ws = torch.zeros(K.decode_q4_workspace_bytes(B, Hkv, Hkv * G, 1, W, D), dtype=torch.uint8, device="cuda")
    out = torch.empty((B, 1, Hkv * G, D), device="cuda")
    torch.cuda.synchronize()
    status = K.lib().kv_attn_decode_q4(qd.data_ptr(), 0, st, ld.data_ptr(), lengths.ctypes.data, B, 1, Hkv * G,
                                       C.c_float(0.0), out.data_ptr(), ws.data_ptr(), ws.numel(), side.cuda_stream)
    assert status == 0, K.lib().kva_last_error()
    side.synchronize()
    for b, L in enumerate(lengths):
        ref = Q.attend_block(q[b], Q.q4_values(*pk)[2 * b], Q.q4_values(*pv)[2 * b], int(L))
        assert row_rel_err(host(out[b]), ref) <= ROW_REL


def test_two_calls_at_once_on_two_streams(K):
    """Two decodes over one cache at once, each with its own workspace, give what one alone gives."""
    torch = _torch()
    rng = seeded("streams")
    B, Hkv, G, D, W = 4, 2, 2, 128, 3000
    cache = filled(K, *random_q4(rng, B, Hkv, W, D), *random_q4(rng, B, Hkv, W, D))
    lengths = np.array([3000, 1, 0, 1777], np.int32)
    ld = dev(lengths)
    qs = [torch.randn((B, Hkv * G, D), device="cuda") for _ in range(2)]
    n = K.decode_q4_workspace_bytes(B, Hkv, Hkv * G, 1, W, D)
    wss = [torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    alone = []
    for q in qs:
        o = torch.empty((B, Hkv * G, D), device="cuda")
        K.kv_attn_decode_q4(q, cache, ld, lengths, o, wss[0])
        torch.cuda.synchronize()
        alone.append(o)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(alone[0]) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for q, ws, s, o in zip(qs, wss, streams, outs):
            K.kv_attn_decode_q4(q, cache, ld, lengths, o, ws, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], alone[0]) and torch.equal(outs[1], alone[1])


def test_offsets_past_32_bits(K):
    """A cache whose last instance lies beyond 2^32 bytes of codes: append, read back, attend."""
    torch = _torch()
    N, Hkv, D, W = 17, 8, 128, 1 << 19                        # 17 x 8 x 524288 rows of 64 bytes: 4.6 GB of K codes
    cache = K.KVCacheQ4.zeros(N, Hkv, W, D)
    rng = seeded("far")
    T = 3
    x = rng.integers(-96, 97, (N, T, Hkv, D)) / 32.0
    slot = np.array([W - 1, 0, W // 2], np.int32)
    xd = dev(x.astype(np.float32))
    K.kv_cache_append_q4(None, xd, xd, None, dev(slot), slot, cache, None, K.Rope("none"))
    out = K.KVCache(*(torch.zeros((N, Hkv, T, D), device="cuda") for _ in range(2)))
    K.kv_cache_expand_q4(cache, dev(slot), slot, out)
    torch.cuda.synchronize()
    want = Q.q4_values(*Q.q4_quantise(x.transpose(0, 2, 1, 3)))
    assert np.array_equal(host(out.k), want) and np.array_equal(host(out.v), want)
    # the last instance's context: zeros but for the two slots, so the weights follow by hand
    lengths = np.zeros(N, np.int32)
    lengths[-1] = W
    q = np.zeros((N, 8, D), np.float32)
    q[-1] = 20.0 * x[-1, 0] / np.sqrt(D)
    ws = torch.zeros(K.decode_q4_workspace_bytes(N, Hkv, 8, 1, W, D), dtype=torch.uint8, device="cuda")
    o = torch.empty((N, 8, D), device="cuda")
    K.kv_attn_decode_q4(dev(q), cache, dev(lengths), lengths, o, ws)
    torch.cuda.synchronize()
    got = host(o)
    assert np.all(got[:-1] == 0)
    for h in range(Hkv):
        s = want[-1, h] @ q[-1, h].astype(np.float64) / np.sqrt(D)
        m = max(s.max(), 0.0)
        p = np.exp(s - m)
        ref = p @ want[-1, h] / (p.sum() + (W - T) * np.exp(-m))
        assert row_rel_err(got[-1, h][None], ref[None]) <= ROW_REL


# ---------------------------------------------------------------------------------------------
# the operators together, as a server uses them
# ---------------------------------------------------------------------------------------------
def test_prompt_then_tokens_then_scores(K):
    """A prompt is appended in 4 bits, read back into a bf16 cache and prefilled there; then draft blocks
    and tokens are appended and attended in 4 bits, and the outputs score tokens over a vocabulary."""
    torch = _torch()
    rng = seeded("together")
    Hkv, G, D, P, W, V = 2, 2, 128, 37, 64, 1003
    Hq = Hkv * G
    rope = K.Rope("1d", 1e6)
    total = P + 4 + 3
    q, k, v = (rng.standard_normal((1, total, h, D)).astype(np.float32) for h in (Hq, Hkv, Hkv))
    pos = np.arange(total, dtype=np.int32)[None, :, None]
    qw, kw = ((1 + 0.1 * rng.standard_normal(D)).astype(np.float32) for _ in range(2))
    cache = K.KVCacheQ4.zeros(1, Hkv, W, D)
    kwargs = dict(q_norm_w=dev(qw), k_norm_w=dev(kw))

    def append(t0, t1):
        slot = np.arange(t0, t1, dtype=np.int32)[None]
        q_out = torch.empty((1, t1 - t0, Hq, D), dtype=torch.bfloat16, device="cuda")
        K.kv_cache_append_q4(dev(q[:, t0:t1]), dev(k[:, t0:t1]), dev(v[:, t0:t1]), dev(pos[:, t0:t1]), dev(slot), slot, cache,
                             q_out, rope, **kwargs)
        return q_out

    q_pre = append(0, P)
    prefix = np.arange(P, dtype=np.int32)
    wide = K.KVCache(*(torch.zeros((1, Hkv, W, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    K.kv_cache_expand_q4(cache, dev(prefix), prefix, wide)
    out_pre = torch.empty((1, P, Hq, D), device="cuda")
    K.kv_attn_prefill(q_pre, wide, out_pre, mask="causal")
    torch.cuda.synchronize()
    vals = lambda: (Q.q4_values(*parts(cache.k, cache.k_scale))[0], Q.q4_values(*parts(cache.v, cache.v_scale))[0])  # noqa: E731
    vk, vv = vals()
    ref = Q.attend_block(host(q_pre)[0], vk, vv, P)
    # the prefill kernel's own tolerance (bf16 probabilities, values rounded to bf16 on the way)
    assert np.max(np.abs(host(out_pre)[0] - ref)) <= 2e-2
    table = (0.05 * rng.standard_normal((V, Hq * D))).astype(np.float32)
    td = dev(table, torch.bfloat16)
    t0 = P
    for T in (4, 1, 1, 1):
        q_new = append(t0, t0 + T)
        t0 += T
        L = np.array([t0], np.int32)
        ws = torch.zeros(K.decode_q4_workspace_bytes(1, Hkv, Hq, T, W, D), dtype=torch.uint8, device="cuda")
        out = torch.empty((1, T, Hq, D), device="cuda")
        K.kv_attn_decode_q4(q_new, cache, dev(L), L, out, ws)
        h = out.view(T, Hq * D)
        targets = rng.integers(0, V, T).astype(np.int32)
        lp, ent = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        ids, top = torch.empty((T, 3), dtype=torch.int32, device="cuda"), torch.empty((T, 3), device="cuda")
        ws2 = torch.empty(K.lmhead_logprobs_workspace_bytes(T, Hq * D, V, 3), dtype=torch.uint8, device="cuda")
        K.lmhead_logprobs(h, td, ws2, targets=dev(targets), out_logprob=lp, out_entropy=ent, top_ids=ids, top_logprobs=top)
        torch.cuda.synchronize()
        vk, vv = vals()
        ref = Q.attend_block(host(q_new)[0], vk, vv, t0)
        assert row_rel_err(host(out)[0], ref) <= ROW_REL
        want = Q.logprobs(ref.reshape(T, -1), host(td), V, targets=targets, top_k=3)
        assert np.allclose(host(lp), want[0], atol=1e-4) and np.allclose(host(ent), want[1], atol=1e-4)
        assert np.allclose(host(top), want[4], atol=1e-4)
