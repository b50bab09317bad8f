"""How many bits the paged attention's weights keep.

Every query row is a unit vector, one key of its sequence scores 0 and one scores -a (exactly: one product each), all others
so little that their weight is 0.  With p = exp(-a) and weights (1, p) a row is (v0 + p v1) / (1 + p), and a value v1 = 1 beside v0 = 0
or v0 = -bf16(p) shows what became of p.

Relative errors of p before it meets V: 2^-22 from the exponential, ln 2 |a log2 e| 3 2^-24 from the exponent's three roundings
(log2 e, product, difference): 2^-22 + 1.8e-7 for a <= 1.  Three products and their sums in the tensor core, cut off: 3 2^-23.  The
sum of weights: the same 2^-22 + 1.8e-7, at most half of it counting.  The division: 2^-23.  Together under 1.2e-6 (PLAIN).  A third
part that is missing leaves up to 2^-18 = 3.8e-6 of p, a second one up to 2^-9."""
import numpy as np
import pytest

import workloads as WL
from helpers import dev, host

PLAIN = 1.2e-6
FAR = -200.0                                      # a score whose weight is 0 in float32


def bf16(x):
    return WL.bf16_bits_to_f32(WL.f32_to_bf16_bits(np.asarray(x, np.float32))).astype(np.float64)


def in_parts(p, parts):
    """p as a sum of so many bf16 numbers."""
    total = np.zeros_like(p)
    for _ in range(parts):
        total = total + bf16(p - total)
    return total


def scores(n):
    """n values a in (0, 1] that bf16 holds."""
    return (128 + np.arange(n) % 128 + 1) / 256.0


def tolerance(out, want, p):
    """bf16 weights in two parts are off by 2^-18 of themselves, and v0 = -bf16(p) makes both terms as large as p."""
    if out == "f32":
        return PLAIN * np.abs(want) + 2.0 ** -24 * np.abs(want)
    return (2 * p / (1 + p)) * (2.0 ** -18 + PLAIN) + 2.0 ** -8 * np.abs(want)


def test_the_tolerances_tell_a_lost_part():
    a = scores(128)
    p = np.exp(-a)
    want = p / (1 + p)
    err = lambda parts: np.abs(in_parts(p, parts) / (1 + p) - want)  # noqa: E731
    assert (err(3) <= tolerance("f32", want, p)).all()
    assert (err(2) > tolerance("f32", want, p)).mean() > 0.2
    want = (p - bf16(p)) / (1 + p)
    err = lambda parts: np.abs((in_parts(p, parts) - bf16(p)) / (1 + p) - want)  # noqa: E731
    assert (err(2) <= tolerance("bf16", want, p)).all()
    assert (err(1) > tolerance("bf16", want, p)).mean() > 0.5


@pytest.fixture(scope="module")
def K():
    from kv_cache_gqa_gb300 import build
    build.build_library(verbose=False)
    import kv_cache_gqa_gb300 as K
    return K


def batch_of(K, new, G, out, Dk, Dv, page=16):
    """Sequences of new[b] tokens, one KV head: slots 0 and 1 hold the keys that count, the others score FAR.  Row (token, head) of
    a sequence has unit vector number (token * G + head) % Dk."""
    import torch
    B = len(new)
    pools = [np.zeros((B * 32 // page, 1, page, D), np.float32) for D in (Dk, Dv)]
    per = 32 // page                                                     # 32 slots a sequence
    lengths = np.array([n + 1 for n in new], np.int32)                   # the first token sees slots 0 and 1
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    a = scores(B * Dk).reshape(B, Dk)
    for b in range(B):
        k, v = (p[b * per:(b + 1) * per, 0].reshape(32, -1) for p in pools)
        k[2:] = FAR
        k[1] = -a[b]
        v[1] = 1.0
        v[2:] = 3.0
        if out == "bf16":                                                # dim d answers to rows whose unit vector is d
            d = np.arange(min(Dk, Dv))
            v[0, d] = -bf16(np.exp(-a[b, d]))
    q = np.zeros((int(start[-1]), G, Dk), np.float32)
    unit = [(t * G + h) % min(Dk, Dv) for n in new for t in range(n) for h in range(G)]
    q.reshape(-1, Dk)[np.arange(len(unit)), unit] = 1.0
    table = np.arange(B * per, dtype=np.int32).reshape(B, per)
    cache = K.PagedKVCache(*(dev(p, torch.bfloat16) for p in pools))
    batch = K.PagedBatch(dev(table), dev(lengths), dev(start), lengths, start, table)
    o = torch.empty((len(q), G, Dv), dtype=torch.float32 if out == "f32" else torch.bfloat16, device="cuda")
    ws = torch.zeros(K.paged_workspace_bytes(1, G, Dv), dtype=torch.uint8, device="cuda")
    K.kv_attn_paged(dev(q, torch.bfloat16), cache, batch, o, ws, scale=1.0)
    torch.cuda.synchronize()
    seq = np.repeat(np.arange(B), np.asarray(new) * G)
    p = np.exp(-a[seq, unit])
    got = host(o).reshape(-1, Dv)
    if out == "bf16":
        return got[np.arange(len(unit)), unit], (p - bf16(p)) / (1 + p), p
    return got, np.repeat((p / (1 + p))[:, None], Dv, 1), np.repeat(p[:, None], Dv, 1)


def check(K, new, G, out, Dk, Dv):
    got, want, p = batch_of(K, new, G, out, Dk, Dv)
    err, tol = np.abs(got - want), tolerance(out, want, p)
    assert (err <= tol).all(), f"worst error {np.max(err / tol):.2f} of the tolerance"


DIMS = [(64, 64), (128, 128), (192, 128)]


@pytest.mark.gpu
@pytest.mark.parametrize("Dk,Dv", DIMS)
@pytest.mark.parametrize("new,G", [([1] * 20, 8), ([1] * 9, 2), ([1] * 12, 16), ([2, 1, 4], 4), ([3, 1, 8], 9), ([20, 7], 1), ([25, 1], 3)])
def test_float32_results_have_weights_of_24_bits(K, new, G, Dk, Dv):
    """Up to 8 rows a KV head, up to 16, and more."""
    check(K, new, G, "f32", Dk, Dv)


@pytest.mark.gpu
@pytest.mark.parametrize("Dk,Dv", DIMS)
@pytest.mark.parametrize("new,G", [([1] * 20, 8), ([1] * 9, 2), ([2, 1, 2], 4)])
def test_bf16_results_of_few_rows_have_weights_of_16_bits(K, new, G, Dk, Dv):
    check(K, new, G, "bf16", Dk, Dv)


@pytest.mark.gpu
@pytest.mark.parametrize("Dk,Dv", DIMS)
def test_sums_over_a_long_run(K, Dk, Dv):
    """304 sequences over the same 32768 slots, one run each: a warp adds 512 tiles.  Additions that round to nearest wander by
    sqrt(512 / 12) 2^-23 / sqrt(3) = 4.5e-7 of the sum (its running value grows evenly), those of the weights as much again (two a
    tile): 6 standard deviations of both are 4e-6.  Sums cut off towards zero lose
    about half a step an addition, always the same way: 1e-5."""
    import torch
    B, L, page = 304, 32768, 256
    r = np.random.default_rng(41)
    pools = [np.zeros((L // page, 1, page, D), np.float32) for D in (Dk, Dv)]
    a = r.integers(0, 129, L) / 128.0                                    # a key's score is minus its a, in dim 0
    pools[0][:, 0, :, 0] = -a.reshape(-1, page)
    v = r.integers(64, 129, (L, Dv)) / 128.0
    pools[1][:, 0] = v.reshape(-1, page, Dv)
    q = np.zeros((B, 1, Dk), np.float32)
    size = (1 + np.arange(B) % 100) / 128.0
    q[:, 0, 0] = size
    lengths = np.full(B, L, np.int32)
    start = np.arange(B + 1, dtype=np.int32)
    table = np.tile(np.arange(L // page, dtype=np.int32), (B, 1))
    cache = K.PagedKVCache(*(dev(p, torch.bfloat16) for p in pools))
    batch = K.PagedBatch(dev(table), dev(lengths), dev(start), lengths, start, table)
    o = torch.empty((B, 1, Dv), device="cuda")
    ws = torch.zeros(K.paged_workspace_bytes(1, 1, Dv), dtype=torch.uint8, device="cuda")
    K.kv_attn_paged(dev(q, torch.bfloat16), cache, batch, o, ws, scale=1.0)
    torch.cuda.synchronize()
    w = np.exp(-size[:, None] * a)
    want = (w @ v) / w.sum(1, keepdims=True)
    err = np.abs(host(o)[:, 0] - want) / want
    assert err.max() <= 4e-6 + PLAIN, err.max()


@pytest.mark.gpu
@pytest.mark.parametrize("Dk,Dv", DIMS)
@pytest.mark.parametrize("new,G", [([1, 8, 1, 1], 2), ([1, 2, 1], 8), ([1] * 5 + [16], 1)])
def test_a_neighbour_takes_no_bits(K, new, G, Dk, Dv):
    """Sequences of up to 16 rows a KV head keep 16 bits, whoever shares their batch."""
    check(K, new, G, "bf16", Dk, Dv)
