"""GPU parity of lmhead_logprobs against the float64 definition (oracle/q4_oracle.py logprobs).

Tolerances: a float32 hidden row meets a bf16 table as two bf16 halves, each product off by at most
2^-18 of itself (float32 and bf16 operands: exact products), and float32 sums of H products add less
than sqrt(H) 2^-24; so a logit is off by at most 2^-18 sum |W h| and, roundings being independent,
by well under 1e-5 of sqrt(sum (W h)^2) + |z|.  The inputs have |z| < 40: 4e-4 would be the worst
case, 2e-5 (1 + |z|max / 10) is the bound used for lse, logprob and entropy.  The listed tokens are
ordered by logits of about twice float32 precision over a row normalised in float32 (2^-23): they
have to be the definition's wherever its neighbouring logits differ by more than 1e-6 (1 + |z|max).
"""
import zlib

import numpy as np
import pytest

import workloads as WL
from helpers import dev, host
from oracle import q4_oracle as Q

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


def run(K, h, W, V, k, norm=None, targets=None, eps=1e-6):
    torch = _torch()
    B, H = h.shape
    out = {n: torch.full((B,), float("nan"), device="cuda") for n in ("lp", "ent", "lse")}
    ids = torch.full((B, k), -7, dtype=torch.int32, device="cuda")
    top = torch.full((B, k), float("nan"), device="cuda")
    ws = torch.full((K.lmhead_logprobs_workspace_bytes(B, H, V, k),), 0xFF, dtype=torch.uint8, device="cuda")
    got = []
    for _ in range(2):
        K.lmhead_logprobs(h, W, ws, targets=targets, out_logprob=out["lp"] if targets is not None else None,
                          out_entropy=out["ent"], out_lse=out["lse"], top_ids=ids if k else None,
                          top_logprobs=top if k else None, norm_w=norm, eps=eps, V=V)
        torch.cuda.synchronize()
        got.append([host(out["lp"]), host(out["ent"]), host(out["lse"]), ids.cpu().numpy().copy(), host(top)])
    for a, b in zip(*got):
        assert np.array_equal(a, b, equal_nan=True), "two calls differ"
    return got[0]


def check(got, h, W, V, k, norm, targets, eps=1e-6):
    lp, ent, lse, ids, top = got
    B = h.shape[0]
    r_lp, r_ent, r_lse, _, _ = Q.logprobs(h, W, V, targets=targets, norm_w=norm, eps=eps)
    full_k = min(V, k + 1)
    _, _, _, r_ids, r_top = Q.logprobs(h, W, V, norm_w=norm, eps=eps, top_k=full_k)
    z = r_top + r_lse[:, None]
    zmax = np.abs(z[:, :1]).max() if full_k else 20.0
    tol = 2e-5 * (1 + zmax / 10)
    assert np.max(np.abs(lse - r_lse)) <= tol and np.max(np.abs(ent - r_ent)) <= tol
    if targets is not None:
        assert np.allclose(lp, r_lp, rtol=0, atol=tol, equal_nan=True)
    if not k:
        return
    assert np.max(np.abs(top - r_top[:, :k])) <= tol
    for b in range(B):
        assert len(set(ids[b].tolist())) == k and ids[b].min() >= 0 and ids[b].max() < V
        for r in range(k):
            near = [abs(z[b, r] - z[b, j]) for j in (r - 1, r + 1) if 0 <= j < full_k]
            if all(g > 1e-6 * (1 + zmax) for g in near):
                assert ids[b, r] == r_ids[b, r], (b, r, ids[b], r_ids[b])


def inputs(rng, B, H, V, wdt, hdt, norm, pull=20.0):
    torch = _torch()
    W = (0.02 * rng.standard_normal((V, H))).astype(np.float32)
    Wd = dev(W, torch.bfloat16) if wdt == "bf16" else dev(W)
    Wh = host(Wd)
    near = rng.integers(0, V, (B, 6))
    h = rng.standard_normal((B, H)) + np.einsum("bj,bjh->bh", pull * rng.random((B, 6)) * 1024 / H, Wh[near])
    hd = dev(h.astype(np.float32), torch.bfloat16 if hdt == "bf16" else None)
    nw = (1 + 0.1 * rng.standard_normal(H)).astype(np.float32) if norm else None
    targets = np.where(rng.random(B) < 0.5, near[:, 0], rng.integers(0, V, B)).astype(np.int32)
    return hd, Wd, Wh, nw, targets


CASES = [
    # B, H, V, table, h, norm, top_k
    (1, 1024, 20000, "bf16", "f32", True, 5), (1, 8, 1, "bf16", "f32", False, 1), (2, 64, 127, "bf16", "bf16", False, 24),
    (3, 128, 128, "bf16", "f32", True, 0), (5, 200, 1009, "bf16", "f32", True, 3), (7, 520, 4099, "f32", "f32", True, 8),
    (16, 192, 257, "bf16", "bf16", True, 10), (17, 1024, 3001, "bf16", "f32", True, 11), (64, 1024, 9001, "bf16", "f32", True, 8),
    (33, 72, 513, "f32", "bf16", False, 4), (127, 256, 2049, "bf16", "bf16", False, 1), (128, 256, 1025, "bf16", "f32", False, 20),
    (129, 128, 1000, "bf16", "f32", True, 5), (300, 64, 333, "bf16", "bf16", False, 2), (1100, 64, 777, "bf16", "f32", True, 1),
    (1, 2048, 5000, "bf16", "bf16", False, 24), (4, 4096, 640, "bf16", "f32", True, 6), (1, 64, 24, "f32", "f32", False, 24),
    (5, 64, 100, "bf16", "f32", True, 13), (70, 128, 6001, "bf16", "f32", True, 20), (2, 128, 700, "bf16", "bf16", False, 21),
]


@pytest.mark.parametrize("B,H,V,wdt,hdt,norm,k", CASES)
def test_parity(K, B, H, V, wdt, hdt, norm, k):
    rng = seeded("logprobs", B, H, V, wdt, hdt, norm, k)
    hd, Wd, Wh, nw, targets = inputs(rng, B, H, V, wdt, hdt, norm)
    targets[0] = -100 if B > 2 else targets[0]
    if B > 3:
        targets[1], targets[2] = V, V - 1
    got = run(K, hd, Wd, V, k, dev(nw) if norm else None, dev(targets))
    check(got, host(hd), Wh, V, k, nw, targets)


# the streaming form's blocks of 1, 2, 4 and 8 rows, full and partly filled, long rows, more blocks than CTAs
@pytest.mark.parametrize("B,H,V,wdt,hdt,norm,k", [
    (2, 136, 333, "f32", "f32", True, 3), (3, 264, 1001, "f32", "bf16", True, 24), (4, 1024, 2050, "f32", "f32", True, 8),
    (8, 520, 70, "bf16", "f32", False, 12), (9, 4096, 515, "f32", "f32", True, 5), (2, 4096, 130, "f32", "bf16", False, 1),
    (2500, 8, 41, "f32", "f32", False, 2), (1, 4088, 260, "bf16", "bf16", True, 9), (3, 72, 90, "f32", "f32", False, 20)])
def test_streaming_form(K, B, H, V, wdt, hdt, norm, k):
    test_parity(K, B, H, V, wdt, hdt, norm, k)


@pytest.mark.parametrize("wdt,hdt,norm", [("bf16", "f32", True), ("bf16", "bf16", False), ("f32", "f32", True), ("f32", "bf16", False)])
def test_inputs_written_just_before_the_call(K, wdt, hdt, norm):
    """Rows and targets change between calls that follow each other without a pause: each call sees its own."""
    torch = _torch()
    rng = seeded("fresh", wdt, hdt, norm)
    B, H, V, calls = 3, 256, 2000, 6
    hd, Wd, Wh, nw, _ = inputs(rng, B, H, V, wdt, hdt, norm)
    nd = dev(nw) if norm else None
    rows = [dev((3 * rng.standard_normal((B, H))).astype(np.float32)).to(hd.dtype) for _ in range(calls)]
    picks = [rng.integers(0, V, B).astype(np.int32) for _ in range(calls)]
    pd = [dev(x) for x in picks]
    td = torch.zeros(B, dtype=torch.int32, device="cuda")
    ws = torch.empty(K.lmhead_logprobs_workspace_bytes(B, H, V, 1), dtype=torch.uint8, device="cuda")
    lps = torch.empty((calls, B), device="cuda")
    torch.cuda.synchronize()
    for i in range(calls):
        hd.copy_(rows[i])
        td.copy_(pd[i])
        K.lmhead_logprobs(hd, Wd, ws, targets=td, out_logprob=lps[i], norm_w=nd)
    torch.cuda.synchronize()
    for i in range(calls):
        want = Q.logprobs(host(rows[i]), Wh, V, targets=picks[i], norm_w=nw if norm else None)[0]
        assert np.allclose(host(lps[i]), want, rtol=0, atol=1e-4), f"call {i}"      # |z| < 40


def test_vocabulary_shorter_than_the_table_and_the_model_size(K):
    rng = seeded("qwen")
    B, H, rows, V = 3, WL.QWEN3_HIDDEN, WL.QWEN3_VOCAB, WL.QWEN3_VOCAB - 267
    hd, Wd, Wh, nw, targets = inputs(rng, B, H, rows, "bf16", "f32", True)
    Wd[V:] = 9.0                                               # rows past the vocabulary: not candidates
    targets[:] = [5, V - 1, V]
    got = run(K, hd, Wd, V, 8, dev(nw), dev(targets))
    check(got, host(hd), Wh, V, 8, nw, targets)


@pytest.mark.parametrize("wdt,H", [("bf16", 128), ("f32", 128), ("bf16", 72)])
def test_ties_go_to_the_lower_id(K, wdt, H):
    """Equal rows all over the table, more of them than the list holds."""
    rng = seeded("ties", wdt)
    B, V, k = 4, 3000, 12
    torch = _torch()
    W = (0.02 * rng.standard_normal((V, H))).astype(np.float32)
    best = rng.choice(V, 60, replace=False)
    W[best] = 0.3 * np.sign(W[7])
    Wd = dev(W, torch.bfloat16) if wdt == "bf16" else dev(W)
    h = dev((np.abs(rng.standard_normal((B, H))) * np.sign(W[7])).astype(np.float32))
    lp, ent, lse, ids, top = run(K, h, Wd, V, k)
    for b in range(B):
        assert list(ids[b]) == sorted(best.tolist())[:k]
        assert len(set(top[b].tolist())) == 1
    # a table of zeros: every logit 0
    lp, ent, lse, ids, top = run(K, h, torch.zeros_like(Wd), V, k, targets=dev(np.array([0, 5, -1, V], np.int32)))
    assert np.all(ids == np.arange(k)) and np.allclose(top, -np.log(V), atol=1e-6) and np.allclose(ent, np.log(V), atol=1e-5)
    assert np.allclose(lp[:2], -np.log(V), atol=1e-6) and lp[2] == 0 and np.isnan(lp[3])


def test_certain_rows(K):
    """One token takes the row: entropy and logprob near 0, lse near the logit, nothing overflows."""
    rng = seeded("certain")
    torch = _torch()
    H, V = 256, 5000
    W = (0.02 * rng.standard_normal((V, H))).astype(np.float32)
    Wd = dev(W, torch.bfloat16)
    Wh = host(Wd)
    pick = np.array([0, 4999, 2500])
    h = (Wh[pick] * 5000).astype(np.float32)                   # logits of about 500
    lp, ent, lse, ids, top = run(K, dev(h), Wd, V, 2, targets=dev(pick.astype(np.int32)))
    z = h.astype(np.float64) @ Wh.T
    assert np.all(ids[:, 0] == pick) and np.all(np.abs(ent) < 1e-6) and np.all(np.abs(lp) < 500 * 2.0 ** -17)
    assert np.allclose(lse, z[np.arange(3), pick], rtol=2.0 ** -17)
    # the same rows shifted far down: every logit below -1000
    lp, ent, lse, ids, top = run(K, dev(-20 * np.abs(h)), dev(np.abs(W) + 0.02), V, 1)
    z = -20 * np.abs(h).astype(np.float64) @ (np.abs(W) + np.float32(0.02)).astype(np.float64).T
    assert np.allclose(lse, z.max(1) + np.log(np.exp(z - z.max(1, keepdims=True)).sum(1)), rtol=2.0 ** -20)


def test_capture_and_replay_on_another_stream(K):
    torch = _torch()
    rng = seeded("graph")
    B, H, V, k = 4, 1024, 3001, 5
    hd, Wd, Wh, nw, targets = inputs(rng, B, H, V, "bf16", "f32", True)
    nd, td = dev(nw), dev(targets)
    ws = torch.empty(K.lmhead_logprobs_workspace_bytes(B, H, V, k), dtype=torch.uint8, device="cuda")
    lp, ids, top = torch.empty(B, device="cuda"), torch.empty((B, k), dtype=torch.int32, device="cuda"), torch.empty((B, k), device="cuda")
    call = lambda: K.lmhead_logprobs(hd, Wd, ws, targets=td, out_logprob=lp, top_ids=ids, top_logprobs=top, norm_w=nd)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(2):
        h = rng.standard_normal((B, H)).astype(np.float32) * 3
        hd.copy_(torch.from_numpy(h))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            g.replay()
        side.synchronize()
        r_lp, _, _, r_ids, r_top = Q.logprobs(h, Wh, V, targets=targets, norm_w=nw, top_k=k)
        assert np.allclose(host(lp), r_lp, atol=5e-5) and np.allclose(host(top), r_top, atol=5e-5)
        assert np.array_equal(ids.cpu().numpy(), r_ids)
