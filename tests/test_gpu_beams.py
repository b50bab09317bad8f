"""Beam search on a GPU: the selection and the reordering against the fp64 definitions, and a small search as a whole."""
import math

import numpy as np
import pytest

from helpers import dev, host
from oracle import paged_oracle as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from kv_cache_gqa_gb300 import build
    build.build_library(verbose=False)
    import kv_cache_gqa_gb300 as K
    return K


def select(K, logits, scores, n, finished=None, end_id=0, ws=None):
    import torch
    B, Kb, V = logits.shape
    ws = torch.zeros(K.beam_workspace_bytes(B, Kb, V), dtype=torch.uint8, device="cuda") if ws is None else ws
    beam, token = (torch.empty((B, n), dtype=torch.int32, device="cuda") for _ in range(2))
    score = torch.empty((B, n), device="cuda")
    K.beam_select(logits, dev(scores.astype(np.float32)), beam, token, score, ws,
                  finished=None if finished is None else dev(finished.astype(np.int32)), end_id=end_id)
    torch.cuda.synchronize()
    assert not ws[:K.beam_workspace_zero_bytes()].any()
    return beam.cpu().numpy(), token.cpu().numpy(), host(score)


def check(got, want):
    """A total is off by half a step of float32 and by about 3e-8 of the sum's logarithm (exponentials off by 2^-22 each, mostly either way:
    1e-6 allows for all of them one way); two totals within that may change places, but not beams of equal rows."""
    beam, token, score = got
    for b, offers in enumerate(want):
        for j, (k, t, total) in enumerate(offers):
            if k < 0:
                assert beam[b, j] == -1 and token[b, j] == -1 and score[b, j] == -math.inf
                continue
            tol = 1e-6 + abs(total) * 2.0 ** -24
            assert abs(score[b, j] - total) <= tol, (b, j, score[b, j], total)
            near = {o[:2] for o in offers if abs(o[2] - total) <= 2 * tol}
            assert (beam[b, j], token[b, j]) in near, (b, j, beam[b, j], token[b, j], k, t)
        named = [(beam[b, j], token[b, j]) for j in range(len(offers)) if beam[b, j] >= 0]
        assert len(set(named)) == len(named)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("B,Kb,V,n,pad", [(1, 1, 1, 1, 0), (1, 4, 151936, 8, 0), (3, 5, 1000, 32, 5), (2, 32, 4097, 32, 0), (7, 3, 33, 6, 3),
                                          (1, 2, 5, 10, 0), (40, 8, 9001, 8, 7), (1, 1, 20000, 32, 0)])
def test_selection(K, B, Kb, V, n, pad, dt):
    """Odd sizes, rows at any alignment, bf16 logits with many equal values."""
    import torch
    r = np.random.default_rng(B + V)
    z = torch.from_numpy(r.standard_normal((B * Kb, V + pad)).astype(np.float32) * 2).cuda()
    z = z.to({"f32": torch.float32, "bf16": torch.bfloat16}[dt])[:, :V].unflatten(0, (B, Kb))
    scores = -10 * r.random((B, Kb)).astype(np.float32)
    check(select(K, z, scores, n), P.beam_step(host(z), scores, n))
    fin = r.random((B, Kb)) < 0.4
    first = np.where(np.arange(Kb) == 0, scores, -np.inf)
    check(select(K, z, scores, n, fin, V - 1), P.beam_step(host(z), scores, n, fin, V - 1))
    check(select(K, z, first, n), P.beam_step(host(z), first, n))


def test_selection_of_equal_and_sorted_rows(K):
    """Ties within a row go to the lower token, between equal beams to the lower beam; rising and falling rows, where every
    value or none of the later ones is better than what came before."""
    import torch
    V = 9000
    flat = torch.zeros((2, 3, V), device="cuda")
    beam, token, score = select(K, flat, np.zeros((2, 3)), 7)
    assert (beam == 0).all() and (token == np.arange(7)).all()
    steps = (torch.arange(V, device="cuda") // 100).float().expand(1, 4, V).contiguous() * 0.25
    beam, token, _ = select(K, steps, np.zeros((1, 4)), 20)
    assert (beam == 0).all() and (token == np.arange(V - 100, V)[:20]).all()
    for row in (torch.arange(V), torch.arange(V).flip(0)):
        z = (row.float().cuda() * 0.01).expand(1, 2, V).contiguous()
        s = np.array([[0.0, -0.005]])
        check(select(K, z, s, 32), P.beam_step(host(z), s, 32))


def test_selection_with_values_out_of_order(K):
    """-infinity is never offered; NaN and +infinity silence a beam; the type's lowest value is an ordinary one; a score of NaN offers nothing."""
    import torch
    r = np.random.default_rng(3)
    z = r.standard_normal((6, 4, 5000)).astype(np.float32)
    z[0, 0, 17], z[0, 1, 4999], z[0, 2, :] = np.nan, np.inf, -np.inf
    z[1, :, 3:] = -np.inf
    z[2] = -np.inf
    z[3, :, 1:] = np.finfo(np.float32).min
    z[4, 1] = np.finfo(np.float32).min
    scores = np.zeros((6, 4), np.float32)
    scores[5, 0], scores[5, 1] = np.nan, -np.inf
    want = P.beam_step(z, scores, 14)
    got = select(K, torch.from_numpy(z).cuda(), scores, 14)
    check([g[[0, 1, 2, 4, 5]] for g in got], [want[i] for i in (0, 1, 2, 4, 5)])
    assert (got[1][3, :4] == 0).all() and sorted(got[0][3, :4]) == [0, 1, 2, 3]
    assert (got[2][3, 4:] < -1e38).all()
    huge = torch.full((1, 2, 300), 3e38, device="cuda")
    beam, token, score = select(K, huge, np.zeros((1, 2)), 4)
    assert (beam == 0).all() and (token == np.arange(4)).all() and np.allclose(score, -math.log(300), atol=1e-6)


def test_selection_on_one_workspace_and_replayed(K):
    import torch
    ws = torch.zeros(K.beam_workspace_bytes(8, 8, 30000), dtype=torch.uint8, device="cuda")
    r = np.random.default_rng(4)
    for B, Kb in ((8, 8), (1, 2), (5, 3)):
        z = torch.from_numpy(r.standard_normal((B, Kb, 30000)).astype(np.float32)).cuda()
        s = -r.random((B, Kb)).astype(np.float32)
        check(select(K, z, s, 4, ws=ws), P.beam_step(host(z), s, 4))
    beam, token = (torch.empty((5, 4), dtype=torch.int32, device="cuda") for _ in range(2))
    score, sd = torch.empty((5, 4), device="cuda"), dev(s)
    call = lambda: K.beam_select(z, sd, beam, token, score, ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for seed in (5, 6):
        z.copy_(torch.from_numpy(np.random.default_rng(seed).standard_normal(z.shape).astype(np.float32)))
        g.replay()
        torch.cuda.synchronize()
        check((beam.cpu().numpy(), token.cpu().numpy(), host(score)), P.beam_step(host(z), s, 4))


# ---------------------------------------------------------------------------------
def reorder(K, pools, parent, table, lengths, spare):
    """The call on copies; outputs as arrays, pools as tensors."""
    import torch
    cache = K.PagedKVCache(*(torch.from_numpy(p.copy()).cuda().to(torch.bfloat16 if p.dtype == np.float64 else torch.float32)
                             for p in pools))
    i32 = lambda x: dev(np.asarray(x, np.int32))  # noqa: E731
    t = i32(table)
    to, lo, so = torch.full_like(t, -9), torch.empty_like(i32(lengths)), torch.empty_like(i32(spare))
    K.kv_cache_reorder_paged(cache, i32(parent), t, i32(lengths), np.maximum(np.asarray(lengths, np.int32), 0), i32(spare), to, lo, so)
    torch.cuda.synchronize()
    return to.cpu().numpy(), lo.cpu().numpy(), so.cpu().numpy(), cache.k, cache.v


@pytest.mark.parametrize("B,Kb,layers,page,Hkv,Dk,Dv,f32", [(1, 1, 1, 16, 1, 64, 64, False), (1, 4, 3, 16, 2, 128, 128, False),
                                                         (5, 3, 2, 32, 3, 192, 128, True), (3, 32, 1, 64, 1, 64, 256, False),
                                                         (30, 8, 2, 16, 2, 64, 64, False)])
def test_reordering(K, B, Kb, layers, page, Hkv, Dk, Dv, f32):
    r = np.random.default_rng(B * 100 + Kb)
    n_pages, W = 20 + 2 * B * Kb, 7
    ids = r.permutation(n_pages)
    pools = [r.integers(-120, 120, (layers, n_pages, Hkv, page, D)).astype(np.float32 if f32 else np.float64) for D in (Dk, Dv)]
    table = ids[r.integers(0, 20, (B, Kb, W))]
    lengths = np.repeat(r.integers(0, W * page + 1, (B, 1)), Kb, 1)
    if Kb > 2:
        lengths[0, 2] = min(W * page, lengths[0, 2] + 3)               # beams of unequal length, one group
    tails = ids[20:20 + B * Kb].reshape(B, Kb)
    for b in range(B):
        for k in range(Kb):
            if lengths[b, k] % page:
                table[b, k, lengths[b, k] // page] = tails[b, k]
    spare = ids[20 + B * Kb:].reshape(B, Kb)
    parent = r.integers(0, Kb, (B, Kb))
    if B > 1:
        parent[1] = -1 if Kb == 1 else np.where(np.arange(Kb) == 1, Kb, parent[1])
    want_pools = [p.astype(np.float64) for p in pools]
    rows, lens, spares = P.reorder(parent.tolist(), table.tolist(), lengths.tolist(), spare.tolist(), want_pools, n_pages)
    to, lo, so, k, v = reorder(K, pools, parent, table, lengths, spare)
    assert np.array_equal(lo, lens) and np.array_equal(so, spares)
    for b in range(B):
        for j in range(Kb):
            row = rows[b][j]
            assert (to[b, j, :len(row)] == row).all() and (to[b, j, len(row):] == -9).all()
    assert np.array_equal(host(k), want_pools[0]) and np.array_equal(host(v), want_pools[1])


def test_reordering_of_beams_that_share_a_page_and_without_spares(K):
    """After a prompt all beams name the same partly filled page; spares that are no pages; lengths below zero."""
    page = 16
    r = np.random.default_rng(1)
    pools = [r.integers(-99, 99, (2, 12, 2, page, 64)).astype(np.float64) for _ in range(2)]
    table = np.tile(np.array([0, 1, 2]), (3, 4, 1))
    lengths = np.array([[37] * 4, [37] * 4, [37, -1, 0, 32]])
    spare = np.array([[3, 4, 5, 6], [7, 12, -1, 8], [9, 10, 11, 3]])
    table[1, :, 2] = 2
    table[0, :, 2] = 1
    parent = np.array([[0, 1, 2, 3], [3, 3, 0, 1], [1, 0, 3, 2]])
    want = [p.copy() for p in pools]
    clean = np.maximum(lengths, 0)
    rows, lens, spares = P.reorder(parent.tolist(), table.tolist(), clean.tolist(), spare.tolist(), want, 12)
    to, lo, so, k, v = reorder(K, pools, parent, table, lengths, spare)
    assert np.array_equal(lo, lens) and np.array_equal(so, spares) and lens[1][1] == lens[1][2] == -1
    for b in range(3):
        for j in range(4):
            row = rows[b][j]
            assert (to[b, j, :len(row)] == row).all() and (to[b, j, len(row):] == -9).all()
    assert np.array_equal(host(k), want[0]) and np.array_equal(host(v), want[1])


def test_binding_refusals(K):
    import torch
    z = torch.zeros((2, 3, 50), device="cuda")
    s, ws = torch.zeros((2, 3), device="cuda"), torch.zeros(K.beam_workspace_bytes(2, 3, 50), dtype=torch.uint8, device="cuda")
    i = torch.zeros((2, 4), dtype=torch.int32, device="cuda")
    f = torch.zeros((2, 4), device="cuda")
    K.beam_select(z, s, i, i.clone(), f, ws)
    for args in ((z[..., ::2], s, i, i, f), (z.double(), s, i, i, f), (z, s[:1], i, i, f), (z, s, i.long(), i, f), (z, s, i, i[:, :2], f),
                 (z.transpose(0, 1), s.T, i, i, f), (z[0], s, i, i, f), (z, s, i, i, f.double()), (z[:, :1].expand(2, 3, 50), s, i, i, f)):
        with pytest.raises(K.KvaError):
            K.beam_select(*args, ws)
    with pytest.raises(K.KvaError):
        K.beam_select(z, s, i, i.clone(), f, ws[:100])
    c = K.PagedKVCache.zeros(5, 1, 16, 64, layers=2)
    p = torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    t = torch.zeros((2, 3, 2), dtype=torch.int32, device="cuda")
    lh = np.zeros((2, 3), np.int32)
    for args in ((p.long(), t, p, lh, p, t.clone(), p.clone(), p.clone()), (p, t, p, lh, p, t, p.clone(), p.clone()),
                 (p, t, p, lh[:1], p, t.clone(), p.clone(), p.clone()), (p, t, p, lh, p, t[:, :, :1], p.clone(), p.clone()),
                 (p, t, p, lh + 33, p, t.clone(), p.clone(), p.clone())):
        with pytest.raises(K.KvaError):
            K.kv_cache_reorder_paged(c, *args)
    torch.cuda.synchronize()


def test_a_search_over_pages(K):
    """Three beams over a toy model whose next-token logits come from attention over what was appended: the calls together, step
    by step, against every hypothesis carried along in 64 bits with a cache of its own."""
    import torch
    r = np.random.default_rng(11)
    Kb, V, D, page, W, steps, prompt = 3, 40, 64, 16, 4, 30, 13
    emb = (r.integers(-8, 9, (V, 3, D)) / 8).astype(np.float32)        # q, k, v of a token, exact in bf16
    head = (0.6 * r.standard_normal((V, D))).astype(np.float32)
    toks = r.integers(0, V, prompt)
    n_pages = 64
    free = list(range(n_pages))
    take = lambda: free.pop()  # noqa: E731
    cache = K.PagedKVCache.zeros(n_pages, 1, page, D, dtype=torch.float32)
    ws = torch.zeros(K.paged_workspace_bytes(1, 1, D), dtype=torch.uint8, device="cuda")
    bws = torch.zeros(K.beam_workspace_bytes(1, Kb, V), dtype=torch.uint8, device="cuda")
    first = [take() for _ in range(-(-prompt // page))]
    table = torch.zeros((1, Kb, W), dtype=torch.int32, device="cuda")
    table[0, :, :len(first)] = dev(np.asarray(first, np.int32))
    spare = dev(np.array([[take() for _ in range(Kb)]], np.int32))

    def step(tokens, tbl, lengths, start):
        batch = K.PagedBatch(tbl, dev(lengths), dev(start), lengths, start)
        e = dev(emb[tokens])
        q = torch.empty((len(tokens), 1, D), device="cuda")
        K.kv_cache_append_paged(e[:, 0:1], e[:, 1:2], e[:, 2:3], None, cache, batch, q, K.Rope("none"))
        o = torch.empty((len(tokens), 1, D), device="cuda")
        K.kv_attn_paged(q, cache, batch, o, ws)
        return o

    o = step(toks, table[0, :1].contiguous(), np.array([prompt], np.int32), np.array([0, prompt], np.int32))
    hidden = o[-1:].expand(Kb, 1, D)
    lengths = np.full((1, Kb), prompt, np.int32)
    scores = torch.tensor([[0.0, -math.inf, -math.inf]], device="cuda")
    hyps = [(list(toks), 0.0)]

    def ref_logits(seq):
        e = emb[seq].astype(np.float64)
        x = e[:, 1] @ e[-1, 0] / math.sqrt(D)
        w = np.exp(x - x.max())
        return head.astype(np.float64) @ (w @ e[:, 2] / w.sum())

    lens = dev(lengths)
    for i in range(steps):
        logits = (hidden[:, 0] @ dev(head).T)[None].contiguous()
        beam, token = (torch.empty((1, Kb), dtype=torch.int32, device="cuda") for _ in range(2))
        score = torch.empty((1, Kb), device="cuda")
        K.beam_select(logits, scores, beam, token, score, bws)
        to, lo, so = torch.zeros_like(table), torch.empty_like(lens), torch.empty_like(spare)
        K.kv_cache_reorder_paged(cache, beam, table, lens, lengths, spare, to, lo, so)
        torch.cuda.synchronize()
        ref = []
        for h, (seq, s) in enumerate(hyps):
            z = ref_logits(seq)
            z = z - z.max() - math.log(np.exp(z - z.max()).sum())
            ref += [(-(s + z[v]), h, v) for v in range(V)]
        ref = sorted(ref)
        got = [hyps[int(k)][0] + [int(t)] for k, t in zip(beam[0].tolist(), token[0].tolist())]
        want = [hyps[h][0] + [v] for _, h, v in ref[:Kb]]
        gaps = [ref[j + 1][0] - ref[j][0] for j in range(Kb)]
        if min(gaps) < 1e-3:                                          # nearly even: the order is not fixed
            want = got
        assert got == want, i
        assert np.allclose(host(score)[0], [-u for u, _, _ in ref[:Kb]], atol=1e-3)
        hyps = [(seq, float(s)) for seq, s in zip(got, host(score)[0])]
        so_h = so.cpu().numpy()
        so_h[so_h < 0] = [take() for _ in range(int((so_h < 0).sum()))]
        table, spare, scores = to, dev(so_h), score
        lengths = lo.cpu().numpy() + 1
        for b in range(Kb):                                           # a page for the new token where the last is full
            if (lengths[0, b] - 1) % page == 0:
                table[0, b, (lengths[0, b] - 1) // page] = take()
        lens = dev(lengths)
        hidden = step(token[0].cpu().numpy(), table[0].contiguous(), lengths[0], np.arange(Kb + 1, dtype=np.int32))
