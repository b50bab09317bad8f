"""Long chunks over the paged cache in bf16 and float32, far pages, and captured calls: the cases of test_gpu_paged_cache.py in
the forms that only long sequences reach.  Tolerances are the ones derived there."""
import numpy as np
import pytest

from helpers import dev, host
from test_gpu_paged_cache import K, Case, attend, check_attention, dtype, values  # noqa: F401

pytestmark = pytest.mark.gpu

CHUNKS = [  # new tokens, lengths, page, Hq, Hkv, Dk, Dv
    ([300, 1, 129, 64], [4500, 30, 129, 3100], 16, 16, 8, 128, 128),     # units of many runs, runs of many units
    ([257], [257], 64, 8, 2, 128, 128),                                  # a prompt from its first token on
    ([65, 66], [2000, 2500], 32, 2, 1, 64, 64),                          # one row tile, and a pair whose second has four rows
    ([17], [5000], 128, 16, 16, 128, 128),                               # 17 rows over a long prefix: both slots on one tile
    ([40, 90], [1300, 90], 256, 5, 1, 128, 128),                         # 128 rows are not whole tokens
    ([30, 31], [700, 31], 16, 40, 2, 192, 128),                          # 20 heads a KV head
    ([150], [1111], 64, 6, 2, 192, 128),
    ([3, 9], [999, 9], 16, 64, 1, 64, 64),                               # two tokens a row tile
    ([100, 100, 100], [100, 20, 0], 16, 4, 2, 128, 128),                 # chunks longer than their sequence: rows of zeros
    ([128, 127, 1], [2049, 2047, 2048], 16, 4, 4, 128, 128),             # lengths about a tile's end
]


@pytest.mark.parametrize("cache,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("i", range(len(CHUNKS)))
def test_chunks(K, i, cache, out):  # noqa: F811
    c = Case(K, 100 + i, *CHUNKS[i], cache=cache).fill()
    q, got = attend(K, c, out)
    check_attention(got, q, c, out)


def test_a_call_twice_and_replayed_gives_the_same_bits(K):  # noqa: F811
    """Units that several CTAs join included."""
    import torch
    c = Case(K, 120, [200, 1, 40], [1900, 1500, 700], 16, 8, 2, 128, 128).fill()
    cache, batch = c.on_gpu(K)
    q = dev(values(c.r, (241, 8, 128), "bf16"), torch.bfloat16)
    ws, outs = c.workspace(K), [torch.empty((241, 8, 128), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    K.kv_attn_paged(q, cache, batch, outs[0], ws)
    K.kv_attn_paged(q, cache, batch, outs[1], ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.kv_attn_paged(q, cache, batch, outs[2], ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("cache", ["bf16", "f32"])
def test_captured_chunk_follows_the_device_lengths(K, cache):  # noqa: F811
    """bf16 outputs of a replayed chunk whose sequences are shorter than the mirror says, down to nothing."""
    import torch
    c = Case(K, 121, [60, 1, 20], [2500, 90, 300], 16, 4, 2, 128, 128, cache=cache).fill()
    pool, batch = c.on_gpu(K)
    q = values(c.r, (81, 4, 128), cache)
    qd, o, ws = dev(q, dtype(cache)), torch.empty((81, 4, 128), dtype=torch.bfloat16, device="cuda"), c.workspace(K)
    K.kv_attn_paged(qd, pool, batch, o, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.kv_attn_paged(qd, pool, batch, o, ws)
    for lens in ([2500, 90, 300], [61, 1, 25], [30, 80, 20], [1499, 0, 0]):
        batch.lengths.copy_(dev(np.asarray(lens, np.int32)))
        g.replay()
        torch.cuda.synchronize()
        c.lengths = np.asarray(lens, np.int32)
        check_attention(host(o), q, c, "bf16")


def test_two_graphs_on_one_workspace(K):  # noqa: F811
    """Two captured calls of other shapes, replayed in turn on one stream and one workspace."""
    import torch
    ws = torch.zeros(K.paged_workspace_bytes(2, 8, 128), dtype=torch.uint8, device="cuda")
    steps = []
    for seed, new, lens in ((122, [90, 1], [1500, 2600]), (123, [1, 1, 33], [900, 3000, 1700])):
        c = Case(K, seed, new, lens, 32, 8, 2, 128, 128).fill()
        pool, batch = c.on_gpu(K)
        q = values(c.r, (sum(new), 8, 128), "bf16")
        qd, o = dev(q, torch.bfloat16), torch.empty((sum(new), 8, 128), dtype=torch.bfloat16, device="cuda")
        K.kv_attn_paged(qd, pool, batch, o, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            K.kv_attn_paged(qd, pool, batch, o, ws)
        steps.append((c, q, o, g, pool, batch, qd))
    for _ in range(3):
        for s in steps:
            s[2].fill_(7)
            s[3].replay()
    torch.cuda.synchronize()
    for c, q, o, *_ in steps:
        check_attention(host(o), q, c, "bf16")


@pytest.mark.parametrize("cache,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_a_bad_page_costs_its_sequence_only(K, cache, out):  # noqa: F811
    """Page ids below and beyond the pool: NaN for the tokens that see them; the other sequences are as they were."""
    import torch
    c = Case(K, 124, [40, 40, 1, 1], [90, 900, 40, 700], 16, 4, 2, 128, 128, cache=cache).fill()
    pool, _ = c.on_gpu(K)
    q = values(c.r, (82, 4, 128), cache)
    table = c.table.copy()
    table[1, 30], table[3, 2] = -1, 2 ** 31 - 1
    batch = K.PagedBatch(dev(table), dev(c.lengths), dev(c.start), c.lengths, c.start)
    o = torch.empty((82, 4, 128), dtype=dtype(out), device="cuda")
    ws = c.workspace(K)
    K.kv_attn_paged(dev(q, dtype(cache)), pool, batch, o, ws)
    torch.cuda.synchronize()
    got = host(o)
    assert np.isnan(got[40:80]).all() and np.isnan(got[81]).all()
    assert not np.isnan(got[:40]).any() and not np.isnan(got[80]).any()
    got[40:80], got[81] = 0, 0
    from oracle import paged_oracle as P
    want, size = P.paged_attention(q, c.pool_k.astype(np.float64), c.pool_v.astype(np.float64), c.table, c.lengths, c.start)
    keep = np.r_[0:40, 80]
    weight = 0.0 if cache == "f32" else (2.0 ** -8 if out == "bf16" else 2.0 ** -16)
    half = 2.0 ** -8 if out == "bf16" else 2.0 ** -24
    tol = size * (weight + 1e-5) + np.abs(want) * half * (1 + weight)
    assert (np.abs(got - want)[keep] <= tol[keep]).all()
    o2 = torch.empty_like(o)                                             # and the workspace is as good as before
    good = K.PagedBatch(dev(c.table), dev(c.lengths), dev(c.start), c.lengths, c.start, c.table)
    K.kv_attn_paged(dev(q, dtype(cache)), pool, good, o2, ws)
    torch.cuda.synchronize()
    check_attention(host(o2), q, c, out)


@pytest.mark.parametrize("cache", ["bf16", "f32"])
def test_pages_farther_apart_than_32_bits(K, cache):  # noqa: F811
    """Append, attention of a token, a block and a chunk, and reordering, over pages that lie more than 2^31 elements from the
    pool's start (a layer of a pool whose layers alternate)."""
    import torch
    page, Hkv, D, n_pages = 64, 2, 64, 9
    gap = 2 ** 28 + 8 * page                                             # elements between pages: page 8 is beyond 2^31
    if torch.cuda.mem_get_info()[0] < 2 * 4 * 9 * gap + 2 ** 30:
        pytest.skip("needs 21 GB of device memory")
    one = Hkv * page * D
    flat = [torch.empty((n_pages - 1) * gap + one, dtype=dtype(cache), device="cuda") for _ in range(2)]
    far = [f.as_strided((n_pages, Hkv, page, D), (gap, page * D, D, 1)) for f in flat]
    for f in far:
        f.zero_()
    pool = K.PagedKVCache(*far)
    r = np.random.default_rng(125)
    new, lens = np.array([1, 4, 50]), np.array([130, 70, 200], np.int32)
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    table = np.array([[0, 7, 8, 0], [2, 1, 0, 0], [3, 4, 5, 6]], np.int32)
    k_old, v_old = (values(r, (n_pages, Hkv, page, D), cache) for _ in range(2))
    for p in range(n_pages):
        far[0][p] = dev(k_old[p], dtype(cache))
        far[1][p] = dev(v_old[p], dtype(cache))
    T = int(start[-1])
    q, k, v = (values(r, (T, h, D), cache) for h in (4, Hkv, Hkv))
    batch = K.PagedBatch(dev(table), dev(lens), dev(start), lens, start, table)
    K.kv_cache_append_paged(None, dev(k, dtype(cache)), dev(v, dtype(cache)), None, pool, batch, None, K.Rope("none"))
    torch.cuda.synchronize()
    from oracle import paged_oracle as P
    pk, pv = k_old.astype(np.float64), v_old.astype(np.float64)
    P.paged_append(k, v, pk, pv, table, lens, start, cache)
    got_k, got_v = (np.stack([host(f[p].contiguous()) for p in range(n_pages)]) for f in far)
    assert np.array_equal(got_k, pk) and np.array_equal(got_v, pv)
    want, size = P.paged_attention(q, pk, pv, table, lens, start)
    ws = torch.zeros(K.paged_workspace_bytes(Hkv, 4, D), dtype=torch.uint8, device="cuda")
    for out in ("bf16", "f32"):
        o = torch.empty((T, 4, D), dtype=dtype(out), device="cuda")
        K.kv_attn_paged(dev(q, dtype(cache)), pool, batch, o, ws)
        torch.cuda.synchronize()
        weight = 0.0 if cache == "f32" else (2.0 ** -8 if out == "bf16" else 2.0 ** -16)
        half = 2.0 ** -8 if out == "bf16" else 2.0 ** -24
        assert (np.abs(host(o) - want) <= size * (weight + 1e-5) + np.abs(want) * half * (1 + weight)).all(), out
    i32 = lambda x: dev(np.asarray(x, np.int32))  # noqa: E731
    beams = np.array([[[0, 7, 0], [1, 8, 0]]], np.int32)                 # the last page of beam 1 is page 8: copied to page 6
    L = np.full((1, 2), 100, np.int32)
    to, lo, so = i32(np.zeros((1, 2, 3))), i32(L), i32([[0, 0]])
    K.kv_cache_reorder_paged(pool, i32([[1, 1]]), i32(beams), i32(L), L, i32([[5, 6]]), to, lo, so)
    torch.cuda.synchronize()
    pk[6, :, :36], pv[6, :, :36] = pk[8, :, :36], pv[8, :, :36]
    got_k, got_v = (np.stack([host(f[p].contiguous()) for p in range(n_pages)]) for f in far)
    assert np.array_equal(got_k, pk) and np.array_equal(got_v, pv)
    assert to.cpu().numpy()[0, :, :2].tolist() == [[1, 8], [1, 6]] and so.cpu().numpy().tolist() == [[5, 7]]


@pytest.mark.parametrize("spread", [0.0, 30.0, 1e30])
def test_selection_of_slices_of_unequal_size(K, spread):  # noqa: F811
    """Rows whose parts differ by e^30 or by powers that no float32 holds, and many equal values at the bound."""
    import torch
    from test_gpu_beams import check, select
    from oracle import paged_oracle as P
    r = np.random.default_rng(126)
    z = r.standard_normal((2, 3, 40001)).astype(np.float32)
    z[:, :, ::3] = np.round(z[:, :, ::3])
    z[0, :, 20000:] -= np.float32(spread)
    z[1, 1, :10] += np.float32(spread)
    s = -r.random((2, 3)).astype(np.float32)
    check(select(K, torch.from_numpy(z).cuda(), s, 32), P.beam_step(z, s, 32))
