"""A prepared call keeps what it was made from, whatever becomes of the descriptors that named it."""
import gc
import weakref

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


def parts(K, seed):
    r = np.random.default_rng(seed)
    pools = [r.standard_normal((6, 1, 16, 64)).astype(np.float32) for _ in range(2)]
    table = np.array([[0, 3, 0], [5, 1, 2]], np.int32)
    lengths, start = np.array([20, 37], np.int32), np.array([0, 1, 4], np.int32)
    cache = K.PagedKVCache(*(dev(p) for p in pools))
    batch = K.PagedBatch(dev(table), dev(lengths), dev(start), lengths.copy(), start.copy(), table.copy())
    return r, pools, table, lengths, start, cache, batch


def replace(cache, batch):
    """Every tensor and host array of the descriptors is another one; what they held before, weakly."""
    held = []
    for x, names in ((cache, ("k", "v")), (batch, ("table", "lengths", "token_start", "lengths_host", "token_start_host", "table_host"))):
        for name in names:
            old = getattr(x, name)
            held.append(weakref.ref(old))
            setattr(x, name, old.copy() if isinstance(old, np.ndarray) else old.clone())
            del old
    gc.collect()
    return held


def test_attention_over_pages(K):
    import torch
    r, pools, table, lengths, start, cache, batch = parts(K, 1)
    q = r.standard_normal((4, 2, 64)).astype(np.float32)
    qd, o = dev(q), torch.empty((4, 2, 64), device="cuda")
    call = K.prepare_attn_paged(qd, cache, batch, o, torch.zeros(K.paged_workspace_bytes(1, 2, 64), dtype=torch.uint8, device="cuda"))
    held = replace(cache, batch)
    assert all(w() is not None for w in held)
    cache.k.zero_()
    call()
    torch.cuda.synchronize()
    want, _ = P.paged_attention(q, pools[0], pools[1], table, lengths, start)
    assert np.abs(host(o) - want).max() < 1e-4


def test_append_over_pages(K):
    import torch
    r, pools, table, lengths, start, cache, batch = parts(K, 2)
    k, v = (r.standard_normal((4, 1, 64)).astype(np.float32) for _ in range(2))
    call = K.prepare_append_paged(None, dev(k), dev(v), None, cache, batch, None, K.Rope("none"))
    was = cache.k, cache.v
    held = replace(cache, batch)
    assert all(w() is not None for w in held)
    call()
    torch.cuda.synchronize()
    P.paged_append(k, v, *pools, table, lengths, start, "f32")
    assert all(np.array_equal(host(t), p) for t, p in zip(was, pools))


def test_reordering(K):
    import torch
    _, _, _, _, _, cache, _ = parts(K, 3)
    i32 = lambda x: dev(np.asarray(x, np.int32))  # noqa: E731
    L = np.array([[5, 5]], np.int32)
    args = [i32([[1, 1]]), i32([[[0], [1]]]), i32(L), L, i32([[2, 3]]), i32([[[9], [9]]]), i32([[0, 0]]), i32([[0, 0]])]
    call = K.prepare_reorder_paged(cache, *args)
    held = [weakref.ref(cache.k), weakref.ref(cache.v)]
    cache.k, cache.v = cache.k.clone(), cache.v.clone()
    gc.collect()
    assert all(w() is not None for w in held)
    call()
    torch.cuda.synchronize()
    assert args[5].cpu().numpy().tolist() == [[[1], [3]]]


def test_the_other_caches(K):
    """The fixed windows' descriptors and the 4-bit ones."""
    import torch
    lengths = np.array([9], np.int32)
    q, o = torch.randn((1, 1, 2, 64), device="cuda"), torch.empty((1, 1, 2, 64), device="cuda")
    q4 = K.KVCacheQ4.zeros(1, 1, 64, 64)
    ws = torch.zeros(K.decode_q4_workspace_bytes(1, 1, 2, 1, 64, 64), dtype=torch.uint8, device="cuda")
    call = K.prepare_decode_q4(q, q4, dev(lengths), lengths, o, ws)
    held = [weakref.ref(getattr(q4, n)) for n in ("k", "v", "k_scale", "v_scale")]
    for n in ("k", "v", "k_scale", "v_scale"):
        setattr(q4, n, getattr(q4, n).clone())
    gc.collect()
    assert all(w() is not None for w in held)
    call()
    plain = K.KVCache(torch.zeros((1, 1, 64, 64), device="cuda"), torch.zeros((1, 1, 64, 64), device="cuda"))
    dws = torch.zeros(K.decode_workspace_bytes(1, 1, 2, 64, 64), dtype=torch.uint8, device="cuda")
    k = torch.zeros((1, 1, 64), device="cuda")
    call = K.prepare_decode_step(q[:, 0], k, k, torch.zeros((1, 1), dtype=torch.int32, device="cuda"), plain, dev(lengths), lengths,
                                 o[:, 0], dws, K.Rope("1d", 1e4))
    held = [weakref.ref(plain.k), weakref.ref(plain.v)]
    plain.k, plain.v = plain.k.clone(), plain.v.clone()
    gc.collect()
    assert all(w() is not None for w in held)
    torch.cuda.synchronize()
