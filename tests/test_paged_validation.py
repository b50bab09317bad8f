"""What the paged cache's and the beams' calls refuse before anything is launched (dummy addresses: hosts without a GPU)."""
import ctypes as C

import numpy as np
import pytest

AT = 1 << 20                         # a 16-byte aligned dummy address: never dereferenced, validation fails first


@pytest.fixture(scope="module")
def K():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("dummy addresses: runs on hosts without a GPU")
    from kv_cache_gqa_gb300 import build
    build.build_library(verbose=False)
    import kv_cache_gqa_gb300.kv_attn as K
    K.lib()
    return K


def cache(K, k=AT, v=AT, dtype=1, hkv=8, d=128, dv=0, page=16, n=100, ps=0, psv=0):
    return K._PagedCache(k, v, dtype, hkv, d, dv, page, n, ps, psv)


KEEP = []


def batch(K, lengths=(5,), start=(0, 1), stride=4, table=AT, table_host=None, B=None, dev=AT):
    lh, sh = np.asarray(lengths, np.int32), np.asarray(start, np.int32)
    th = None if table_host is None else np.asarray(table_host, np.int32)
    KEEP.append((lh, sh, th))
    return K._PagedBatch(table, stride, dev, dev, None if th is None else th.ctypes.data, lh.ctypes.data, sh.ctypes.data,
                         len(lengths) if B is None else B)


def rope(K, kind=1, n_axes=1, base=1e6, off=0, dim=0, secs=(0, 0, 0, 0)):
    return K._Rope(kind, n_axes, (C.c_int32 * 4)(*secs), base, off, dim)


def append(K, c=None, b=None, q=AT, qs=0, k=AT, ks=0, v=AT, vs=0, dt=1, Hq=16, pos=AT, norm=None, r=None, sc=None, qo=AT):
    return K.lib().kv_cache_append_paged(q, qs, k, ks, v, vs, dt, Hq, pos, norm or K._Norm(None, None, 0, 1e-6, 0),
                                         r or rope(K), sc or K._RopeScale(), qo, c or cache(K), b or batch(K), None)


def attn(K, c=None, b=None, q=AT, dt=1, Hq=16, out=AT, odt=1, ws=AT, wsb=1 << 30):
    return K.lib().kv_attn_paged(q, dt, c or cache(K), b or batch(K), Hq, 0.0, out, odt, ws, wsb, None)


def test_empty_calls_are_no_ops(K):
    for f in (append, attn):
        assert f(K, b=batch(K, (), (0,))) == K.KVA_OK
        assert f(K, b=batch(K, (3, 0), (0, 0, 0))) == K.KVA_OK                   # sequences without new tokens
        assert f(K, b=batch(K, B=-1)) == K.KVA_EINVAL


def test_cache_refusals(K):
    for f in (append, attn):
        for c, want in ((dict(k=None), K.KVA_EINVAL), (dict(v=None), K.KVA_EINVAL), (dict(dtype=2), K.KVA_EINVAL),
                        (dict(hkv=0), K.KVA_EINVAL), (dict(n=0), K.KVA_EINVAL), (dict(page=0), K.KVA_EINVAL),
                        (dict(page=8), K.KVA_EUNSUPPORTED), (dict(page=48), K.KVA_EUNSUPPORTED),
                        (dict(page=512), K.KVA_EUNSUPPORTED), (dict(d=72), K.KVA_EUNSUPPORTED),
                        (dict(d=320), K.KVA_EUNSUPPORTED), (dict(dv=100), K.KVA_EUNSUPPORTED), (dict(dv=-64), K.KVA_EINVAL),
                        (dict(ps=8 * 16 * 128 - 8), K.KVA_EINVAL), (dict(psv=-8), K.KVA_EINVAL),
                        (dict(ps=8 * 16 * 128 + 4), K.KVA_EALIGN), (dict(k=AT + 8), K.KVA_EALIGN)):
            assert f(K, c=cache(K, **c)) == want, (f.__name__, c)


def test_batch_refusals(K):
    for f in (append, attn):
        for b, want in ((dict(table=None), K.KVA_EINVAL), (dict(dev=None), K.KVA_EINVAL), (dict(stride=0), K.KVA_EINVAL),
                        (dict(start=(1, 2)), K.KVA_EINVAL), (dict(start=(0, -1)), K.KVA_EINVAL),
                        (dict(lengths=(5, 5), start=(0, 2, 1)), K.KVA_EINVAL),
                        (dict(lengths=(65,)), K.KVA_ECAPACITY), (dict(lengths=(-1,)), K.KVA_ECAPACITY),
                        (dict(lengths=(17,), table_host=[[3, 100, 0, 0]]), K.KVA_ECAPACITY),
                        (dict(lengths=(17,), table_host=[[-1, 3, 0, 0]]), K.KVA_ECAPACITY)):
            assert f(K, b=batch(K, **b)) == want, (f.__name__, b)
    assert append(K, b=batch(K, (1,), (0, 2))) == K.KVA_ECAPACITY                 # fewer slots than new tokens
    big = 1 << 30
    assert attn(K, c=cache(K, page=256), b=batch(K, ((1 << 31) - 1,), stride=big)) == K.KVA_ECAPACITY


def test_append_refusals(K):
    N = K._Norm
    for kw, want in ((dict(Hq=12), K.KVA_EINVAL), (dict(q=None), K.KVA_EINVAL), (dict(qo=None), K.KVA_EINVAL),
                     (dict(k=None), K.KVA_EINVAL), (dict(pos=None), K.KVA_EINVAL), (dict(dt=3), K.KVA_EINVAL),
                     (dict(norm=N(AT, None, 0, 1e-6, 0)), K.KVA_EINVAL), (dict(norm=N(AT, AT, 0, -1.0, 0)), K.KVA_EINVAL),
                     (dict(norm=N(AT + 4, AT, 0, 1e-6, 0)), K.KVA_EALIGN),
                     (dict(ks=8 * 128 + 4), K.KVA_EALIGN), (dict(q=AT + 8), K.KVA_EALIGN),
                     (dict(b=batch(K, (5,), (0, 2)), vs=8 * 128 - 8), K.KVA_EINVAL),
                     (dict(r=rope(K, off=8)), K.KVA_EINVAL), (dict(r=rope(K, kind=9)), K.KVA_EINVAL),
                     (dict(r=rope(K, kind=3, n_axes=1)), K.KVA_EINVAL),
                     (dict(sc=K._RopeScale(0.5, 0, 0, 0, 1)), K.KVA_EINVAL),
                     (dict(sc=K._RopeScale(float("nan"), 0, 0, 0, 1)), K.KVA_EINVAL),
                     (dict(sc=K._RopeScale(2, -1, 0, 0, 1)), K.KVA_EINVAL),
                     (dict(sc=K._RopeScale(2, 4096, 4, 4, 1)), K.KVA_EINVAL),
                     (dict(sc=K._RopeScale(2, 0, 0, 0, float("inf"))), K.KVA_EINVAL)):
        assert append(K, **kw) == want, kw


def test_attention_refusals(K):
    for kw, want in ((dict(Hq=12), K.KVA_EINVAL), (dict(dt=0), K.KVA_EINVAL), (dict(odt=5), K.KVA_EINVAL),
                     (dict(q=None), K.KVA_EINVAL), (dict(out=None), K.KVA_EINVAL), (dict(out=AT + 8), K.KVA_EALIGN),
                     (dict(ws=None), K.KVA_EWORKSPACE), (dict(wsb=1000), K.KVA_EWORKSPACE), (dict(ws=AT + 8), K.KVA_EALIGN),
                     (dict(c=cache(K, d=256)), K.KVA_EUNSUPPORTED), (dict(c=cache(K, d=192)), K.KVA_EUNSUPPORTED),
                     (dict(c=cache(K, d=64, dv=128)), K.KVA_EUNSUPPORTED), (dict(c=cache(K, hkv=1), Hq=65), K.KVA_EUNSUPPORTED)):
        assert attn(K, **kw) == want, kw
    size = K.lib().kva_paged_workspace_size
    assert size(8, 16, 128) == K.workspace_bytes("attn_paged", n_kv_heads=8, n_q_heads=16, head_dim=128) > 0
    assert size(8, 12, 128) == 0 and size(0, 8, 128) == 0 and 0 < K.lib().kva_paged_workspace_zero_bytes() < size(1, 1, 64)


def beam(K, logits=AT, dt=0, row=0, B=2, Kb=4, V=100, scores=AT, fin=None, end=0, n=4, o=AT, ws=AT, wsb=1 << 30):
    return K.lib().beam_select(logits, dt, row, B, Kb, V, scores, fin, end, n, o, AT, AT, ws, wsb, None)


def test_beam_refusals(K):
    assert beam(K, B=0) == K.KVA_OK
    for kw, want in ((dict(B=-1), K.KVA_EINVAL), (dict(Kb=0), K.KVA_EINVAL), (dict(Kb=33), K.KVA_EINVAL), (dict(n=0), K.KVA_EINVAL),
                     (dict(n=33), K.KVA_EINVAL), (dict(V=0), K.KVA_EINVAL), (dict(V=2, Kb=1, n=3), K.KVA_EINVAL),
                     (dict(row=99), K.KVA_EINVAL), (dict(dt=2), K.KVA_EINVAL), (dict(logits=None), K.KVA_EINVAL),
                     (dict(scores=None), K.KVA_EINVAL), (dict(o=None), K.KVA_EINVAL), (dict(fin=AT, end=100), K.KVA_EINVAL),
                     (dict(fin=AT, end=-1), K.KVA_EINVAL), (dict(B=4097), K.KVA_EUNSUPPORTED),
                     (dict(logits=AT + 2), K.KVA_EALIGN), (dict(ws=None), K.KVA_EWORKSPACE), (dict(wsb=100), K.KVA_EWORKSPACE)):
        assert beam(K, **kw) == want, kw
    size = K.lib().kva_beam_workspace_size
    for V in (1, 1000, 151936):                    # a workspace for the largest batch serves smaller ones
        last = 0
        for rows in range(1, 700):
            assert size(rows, 1, V) >= last
            last = size(rows, 1, V)
    assert K.workspace_bytes("beam_select", B=3, block=5, vocab=999) == size(3, 5, 999) > 0 == size(3, 33, 999)


def reorder(K, c=None, layers=1, ls=0, lsv=0, B=2, Kb=2, parent=AT, table=AT, stride=4, lengths=AT, lens=(5, 5, 5, 5), spare=AT,
            to=AT + 4096, lo=AT + 4096, so=AT + 4096):
    lh = np.asarray(lens, np.int32)
    KEEP.append(lh)
    return K.lib().kv_cache_reorder_paged(c or cache(K), layers, ls, lsv, B, Kb, parent, table, stride, lengths, lh.ctypes.data,
                                          spare, to, lo, so, None)


def test_reorder_refusals(K):
    page = 8 * 16 * 128
    assert reorder(K, B=0) == K.KVA_OK
    for kw, want in ((dict(B=-1), K.KVA_EINVAL), (dict(Kb=0), K.KVA_EINVAL), (dict(Kb=33), K.KVA_EINVAL), (dict(layers=0), K.KVA_EINVAL),
                     (dict(parent=None), K.KVA_EINVAL), (dict(spare=None), K.KVA_EINVAL), (dict(to=AT), K.KVA_EINVAL),
                     (dict(lo=AT), K.KVA_EINVAL), (dict(so=AT), K.KVA_EINVAL), (dict(stride=0), K.KVA_EINVAL),
                     (dict(layers=2, ls=page - 8, lsv=page), K.KVA_EINVAL), (dict(layers=2, ls=page + 4, lsv=page), K.KVA_EALIGN),
                     (dict(lens=(5, 65, 5, 5)), K.KVA_ECAPACITY), (dict(c=cache(K, page=24)), K.KVA_EUNSUPPORTED)):
        assert reorder(K, **kw) == want, kw
