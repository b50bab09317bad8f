"""Host-side refusals of the 4-bit cache calls and lmhead_logprobs: the documented status before
anything is launched (dummy addresses; runs on hosts without a GPU)."""
import numpy as np
import pytest

FAKE = 1 << 20


@pytest.fixture(scope="module")
def K():
    try:
        import torch
        if torch.cuda.is_available():
            pytest.skip("ABI validation tests run on hosts without a GPU")
    except ImportError:
        pass
    from kv_cache_gqa_gb300 import build
    build.build_library(verbose=False)
    import kv_cache_gqa_gb300.kv_attn as K
    K.lib()
    return K


def q4(K, ptr=FAKE, hkv=8, d=128, cap=64, dv=0, rows=0, scale=FAKE):
    return K._CacheQ4(ptr, FAKE, scale, FAKE, hkv, d, cap, dv, rows)


def norm(K, q=None, k=None, stride=0, eps=1e-6):
    return K._Norm(q, k, stride, eps, 0)


def rope(K, kind=0, rot_offset=0, rot_dim=0):
    import ctypes as C
    return K._Rope(kind, 1 if kind else 0, (C.c_int32 * 4)(), 1e6, rot_offset, rot_dim)


def test_append(K):
    L = K.lib()

    def call(slots=(0, 1), N=1, cache=None, q=FAKE, q_out=FAKE, k=FAKE, Hq=16, rp=None, pos=FAKE, nm=None, dt=0, stride=0):
        sh = np.asarray(slots, np.int32)
        T = sh.shape[-1]
        return L.kv_cache_append_q4(q, k, FAKE, dt, N, T, Hq, pos, 0, FAKE, stride, sh.ctypes.data,
                                    nm or norm(K), rp or rope(K), q_out, 0, cache or q4(K), None)
    assert call(slots=()) == K.KVA_OK and call(N=0) == K.KVA_OK
    assert call(N=-1) == K.KVA_EINVAL
    assert call(slots=(0, 64)) == K.KVA_ECAPACITY and call(slots=(-1,)) == K.KVA_ECAPACITY
    assert call(slots=(3, 5, 3)) == K.KVA_EINVAL               # written twice
    assert call(slots=(5, 5)) == K.KVA_EINVAL
    assert call(slots=((0, 1), (2, 2)), N=2, stride=2) == K.KVA_EINVAL
    assert call(q=None) == K.KVA_EINVAL and call(q_out=None) == K.KVA_EINVAL
    assert call(k=None) == K.KVA_EINVAL and call(Hq=12) == K.KVA_EINVAL and call(dt=2) == K.KVA_EINVAL
    assert call(k=FAKE + 8) == K.KVA_EALIGN
    assert call(rp=rope(K, 1), pos=None) == K.KVA_EINVAL
    assert call(rp=rope(K, 1, 100, 64)) == K.KVA_EINVAL        # rotary range outside the head
    assert call(nm=norm(K, q=FAKE)) == K.KVA_EINVAL and call(nm=norm(K, FAKE, FAKE, 3)) == K.KVA_EALIGN
    for bad, status in ((q4(K, d=72), K.KVA_EALIGN), (q4(K, d=320), K.KVA_EUNSUPPORTED), (q4(K, cap=62), K.KVA_EALIGN),
                        (q4(K, ptr=0), K.KVA_EINVAL), (q4(K, scale=FAKE + 4), K.KVA_EALIGN), (q4(K, hkv=0), K.KVA_EINVAL),
                        (q4(K, rows=-4), K.KVA_EINVAL), (q4(K, dv=100), K.KVA_EALIGN), (q4(K, rows=8 * 64 + 2), K.KVA_EALIGN)):
        assert call(cache=bad) == status, L.kva_last_error()
    assert call(cache=q4(K, rows=8 * 64 - 4), N=2, slots=((0,), (0,)), stride=1) == K.KVA_EINVAL


def test_expand(K):
    L = K.lib()

    def call(slots=(0, 1), N=1, cache=None, first=0, d=128, dv=0, hkv=8, cap=8, dtype=1, slot=FAKE):
        sh = np.asarray(slots, np.int32)
        dst = K._Cache(FAKE, FAKE, dtype, hkv, d, cap, hkv * cap * d, dv, hkv * cap * dv)
        return L.kv_cache_expand_q4(cache or q4(K), slot, 0, sh.ctypes.data, N, len(slots), dst, first, None)
    assert call(N=0) == K.KVA_OK and call(slots=()) == K.KVA_OK
    assert call(slots=(64,)) == K.KVA_ECAPACITY and call(first=7) == K.KVA_ECAPACITY and call(first=-1) == K.KVA_ECAPACITY
    assert call(d=64) == K.KVA_EINVAL and call(hkv=4) == K.KVA_EINVAL and call(dv=64) == K.KVA_EINVAL
    assert call(slot=None) == K.KVA_EINVAL and call(dtype=3) == K.KVA_EINVAL and call(N=-1) == K.KVA_EINVAL


def test_decode(K):
    L = K.lib()

    def call(lens=(3,), T=1, cache=None, Hq=16, ws=FAKE, n=1 << 30, q=FAKE, out=FAKE, dt=1, B=None):
        lh = np.asarray(lens, np.int32)
        return L.kv_attn_decode_q4(q, dt, cache or q4(K), FAKE, lh.ctypes.data, len(lens) if B is None else B, T, Hq, 0.0, out,
                                   ws, n, None)
    assert call(lens=()) == K.KVA_OK
    assert call(B=-1) == K.KVA_EINVAL
    assert call(lens=(65,)) == K.KVA_ECAPACITY and call(lens=(-1,)) == K.KVA_ECAPACITY
    assert call(T=0) == K.KVA_EINVAL and call(T=65) == K.KVA_EINVAL
    assert call(Hq=12) == K.KVA_EINVAL and call(q=None) == K.KVA_EINVAL and call(dt=7) == K.KVA_EINVAL
    assert call(cache=q4(K, d=256)) == K.KVA_EUNSUPPORTED and call(cache=q4(K, d=128, dv=192)) == K.KVA_EUNSUPPORTED
    assert call(ws=None) == K.KVA_EWORKSPACE and call(n=16) == K.KVA_EWORKSPACE and call(ws=FAKE + 8) == K.KVA_EALIGN
    assert call(out=FAKE + 4) == K.KVA_EALIGN
    for B, Hkv, Hq, T, n, dv in ((1, 8, 16, 1, 768, 128), (64, 8, 16, 16, 32768, 128), (3, 2, 18, 5, 100000, 64)):
        size = L.kva_decode_q4_workspace_size(B, Hkv, Hq, T, n, dv)
        assert size > L.kva_decode_q4_workspace_zero_bytes(B, Hkv, Hq, T) > 0
        assert K.workspace_bytes("decode_q4", B=B, n_kv_heads=Hkv, n_q_heads=Hq, max_len=n, head_dim=dv, block=T) == size
        assert size >= L.kva_decode_q4_workspace_size(B, Hkv, Hq, T, n // 2, dv)   # any shorter plan fits
    assert L.kva_decode_q4_workspace_size(1, 8, 12, 1, 64, 128) == 0 and L.kva_decode_q4_workspace_zero_bytes(0, 8, 16, 1) == 0


def test_logprobs(K):
    L = K.lib()

    def call(B=1, H=1024, V=100, rows=100, k=4, ids=FAKE, ws=FAKE, n=1 << 30, t=FAKE, lp=FAKE, ent=FAKE, h=FAKE, nw=None, eps=1e-6,
             hd=0, wd=1):
        return L.lmhead_logprobs(h, hd, nw, eps, FAKE, wd, B, H, V, rows, t, lp, ent, None, k, ids, None, ws, n, None)
    assert call(B=0) == K.KVA_OK and call(B=-1) == K.KVA_EINVAL
    assert call(k=-1) == K.KVA_EINVAL and call(k=25) == K.KVA_EINVAL and call(k=4, V=3, rows=3) == K.KVA_EINVAL
    assert call(V=101) == K.KVA_EINVAL and call(ids=None) == K.KVA_EINVAL and call(t=None) == K.KVA_EINVAL
    assert call(lp=None) == K.KVA_EINVAL and call(t=None, lp=None, ent=None, k=0, ids=None) == K.KVA_EINVAL
    assert call(nw=FAKE, eps=-1.0) == K.KVA_EINVAL and call(nw=FAKE + 4) == K.KVA_EALIGN
    assert call(H=1020) == K.KVA_EALIGN and call(h=FAKE + 8) == K.KVA_EALIGN and call(H=8192) == K.KVA_EUNSUPPORTED
    assert call(hd=2) == K.KVA_EINVAL and call(wd=-1) == K.KVA_EINVAL and call(B=70000) == K.KVA_EUNSUPPORTED
    assert call(ws=None) == K.KVA_EWORKSPACE and call(n=16) == K.KVA_EWORKSPACE and call(ws=FAKE + 1) == K.KVA_EALIGN
    size = L.kva_lmhead_logprobs_workspace_size(64, 1024, 151936, 8)
    assert size == K.workspace_bytes("lmhead_logprobs", B=64, hidden=1024, vocab=151936, block=8) > 0
    assert K.workspace_bytes("lmhead_logprobs", B=1, hidden=64, vocab=9, block=0) > 0
    assert L.kva_lmhead_logprobs_workspace_size(64, 1024, 151936, 25) == 0


def test_binding_checks(K):
    torch = pytest.importorskip("torch")
    with pytest.raises(K.KvaError):
        K.KVCacheQ4(torch.zeros((1, 1, 4, 32), dtype=torch.uint8), torch.zeros((1, 1, 4, 32), dtype=torch.uint8),
                    torch.zeros((1, 1, 4, 1, 2)), torch.zeros((1, 1, 4, 1, 2), dtype=torch.bfloat16)).struct
    with pytest.raises(K.KvaError):
        K._want(torch.zeros(3), "x", (3,), (torch.float32,))
