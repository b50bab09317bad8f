"""What the Python calls of the 4-bit cache refuse before a launch: index tensors that the kernels would read wrongly."""
import numpy as np
import pytest

from helpers import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from kv_cache_gqa_gb300 import build
    build.build_library(verbose=False)
    import kv_cache_gqa_gb300 as K
    return K


def _case(K, N, T):
    import torch
    cache = K.KVCacheQ4.zeros(N, 2, 16, 64)
    x = torch.randn((N, T, 2, 64), device="cuda")
    slot = np.tile(np.arange(T, dtype=np.int32), (N, 1))
    return cache, x, slot


def test_slots_of_another_type_with_a_stride_given(K):
    """A stride given by the caller does not make int64, strided or host slots readable."""
    import torch
    cache, x, slot = _case(K, 2, 3)
    dst = K.KVCache(*(torch.zeros((2, 2, 16, 64), device="cuda") for _ in range(2)))
    good = dev(slot)
    for bad in (good.long(), dev(np.repeat(slot, 2, 1))[:, ::2], torch.from_numpy(slot)):
        with pytest.raises(K.KvaError):
            K.kv_cache_append_q4(None, x, x, None, bad, slot, cache, None, K.Rope("none"), slot_inst_stride=3)
        with pytest.raises(K.KvaError):
            K.kv_cache_expand_q4(cache, bad, slot, dst, slot_inst_stride=3)
    K.kv_cache_append_q4(None, x, x, None, good, slot, cache, None, K.Rope("none"), slot_inst_stride=3)
    K.kv_cache_expand_q4(cache, good, slot, dst, slot_inst_stride=3)
    torch.cuda.synchronize()
    assert not bool((dst.k[1, :, :3] == 0).all())


def test_positions_of_one_token_each_without_their_token_axis(K):
    """[N, n_axes] is how kv_attn_decode_step takes them; the append takes [N, T, n_axes], and [T, n_axes] shared by all."""
    import torch
    cache, x, slot = _case(K, 3, 1)
    pos = dev(np.array([[5], [6], [7]], np.int32))
    with pytest.raises(K.KvaError):
        K.kv_cache_append_q4(None, x, x, pos, dev(slot), slot, cache, None, K.Rope("1d"))
    out = []
    for p in (pos[:, None], pos[1:2], pos[1:2, None]):
        K.kv_cache_append_q4(None, x, x, p, dev(slot), slot, cache, None, K.Rope("1d"))
        dst = K.KVCache(*(torch.zeros((3, 2, 1, 64), device="cuda") for _ in range(2)))
        K.kv_cache_expand_q4(cache, dev(slot), slot, dst)
        torch.cuda.synchronize()
        out.append(dst.k)
    assert torch.equal(out[1], out[2]) and torch.equal(out[0][1], out[1][1]) and not torch.equal(out[0][0], out[1][0])
