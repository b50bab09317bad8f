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

