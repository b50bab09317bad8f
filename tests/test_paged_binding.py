"""Pools that the Python binding refuses before it reads an address (CPU tensors)."""
import pytest


@pytest.fixture(scope="module")
def K():
    pytest.importorskip("torch")
    import kv_cache_gqa_gb300.kv_attn as K
    return K


def test_pages_that_overlap(K):
    """A pool made by expand() has pages 0 elements apart, which the C call reads as packed: 8 pages where memory holds one."""
    import torch
    one = torch.zeros((1, 2, 16, 64))
    good = torch.zeros((8, 2, 16, 64))
    closer = torch.zeros(8 * 2 * 16 * 64).as_strided((8, 2, 16, 64), (16 * 64, 16 * 64, 64, 1))
    for k, v in ((one.expand(8, 2, 16, 64), good), (good, one.expand(8, 2, 16, 64)), (closer, good),
                 (one.expand(8, 2, 16, 64).expand(3, 8, 2, 16, 64), good.expand(3, 8, 2, 16, 64))):
        with pytest.raises(K.KvaError, match="overlap"):
            K.PagedKVCache(k, v).struct


def test_layers_that_overlap(K):
    import torch
    good = torch.zeros((3, 8, 2, 16, 64))
    for k, v in ((good[:1].expand(3, 8, 2, 16, 64), good), (good, good[:1].expand(3, 8, 2, 16, 64))):
        with pytest.raises(K.KvaError, match="overlap"):
            K.PagedKVCache(k, v).struct
    for t in (good, good.transpose(0, 1).contiguous().transpose(0, 1)):      # layers apart, or alternating within a page
        with pytest.raises(K.KvaError, match="CUDA"):
            K.PagedKVCache(t, t).struct
