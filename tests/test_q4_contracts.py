"""What the header promises of the 4-bit cache calls and lmhead_logprobs, where it shows without a GPU:
sizes, and the order in the kernels' sources."""
import pytest


@pytest.fixture(scope="module")
def K():
    from kv_cache_gqa_gb300 import build
    build.build_library(verbose=False)
    import kv_cache_gqa_gb300.kv_attn as K
    K.lib()
    return K


def test_decode_q4_counters_lie_in_the_same_bytes_whatever_the_shape(K):
    """Else a call writes partial results where a wider one counts, on a workspace that both use."""
    L = K.lib()
    shapes = [(B, Hkv, Hkv * G, T) for B in (1, 8, 64, 4096) for Hkv in (1, 8, 32) for G in (1, 2, 16) for T in (1, 5, 16, 64)]
    zero = {L.kva_decode_q4_workspace_zero_bytes(*s) for s in shapes}
    assert len(zero) == 1 and zero.pop() > 0
    for B, Hkv, Hq, T in shapes:                               # the widest block's workspace serves the narrower ones
        need = L.kva_decode_q4_workspace_size(B, Hkv, Hq, T, 1000, 128)
        assert need <= L.kva_decode_q4_workspace_size(4096, 32, 512, 64, 1000, 128)
