"""What the header promises of the 4-bit cache calls and lmhead_logprobs, where it shows without a GPU:
sizes, and the order in the kernels' sources."""
import glob
import os
import re

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kv_cache_gqa_gb300", "csrc")


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


def _block_end(src, at):
    """Past the } of the { at src[at]."""
    depth = 0
    for end in range(at, len(src)):
        depth += {"{": 1, "}": -1}.get(src[end], 0)
        if depth == 0:
            return end + 1
    raise AssertionError("unbalanced braces")


def _kernels():
    """(file, kernel, body) of every __global__ function that waits for the kernel before it."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        src = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__[^;{]*?(\w+)\(const[^{]*\{", src):
            body = src[m.end() - 1:_block_end(src, m.end() - 1)]
            if "griddep_wait()" in body:
                yield os.path.basename(path), m.group(1), body


def _without_lambdas(text):
    """A lambda runs where it is called, not where it stands."""
    while True:
        m = re.search(r"auto \w+ = \[&\]\([^)]*\)(?: -> \w+)? \{", text)
        if not m:
            return text
        text = text[:m.start()] + text[_block_end(text, m.end() - 1):]


READS = re.compile(r"\b[ap]\.\w+\s*\[|\b(?:__ldg|__ldcg|load1|load8|hidden_at|dot_again|tma_load_4d|bulk_g2s|load|issue)\s*[<(]")


def test_no_kernel_reads_global_memory_before_its_dependency_wait():
    """A kernel that starts while the one before it runs sees memory only after griddep_wait(): what earlier
    kernels wrote is visible to the grid that has waited, however long ago they ended.  (Prefetches into L2
    return no data.)"""
    names = []
    for path, kernel, body in _kernels():
        names.append(kernel)
        early = READS.search(_without_lambdas(body[:body.index("griddep_wait()")]))
        assert not early, f"{path}: {kernel} reads before the wait: {early.group(0)}"
    assert {"append_q4_kernel", "expand_q4_kernel", "decode_q4_kernel", "logprob_prep_kernel", "logprob_stream_kernel",
            "logprob_tc_kernel", "logprob_merge_kernel", "decode_mma_kernel", "verify_tc_kernel"} <= set(names)


def test_capacities_at_the_end_of_32_bits_are_refused(K):
    """A length just below 2^31 does not round up to whole stages in 32 bits."""
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("dummy addresses: runs on hosts without a GPU")
    L, at = K.lib(), 1 << 20
    lengths = np.array([5], np.int32)
    cache = K._CacheQ4(at, at, at, at, 1, 64, (1 << 31) - 4, 0, 0)
    assert L.kv_attn_decode_q4(at, 1, cache, at, lengths.ctypes.data, 1, 1, 1, 0.0, at, at, 1 << 30, None) == K.KVA_EUNSUPPORTED
    lengths[0] = cache.capacity
    assert L.kv_attn_decode_q4(at, 1, cache, at, lengths.ctypes.data, 1, 1, 1, 0.0, at, at, 1 << 30, None) == K.KVA_EUNSUPPORTED


def test_a_logprobs_workspace_serves_fewer_rows_and_alternatives(K):
    """A server sizes it for its largest batch and list; a smaller call splits the vocabulary more."""
    L = K.lib()
    size = L.kva_lmhead_logprobs_workspace_size
    for H, V in ((64, 333), (128, 9729), (72, 20000), (1024, 151936)):
        for k in (0, 5, 12, 20, 24):
            last = 0
            for B in list(range(1, 300)) + [1000, 1024, 1025, 1151, 1152, 1153, 4096]:
                now = size(B, H, V, k)
                assert now >= last, (B, H, V, k)
                last = now
        for B in (1, 4, 5, 128, 129, 2000):
            sizes = [size(B, H, V, k) for k in range(25)]
            assert sizes == sorted(sizes), (B, H, V)
