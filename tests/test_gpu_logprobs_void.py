"""Rows of lmhead_logprobs that have no softmax.  A kernel whose wait gives up leaves statistics of NaN beside the
other parts' valid lists; a NaN in one table row puts every row into the same state without a wait."""
import numpy as np
import pytest

from helpers import dev, host
from test_gpu_logprobs import inputs, run, seeded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from kv_cache_gqa_gb300 import build
    build.build_library(verbose=False)
    import kv_cache_gqa_gb300 as K
    return K


@pytest.mark.parametrize("what", [float("nan"), float("inf")])
@pytest.mark.parametrize("B,H,V,wdt,hdt,norm,k", [(1, 128, 9000, "bf16", "f32", True, 5), (64, 64, 3000, "bf16", "bf16", False, 20),
                                                  (150, 128, 700, "bf16", "f32", False, 1), (5, 72, 3000, "bf16", "f32", True, 3),
                                                  (2, 136, 333, "f32", "f32", False, 24)])
def test_no_id_where_a_logit_is_nan(K, B, H, V, wdt, hdt, norm, k, what):
    rng = seeded("void", B, H, V, wdt, hdt, norm, k)
    hd, Wd, _, nw, targets = inputs(rng, B, H, V, wdt, hdt, norm)
    hd.abs_().add_(0.5)                                        # every product with the bad row is NaN or +infinity
    nw = np.abs(nw) if norm else None
    Wd[V // 3] = what
    targets[targets == V // 3] = 0
    if B > 1:
        targets[1] = -1
    lp, ent, lse, ids, top = run(K, hd, Wd, V, k, dev(nw) if norm else None, dev(targets))
    assert np.all(ids == -1) and np.all(np.isnan(top)) and np.all(np.isnan(ent))
    assert np.all(np.isnan(lp[targets >= 0])) and np.all(lp[targets < 0] == 0)
    assert np.all(np.isnan(lse))


def test_one_row_without_a_softmax_leaves_the_others(K):
    rng = seeded("one-void")
    B, H, V, k = 9, 128, 2000, 4
    hd, Wd, _, _, _ = inputs(rng, B, H, V, "bf16", "f32", False)
    clean = run(K, hd, Wd, V, k)
    hd[3, 17] = float("nan")
    got = run(K, hd, Wd, V, k)
    rest = np.arange(B) != 3
    for a, b in zip(got[1:], clean[1:]):
        assert np.array_equal(a[rest], b[rest])
    assert np.all(got[3][3] == -1) and np.all(np.isnan(got[4][3])) and np.isnan(got[1][3]) and np.isnan(got[2][3])
