"""Attention over pages where slots that only later tokens see hold NaN or infinities: a token's output depends on the slots that it
sees alone.  Tolerances are the ones derived in test_gpu_paged_cache.py."""
import numpy as np
import pytest

from helpers import dev, host
from oracle import paged_oracle as P
from test_gpu_paged_cache import HALF, K, Case, dtype, values  # noqa: F401

pytestmark = pytest.mark.gpu

FORMS = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]
BAD = [np.nan, np.inf, -np.inf]

SHAPES = [  # new tokens, lengths, page, Hq, Hkv, Dk, Dv
    ([4, 2, 1], [40, 2, 9], 16, 4, 2, 64, 64),                           # up to 8 rows a KV head
    ([7, 3, 8], [300, 3, 130], 32, 2, 1, 128, 128),                      # up to 16
    ([5, 16], [1000, 16], 16, 3, 3, 192, 128),
    ([40, 20], [700, 21], 64, 4, 2, 128, 128),                           # one row tile
    ([100], [3000], 16, 8, 2, 128, 128),                                 # four, units of several runs
    ([130, 65, 1], [130, 1400, 60], 128, 5, 1, 64, 64),
    ([300], [300], 256, 16, 8, 128, 128),                                # a prompt from its first token on
    ([200, 33], [260, 33], 32, 6, 2, 192, 128),
    ([90, 64], [50, 0], 16, 4, 2, 128, 128),                             # tokens that see nothing
]


def compare(K, c, q, out, want, size):  # noqa: F811
    import torch
    cache, batch = c.on_gpu(K)
    o = torch.empty((len(q), c.Hq, c.Dv), dtype=dtype(out), device="cuda")
    K.kv_attn_paged(dev(q, dtype(c.cache)), cache, batch, o, c.workspace(K))
    torch.cuda.synchronize()
    got = host(o)
    fine = np.isfinite(want)                                             # NaN or infinite: a weight's parts have either sign, and
    assert np.array_equal(np.isfinite(got), fine)                        # two of them times an infinity may give NaN
    weight = 0.0 if c.cache == "f32" else (2.0 ** -8 if out == "bf16" else 2.0 ** -16)
    tol = size * (weight + 1e-5) + np.abs(np.where(fine, want, 0)) * HALF[out] * (1 + weight)
    assert (np.abs(got[fine] - want[fine]) <= tol[fine]).all()


def plain(c, q):
    """The definition, and its sums of weight * |value| over the finite values."""
    pk, pv = c.pool_k.astype(np.float64), c.pool_v.astype(np.float64)
    with np.errstate(invalid="ignore"):
        want, _ = P.paged_attention(q, pk, pv, c.table, c.lengths, c.start)
    return want, P.paged_attention(q, pk, np.where(np.isfinite(pv), pv, 0.0), c.table, c.lengths, c.start)[1]


@pytest.mark.parametrize("cache,out", FORMS)
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_values_that_later_tokens_see(K, i, cache, out):  # noqa: F811
    """NaN and infinities of either sign in single values of V, in slots of new tokens: tokens before them keep their finite
    results, those from them on get none."""
    c = Case(K, 200 + i, *SHAPES[i], cache=cache).fill()
    q = values(c.r, (int(c.start[-1]), c.Hq, c.Dk), cache)
    for b, (n, L) in enumerate(zip(c.new, c.lengths)):
        for j in range(min(6, int(L))):
            slot = int(L) - 1 - int(c.r.integers(0, min(n, L)))
            if j == 0:
                slot = int(L) - 1                                        # the last token's own
            c.pool_v[c.table[b, slot // c.page], c.r.integers(0, c.Hkv), slot % c.page, c.r.integers(0, c.Dv)] = BAD[j % 3]
    want, size = plain(c, q)
    assert np.isfinite(want).mean() > 0.5
    compare(K, c, q, out, want, size)


@pytest.mark.parametrize("cache,out", FORMS)
def test_a_whole_row_and_keys(K, cache, out):  # noqa: F811
    """A token whose K and V rows are NaN throughout: the ones before it are as they were, it and the ones behind it are NaN."""
    for new, L, bad in ((5, 100, 96), (60, 500, 470), (200, 200, 128), (200, 1000, 999)):
        c = Case(K, 220, [new], [L], 16, 4, 2, 128, 128, cache=cache).fill()
        q = values(c.r, (new, 4, 128), cache)
        want, size = plain(c, q)
        c.pool_k[c.table[0, bad // 16], :, bad % 16] = np.nan
        c.pool_v[c.table[0, bad // 16], :, bad % 16] = np.nan
        want[bad - (L - new):] = np.nan
        compare(K, c, q, out, want, size)


@pytest.mark.parametrize("cache,out", FORMS)
def test_values_that_all_tokens_see(K, cache, out):  # noqa: F811
    """Slots before the new ones, and the first new one's own."""
    for new, L in ((3, 90), (40, 600)):
        c = Case(K, 221, [new], [L], 32, 4, 2, 128, 128, cache=cache).fill()
        q = values(c.r, (new, 4, 128), cache)
        for slot, d, x in ((5, 7, np.nan), (L - new - 1, 90, np.inf), (L - new, 64, -np.inf), (20, 3, np.inf), (21, 3, -np.inf)):
            c.pool_v[c.table[0, slot // 32], 1, slot % 32, d] = x
        want, size = plain(c, q)
        compare(K, c, q, out, want, size)
