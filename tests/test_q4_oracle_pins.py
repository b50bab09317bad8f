"""Hand-worked pins of the 4-bit cache and vocabulary-scoring oracle (CPU)."""
import math

import numpy as np
import pytest

from oracle import kv_oracle as O
from oracle import q4_oracle as Q


def test_quantiser_by_hand():
    x = np.zeros(64)
    x[:16] = np.arange(16)                         # 0..15: scale 1, mid 8, every value exact
    u, scale, mid = Q.q4_quantise(x)
    assert scale[0] == 1.0 and mid[0] == 8.0
    assert list(u[0, :16]) == list(range(16)) and u[0, 20] == 0
    assert np.array_equal(Q.q4_values(u, scale, mid), x)
    x = np.zeros(64)
    x[0], x[1], x[2], x[3] = -7.5, 7.5, 0.5, 1.5   # spread 15: scale 1, mid 0.5: quotients -8, 7, 0, 1
    u, scale, mid = Q.q4_quantise(x)
    assert (scale[0], mid[0]) == (1.0, 0.5)
    assert list(u[0, :4]) == [0, 15, 8, 9]
    assert u[0, 4] == 8                            # -0.5 rounds half to even: 0
    x = np.full(64, 0.1)                           # equal values: scale 0, their bf16 rounding
    u, scale, mid = Q.q4_quantise(x)
    assert scale[0] == 0 and np.all(Q.q4_values(u, scale, mid) == O.bf16_round(np.array(0.1)))
    x = np.zeros(128)
    x[70] = np.nan                                 # the second group only
    v = Q.q4_values(*Q.q4_quantise(x))
    assert np.all(v[:64] == 0) and np.all(np.isnan(v[64:]))


def test_quantiser_error_bound_and_scale_rounding():
    x = np.random.default_rng(0).standard_normal((500, 128)) * np.exp(np.random.default_rng(1).normal(size=(500, 1)))
    u, scale, mid = Q.q4_quantise(x)
    v = Q.q4_values(u, scale, mid).reshape(500, 2, 64)
    g = x.reshape(500, 2, 64)
    assert np.all(np.abs(v - g) <= (scale / 2 + np.abs(mid) * 2.0 ** -9)[..., None] * (1 + 1e-12))
    spread = g.max(-1) - g.min(-1)
    assert np.all(15 * scale >= spread * (1 - 1e-15)) and np.all(15 * scale <= spread * (1 + 2.0 ** -7))


@pytest.mark.parametrize("G", [1, 2, 3, 4])
def test_pack_layout(G):
    u = np.zeros((G, 64), np.int64)
    u[G - 1, 8 * 5 + 2] = 9                        # dim 64 (G-1) + 42: word 5 G + G - 1, nibble 2
    b = Q.q4_pack(u)
    assert b.shape == (32 * G,)
    word = 5 * G + G - 1
    assert b[4 * word + 1] == 9 and b.astype(int).sum() == 9
    r = np.random.default_rng(G).integers(0, 16, (3, G, 64))
    assert np.array_equal(Q.q4_unpack(Q.q4_pack(r)), r)


def test_attend_block_is_causal_and_empty_rows_are_zero():
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((3, 2, 8)), rng.standard_normal((1, 9, 8)), rng.standard_normal((1, 9, 8))
    o = Q.attend_block(q, k, v, 2)                 # three tokens, two slots: the first sees nothing
    assert np.all(o[0] == 0)
    assert np.allclose(o[1], v[0, :1])             # one slot: its value
    assert np.allclose(Q.attend_block(q, k, v, 7)[2], O.decode(q[2], k, v, 7))


def test_logprobs_by_hand():
    W = np.array([[1.0, 0.0], [0.0, 1.0], [1.0, 0.0]])
    h = np.array([[math.log(2.0), 0.0]])           # logits ln2, 0, ln2: probabilities 2/5, 1/5, 2/5
    lp, ent, lse, ids, top = Q.logprobs(h, W, 3, targets=[1], top_k=2)
    assert lp[0] == pytest.approx(math.log(0.2)) and lse[0] == pytest.approx(math.log(5.0))
    assert ent[0] == pytest.approx(-(0.8 * math.log(0.4) + 0.2 * math.log(0.2)))
    assert list(ids[0]) == [0, 2] and top[0, 1] == pytest.approx(math.log(0.4))
    lp, *_ = Q.logprobs(np.repeat(h, 3, 0), W, 2, targets=[-1, 2, 0])
    assert lp[0] == 0 and np.isnan(lp[1]) and lp[2] == pytest.approx(math.log(2 / 3))
