"""Beam selection over logits and scores of any finite size: masked tokens whose logit is a large negative number, large positive
ones, rows far from zero.  Tolerances are the ones derived in test_gpu_beams.py: half a step of the float32 total and 1e-6 of the sum's
logarithm."""
import numpy as np
import pytest

import workloads as WL
from oracle import paged_oracle as P
from test_gpu_beams import K, check, select  # noqa: F401

pytestmark = pytest.mark.gpu

FILLS = [5e9, 1e10, 1e12, 1e15, 1e20, 9e29, 1e38]


def given(z, dt):
    """The logits on the GPU and as the type holds them."""
    import torch
    z = z.astype(np.float32)
    if dt == "bf16":
        z = WL.bf16_bits_to_f32(WL.f32_to_bf16_bits(z))
    return torch.from_numpy(z).cuda().to({"f32": torch.float32, "bf16": torch.bfloat16}[dt]), z


def run(K, z, scores, n, dt):  # noqa: F811
    t, held = given(z, dt)
    got = select(K, t, scores, n)
    assert (got[0] >= 0).all()                                           # there are always n offers here
    want = P.beam_step(held, scores, n)
    if held.shape[1] == 1:
        # totals of one beam differ by what its logits differ by, so theirs is the order: -1e20 + 3 and -1e20 are one number in 64 bits
        for b, row in enumerate(held[:, 0]):
            best = np.lexsort((np.arange(row.size), -row.astype(np.float64)))[:n]
            want[b] = [(0, int(t), w[2]) for t, w in zip(best, want[b])]
            assert (got[1][b] == best).all()
    check(got, want)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("fill", FILLS)
def test_masked_tokens(K, fill, dt):  # noqa: F811
    """Masked values that fill some threads' batches (16 or 32 values), a whole slice, the row's first or last values, all of the
    row, or every second value."""
    V = 40001
    r = np.random.default_rng(31)
    z = 3 * r.standard_normal((2, 5, V)).astype(np.float32)
    z[0, 0, :64] = -fill
    z[0, 1, 8192:24576] = -fill
    z[0, 2, 20:] = -fill
    z[0, 3, :-5] = -fill
    z[0, 4, ::2] = -fill
    z[1] = -fill                                                         # a beam's total is then its score - log V
    z[1, 1, 30000] = 0.0
    scores = -r.random((2, 5)).astype(np.float32)
    run(K, z, scores, 7, dt)
    run(K, z[:, 2:3], scores[:, 2:3], 32, dt)                            # more offers than values that are not masked


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("fill", FILLS)
def test_large_values(K, fill, dt):  # noqa: F811
    """Some values tower over the row, first, last or in the middle; rows of large values of either sign."""
    V = 30011
    r = np.random.default_rng(32)
    z = r.standard_normal((1, 5, V)).astype(np.float32)
    z[0, 0, :3] = fill
    z[0, 1, -1:] = fill
    z[0, 2, 10000:10100] = fill
    z[0, 3] *= fill / 8
    z[0, 4] = fill
    scores = -r.random((1, 5)).astype(np.float32)
    run(K, z, scores, 9, dt)
    for k in range(5):
        run(K, z[:, k:k + 1], scores[:, k:k + 1], 9, dt)


@pytest.mark.parametrize("at", [1e3, -1e3, 1e5, -1e6, 1e7, -1e7, 1e8, -1e9, 1.0737e9, -1.0738e9, 4e9])
def test_rows_far_from_zero(K, at):  # noqa: F811
    """A few steps of the type around one value: steps of 2^-14 to 2^9, which all count, or of which only the largest does."""
    V = 20000
    r = np.random.default_rng(33)
    step = float(np.spacing(np.float32(abs(at))))
    z = (at + step * r.integers(-6, 7, (1, 3, V))).astype(np.float32)
    z[0, 2, : V // 2] -= np.float32(abs(at))                            # half of the row as far again
    run(K, z, -r.random((1, 3)).astype(np.float32), 32, "f32")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_scores_that_are_no_numbers(K, dt):  # noqa: F811
    """+infinity, -infinity and NaN: such a beam offers nothing, finished or not; scores of the type's largest size are ordinary."""
    r = np.random.default_rng(34)
    t, z = given(r.standard_normal((3, 5, 700)), dt)
    scores = -r.random((3, 5)).astype(np.float32)
    scores[0, :3] = np.inf, -np.inf, np.nan
    scores[1] = np.inf, np.inf, -np.inf, np.nan, np.inf
    scores[2] = 3e38, -3e38, np.inf, 1e30, -1e30
    for finished in (None, np.tile([True, True, True, False, False], (3, 1)), np.tile([False, False, False, True, True], (3, 1))):
        beam, token, score = got = select(K, t, scores, 4, finished, 6)
        want = P.beam_step(z, scores, 4, finished, 6)
        check([x[:2] for x in got], want[:2])
        assert (beam[1] == -1).all() and (token[1] == -1).all() and (score[1] == -np.inf).all()
        first = [b for b, _, _ in want[2]]
        assert beam[2].tolist() == first and np.allclose(score[2], [u for _, _, u in want[2]], rtol=2.0 ** -23)
