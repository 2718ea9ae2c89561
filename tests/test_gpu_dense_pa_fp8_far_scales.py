"""bsp_dense_pa_decode_fp8 where the V scales that a row sees lie farther apart than
fp32's exponents: every token keeps its share of the softmax's sum, whatever its block's
scale.  (kv_scaled_write makes scales from 2^-60, of a block of zeros, to 2^119.)

Tolerances are those of test_gpu_dense_pa_fp8 but for one term: a token's weight counts its
block's scale, so of scales up to 2^128 its logit is rounded once more at |t| < 2^8, off by
2^-16 at most, which is 2^-17 and less of a weight and lies within the 2^-10 there.  What f16
weights lose of a block 2^32 below the largest is below 2^-32 of a, as V's bytes here are
at least 2^-9 and at most 448 of a scale and every dim has some of the largest scale."""
import numpy as np
import pytest

import plain64_scaled as P
from test_gpu_dense_pa_fp8 import attend, close, expected, problem

pytestmark = pytest.mark.gpu


def with_scales(p, exponents, flat):
    """V scales 2^exponents[i] of a sequence's i-th block; flat: logits of 0."""
    for s in range(p["table"].shape[0]):
        for i, e in enumerate(exponents):
            p["scales"][1][p["table"][s, i]] = 2.0 ** e
    if flat:
        p["scales"][0][:] = 0
    return p


@pytest.mark.parametrize("flat", [True, False])
@pytest.mark.parametrize("q_len,group,q8", [(1, 16, False), (1, 4, True), (2, 16, True), (4, 16, False)])
@pytest.mark.parametrize("low,high", [(-60, 70), (-60, 81), (-60, 119), (-3, 119)])
def test_small_scale_first_and_last(low, high, q_len, group, q8, flat):
    for exponents in ((low, high), (high, low), (low, high, low), (high, low, low, high), (low, 0, high, 0, low)):
        p = problem(30 + len(exponents), 2, q_len, 1, group, (128 * len(exponents), 128 * len(exponents) - 5), q8)
        p = with_scales(p, exponents, flat)
        close(attend(p), *expected(p))


@pytest.mark.parametrize("low,high", [(-60, 70), (-60, 119)])
@pytest.mark.parametrize("q_len,group,hkv", [(1, 16, 1), (4, 16, 1), (1, 4, 2)])
def test_pieces_of_a_unit_far_apart(low, high, q_len, group, hkv):
    """One long sequence that many CTAs share: whole pieces of the small scale, of the large one, and of both."""
    n = 200
    for turn in range(2):
        exponents = [(low, high)[(i * 2 // n) ^ turn] if i % 7 else high for i in range(n)]
        if turn:
            exponents = [low] * 150 + [high] * 50
        p = with_scales(problem(40 + turn, 1, q_len, hkv, group, (128 * n - 3,), False), exponents, True)
        close(attend(p), *expected(p))


def test_a_block_of_zeros_before_large_values():
    """The writer gives zeros the scale 2^-60: half of the tokens are zeros, so the mean halves the rest."""
    p = with_scales(problem(50, 1, 1, 1, 4, (256,), False), (-60, 70), True)
    at = P.block_addresses(1, p["table"][0, 0], 0, 1)
    p["cache"][at] = 0
    o, a = expected(p)
    got = P.bits_f64(attend(p))
    want = P.block_values(p["cache"], p["scales"], 1, p["table"][0, 1], 0, 1).sum(0) / 256
    assert np.allclose(o[0, 0], want, rtol=1e-12)
    assert (np.abs(got - o) <= (2.0 ** -11 + 2.0 ** -10) * a + 2.0 ** -8 * np.abs(o)).all()


def test_blocks_left_out_and_nan_scales_beside_far_ones():
    """A bad block among blocks far apart adds nothing; a row that does not see a block with the scale NaN
    is as without it."""
    import torch
    p = with_scales(problem(51, 2, 1, 1, 4, (512, 300), False, nb=4), (119, -60, 0, -60), True)
    p["table"][0, 1] = -1
    p["scales"][1][p["table"][1, 3]] = np.nan
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = attend(p, err=err)
    assert err.item() == 2
    r = {**p, "table": np.array([p["table"][0, [0, 2, 3, 3]], p["table"][1]], np.int32),
         "row_len": np.array([384, 300], np.int32)}
    close(got, *expected(r))
