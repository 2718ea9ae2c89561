"""Repeated slots of bsp_kv_scaled_write: rows that a later one of the run replaces count for nothing, neither
for the bytes nor for the block's scale."""
import numpy as np
import pytest
import torch

from test_gpu_kv_scaled import check, make, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("before", [0, 20])
@pytest.mark.parametrize("runs", [1, 3])
@pytest.mark.parametrize("first", [0, 9])
def test_a_replaced_row_does_not_raise_the_scale(first, runs, before):
    """Runs of a few tokens (one, or several that lie close together) and of many: the replaced rows hold the
    largest values, an infinity among them, and are replaced by rows far below 1."""
    rng = np.random.default_rng(first + before)
    cache, scales = make(rng, 2, 4)
    for s in scales:
        s[:] = 2.0 ** -9
    slot, size = [], []
    for r in range(runs):
        own = list(range(first, first + before + 3))
        slot += [r * 128 + o for o in own + [first, first + 1]]
        size += [100.0, 300.0] + [2.0 ** -6] * (len(own) - 2) + [2.0 ** -6, 2.0 ** -7]
    k, v = (rows(rng, len(slot), 2, 0).clamp(-4, 4) * torch.tensor(size).bfloat16()[:, None, None] for _ in range(2))
    k[1, 0, 5] = float("inf")
    dev = check(cache, scales, 2, 4, k, v, np.array(slot, np.int64), 0)
    # 4 * 2^-6 = 448 * 2^-12.8 at most, where the replaced rows alone would ask for 2^-2 and more
    assert (dev.k_scales[:runs] <= 2.0 ** -9).all() and (dev.v_scales[:runs] <= 2.0 ** -9).all()
