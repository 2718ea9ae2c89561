"""bsp_kv_scaled_write on both sides of its choice between a token and 32 tokens a CTA: single tokens of many
requests, whose blocks' scales grow for some and not for others."""
import numpy as np
import pytest
import torch

from test_gpu_kv_scaled import check, make, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads", [1, 2, 4])
@pytest.mark.parametrize("more", [0, 1])
def test_decode_tokens(heads, more):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    T = 4 * sms // (2 * heads) + more
    rng = np.random.default_rng(heads + more)
    cache, scales = make(rng, heads, T + 1)
    for s in scales:
        s[::3] = 2.0 ** -20
    slot = rng.permutation(T) * 128 + rng.integers(0, 128, T)
    check(cache, scales, heads, T + 1, rows(rng, T, heads), rows(rng, T, heads), slot.astype(np.int64), 0)
