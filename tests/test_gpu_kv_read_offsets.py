"""Reads of consecutive fp8 slots from every offset in a page, over block borders, from the definition:
sixteen tokens in a row of a block take a way of their own (8-byte pieces of V's dims, put together at the offset).

e4m3 * scale is one fp32 product, exact for a power of two, and one bf16 rounding, exact then too; else off by at
most 2^-8 + 2^-24 of the value."""
import numpy as np
import pytest
import torch

import plain64_scaled as P
from test_gpu_kv_scaled import device_cache, make

pytestmark = pytest.mark.gpu


def agrees(got, want, pow2):
    tol = 0 if pow2 else (2.0 ** -8 + 2.0 ** -24) * np.abs(want)
    ok = (np.abs(got - want) <= tol) | (np.isnan(want) & np.isnan(got))
    assert ok.all(), np.argwhere(~ok)[:4]


@pytest.mark.parametrize("pow2", [True, False])
@pytest.mark.parametrize("hkv", [1, 3])
@pytest.mark.parametrize("start", list(range(16)) + [117, 127])
def test_block_scaled(start, hkv, pow2):
    from block_sparse_paged_score_gb300 import bsp
    rng = np.random.default_rng(start)
    order = np.array([3, 0, 4, 1])
    cache, scales = make(rng, hkv, 5, pow2)
    cache[1::53] = 0x7F
    t = start + np.arange(128 * 2 + 41)
    slot = (order[t // 128] * 128 + t % 128).astype(np.int64)
    got = bsp.kv_scaled_read(device_cache(cache, scales, hkv, 5), torch.from_numpy(slot).cuda())
    for side in (0, 1):
        for h in range(hkv):
            values = np.stack([P.block_values(cache, scales, hkv, b, h, side) for b in range(5)])
            agrees(P.bits_f64(got[side])[:, h], values[slot // 128, slot % 128], pow2)


@pytest.mark.parametrize("start", range(16))
def test_per_tensor_scales(start):
    from block_sparse_paged_score_gb300 import bsp
    rng = np.random.default_rng(100 + start)
    cache, _ = make(rng, 2, 3)
    kv = bsp.KvCache(bsp.FP8_E4M3, 2, 3, 0.25, 2.0, buffer=torch.from_numpy(cache.copy()).cuda())
    slot = start + 128 + np.arange(200, dtype=np.int64)
    got = bsp.kv_page_read(kv, None, torch.from_numpy(slot).cuda())
    scales = [np.full((3, 2), x, np.float32) for x in (0.25, 2.0)]
    for side in (0, 1):
        for h in range(2):
            values = np.stack([P.block_values(cache, scales, 2, b, h, side) for b in range(3)])
            agrees(P.bits_f64(got[side])[:, h], values[slot // 128, slot % 128], True)
