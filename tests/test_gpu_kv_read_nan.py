"""bsp_kv_page_read of the e8m0 bytes at the ends: 255 is NaN, as the dense
attention takes it; 0 is 2^-127, whose multiples bf16 holds as subnormals."""
import numpy as np
import pytest
import torch

from plain64 import MX, bf16_to_f64, mx_row

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("index", [False, True])
def test_scale_bytes_at_the_ends(index):
    from block_sparse_paged_score_gb300 import bsp
    r = np.random.default_rng(8)
    raw = r.integers(0, 256, 4 * 8704, dtype=np.uint8).reshape(4, 8704)
    raw[:, 8192:] = r.choice(np.array([0, 1, 2, 100, 252, 255], np.uint8), (4, 512))
    buf = torch.from_numpy(raw.reshape(-1).copy()).cuda()
    slot = torch.arange(256, device="cuda")
    if index:
        got = [bsp.kv_page_read(None, bsp.IndexCache(MX, 2, 2, buffer=buf), slot)[2][:, h] for h in range(2)]
        fields = [(0, 2), (1, 3)]
    else:
        got = [x[:, 0] for x in bsp.kv_page_read(bsp.KvCache(MX, 1, 2, buffer=buf), None, slot)[:2]]
        fields = [(0, 2), (1, 3)]
    for g, (a, b) in zip(got, fields):
        v = bf16_to_f64(g.contiguous().view(torch.int16).cpu().numpy().view(np.uint16))
        for t in range(256):
            f = raw[a if t < 128 else b]
            want = mx_row(f, t % 128)
            nan = np.repeat(f[8192 + 4 * (t % 128):8196 + 4 * (t % 128)] == 255, 32)
            assert np.array_equal(np.isnan(v[t]), nan) and np.array_equal(v[t][~nan], want[~nan]), t
