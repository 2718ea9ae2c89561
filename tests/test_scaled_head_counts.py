"""The head counts that the block-scaled cache's calls take (no GPU needed: the addresses are never dereferenced;
with a GPU the tests are left out, as a case that should have been refused would launch)."""
import ctypes as C

import pytest
import torch

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="fake device addresses must never reach a GPU")
UNSUPPORTED, LAUNCHED = 2, 4  # a launch fails without a device


@pytest.mark.parametrize("heads,write,read", [(65535, LAUNCHED, LAUNCHED), (65536, UNSUPPORTED, LAUNCHED),
                                              (65537, UNSUPPORTED, UNSUPPORTED)])
def test_most_heads(heads, write, read):
    from block_sparse_paged_score_gb300 import bsp
    L, kv = bsp.lib(), bsp.KvCacheDesc()
    assert L.bsp_kv_cache_interleaved(1, heads, 1 << 44, 2, 1.0, 1.0, C.byref(kv)) == 0
    ks, vs, k, v, slot = (i << 36 for i in range(1, 6))
    s = bsp.KvScalesDesc(ks, vs)
    assert L.bsp_kv_scaled_write(C.byref(kv), C.byref(s), k, heads * 128, v, heads * 128, slot, 2, None, None) == write
    assert L.bsp_kv_scaled_read(C.byref(kv), C.byref(s), slot, 2, k, v, None, None) == read
