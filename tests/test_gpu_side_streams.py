"""Calls on a stream of their own whose outputs and workspaces they make
themselves, while the current stream allocates and writes without a pause."""
import numpy as np
import pytest
import torch

from test_gpu_dense_pa import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q_len", [1, 4])
def test_dense_attention_without_a_workspace_on_a_side_stream(q_len):
    c = Case([30000, 1, 900, 12000], q_len=q_len, seed=q_len).device()
    want = c.call().clone()
    n = c.bsp.dense_pa_workspace_bytes(len(c.row_len), 1, 16, q_len)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(20):
        # memory that the current stream is still writing goes back to its pool
        for _ in range(3):
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0x5A)
        out = c.call(stream=side)
        # and what the call gave back would be handed out at once
        busy = [torch.empty(m, dtype=torch.uint8, device="cuda").fill_(0x7F) for m in (n, n, 2 * out.numel())]
        side.synchronize()
        assert torch.equal(out, want), i
        del busy
    torch.cuda.synchronize()
    assert c.err.item() == 0


def test_cache_read_on_a_side_stream():
    from block_sparse_paged_score_gb300 import bsp
    r = np.random.default_rng(5)
    kv = bsp.KvCache(bsp.BF16, 2, 40, buffer=torch.from_numpy(r.integers(0, 256, 40 * bsp.kv_block_bytes(0, 2), dtype=np.uint8)).cuda())
    idx = bsp.IndexCache(bsp.MXFP4, 2, 40)
    idx.buffer.fill_(0x33)
    slot = torch.randperm(40 * 128, device="cuda")
    want = [x.clone() for x in bsp.kv_page_read(kv, idx, slot)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(20):
        for _ in range(4):
            torch.empty(want[0].shape, dtype=torch.bfloat16, device="cuda").fill_(3.0)
        got = bsp.kv_page_read(kv, idx, slot, stream=side)
        side.synchronize()
        assert all(torch.equal(g.view(torch.int16), w.view(torch.int16)) for g, w in zip(got, want)), i
