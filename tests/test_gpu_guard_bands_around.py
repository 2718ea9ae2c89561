"""Guard bands and sentinels around the outputs of the step tables, the norm's
writer, the cache read and the dense attention, as test_gpu_guard_bands has
them around the path's calls: nothing is written outside an output, and no
element that the call defines is left."""
import numpy as np
import pytest
import torch

from plain64 import BF16, FP8, MX
from test_gpu_guard_bands import E4M3_NAN, ID_SENTINEL, NAN16, Guarded, check

pytestmark = pytest.mark.gpu


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("n,capacity", [(1, 1), (3, 700), (257, 1000), (2500, 9001)])
def test_step_tables(n, capacity):
    from block_sparse_paged_score_gb300 import step
    r = np.random.default_rng(n)
    ctx, new = r.integers(0, 400, n), r.integers(0, max(2, 2 * capacity // n), n)
    width, free = 12, np.arange(4000)
    t = step.StepTables(n, width, capacity, 4000)
    g = dict(seq_lens=Guarded((n,), torch.int32, ID_SENTINEL), cu_tokens=Guarded((n + 1,), torch.int32, ID_SENTINEL),
             blocks_taken=Guarded((1,), torch.int32, ID_SENTINEL), query_req_id=Guarded((capacity,), torch.int32, ID_SENTINEL),
             query_abs_pos=Guarded((capacity,), torch.int32, ID_SENTINEL), block_table=Guarded((n, width), torch.int32, 7))
    for k, b in g.items():
        setattr(t.args, k, b.t.data_ptr())
    slot = torch.full((capacity + 128,), 1 << 60, device="cuda")
    t.args.slot = slot[64:].data_ptr()
    t.run(_i32(*ctx), _i32(*new), _i32(*free))
    torch.cuda.synchronize()
    for k, b in g.items():
        check(k, b, complete=k != "block_table")
    assert (slot[:64] == 1 << 60).all() and (slot[64 + capacity:] == 1 << 60).all()
    assert (slot[64:64 + capacity] < 1 << 60).all()
    # table entries before and behind a step's fresh blocks stay
    bt = g["block_table"].t.cpu().numpy()
    have, want = np.minimum(-(-ctx // 128), width), np.minimum(-(-(ctx + new) // 128), width)
    col = np.arange(width)
    assert (bt[(col < have[:, None]) | (col >= want[:, None])] == 7).all()


@pytest.mark.parametrize("T", [1, 37, 4001])
@pytest.mark.parametrize("kv,idx,q8", [(BF16, FP8, False), (FP8, MX, True), (MX, BF16, False)])
def test_norm_rope_write(T, kv, idx, q8):
    from block_sparse_paged_score_gb300 import bsp, step
    hkv, group, blocks = 2, 3, T // 64 + 1
    kvg = Guarded((blocks * bsp.kv_block_bytes(kv, hkv),), torch.uint8)
    idxg = Guarded((blocks * hkv * bsp.index_field_bytes(idx),), torch.uint8)
    K, I = bsp.KvCache(kv, hkv, blocks, buffer=kvg.t), bsp.IndexCache(idx, hkv, blocks, buffer=idxg.t)
    qt = bsp.FP8_E4M3 if q8 else bsp.BF16
    op = step.NormRopeWrite(K, I, hkv * group, T, q_dtype=qt, idx_q_dtype=qt, rope_table=step.rope_table(100, 64))
    dt, bad = (torch.uint8, E4M3_NAN) if q8 else (torch.bfloat16, NAN16)
    out = {n: Guarded((T, h, 128), dt if n != "k_out" else torch.bfloat16, bad if n != "k_out" else NAN16)
           for n, h in (("q_out", hkv * group), ("idx_q_out", hkv), ("k_out", hkv))}
    op.q_out, op.idx_q_out = out["q_out"].t, out["idx_q_out"].t
    op.args.q_out, op.args.k_out = out["q_out"].t.data_ptr(), out["k_out"].t.data_ptr()
    x = [torch.randn(T, h, 128, device="cuda").bfloat16() for h in (hkv * group, hkv, hkv, hkv, hkv)]
    pos = torch.arange(T, dtype=torch.int32, device="cuda") % 100
    op.run(*x, pos, torch.randperm(blocks * 128, device="cuda")[:T])
    torch.cuda.synchronize()
    for n, b in out.items():
        check(n, b)
    check("K/V cache", kvg, complete=False)
    check("index cache", idxg, complete=False)
    assert op.dev_err.item() == 0


@pytest.mark.parametrize("dtype", [BF16, FP8, MX])
@pytest.mark.parametrize("T", [1, 15, 1000])
def test_kv_page_read(T, dtype):
    from block_sparse_paged_score_gb300 import bsp
    kv, idx = bsp.KvCache(dtype, 2, 9), bsp.IndexCache(dtype, 2, 9)
    out = [Guarded((T, 2, 128), torch.bfloat16, NAN16) for _ in range(3)]
    slot = torch.randint(-1, 9 * 128, (T,), device="cuda")
    bsp.kv_page_read(kv, idx, slot, *(g.t for g in out))
    torch.cuda.synchronize()
    for n, g in zip(("k", "v", "idx_k"), out):
        check(n, g)


@pytest.mark.parametrize("q_len,group,hkv", [(1, 16, 1), (3, 4, 2), (4, 16, 1), (8, 16, 1)])
@pytest.mark.parametrize("lens", [[0], [5, 900, 0, 129], [20000], [40] * 700])
def test_dense_attention(lens, q_len, group, hkv):
    from test_gpu_dense_pa import Case
    c = Case(lens, hkv, group, q_len, seed=1).device()
    out = Guarded((len(lens) * q_len, hkv * group, 128), torch.bfloat16, NAN16)
    ws = Guarded((c.bsp.dense_pa_workspace_bytes(len(c.row_len), hkv, group, q_len),), torch.uint8, 0xFF)
    cache = c.buf.clone()
    c.call(out=out.t, ws=ws.t)
    torch.cuda.synchronize()
    check("out", out)
    check("workspace", ws, complete=False)
    assert torch.equal(cache, c.buf) and c.err.item() == 0
