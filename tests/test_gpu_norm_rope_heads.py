"""bsp_norm_rope_write with many heads and with many tokens of few heads, on both
sides of where a half-warp takes all heads of its token."""
import pytest
import torch

import test_gpu_norm_rope as base
from plain64 import BF16, FP8, MX
from test_gpu_norm_rope_values import _check, strict  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv,idx,rot,pairs,q8", [(BF16, BF16, 64, False, True), (FP8, FP8, 128, True, False),
                                                 (MX, MX, 64, False, False), (FP8, MX, 0, False, True)])
@pytest.mark.parametrize("T,hkv,group", [(2801, 1, 60), (2600, 1, 60), (5003, 2, 4), (7500, 1, 4)])
def test_values(T, hkv, group, kv, idx, rot, pairs, q8):
    _check(base.Case(T, hkv, group, kv, idx, rot, pairs, q8, pads=5, seed=T + kv))


@pytest.mark.parametrize("T,hkv,group", [(2801, 1, 60), (7500, 1, 4), (5003, 3, 2)])
@pytest.mark.parametrize("kv,idx,pairs", [(MX, FP8, False), (FP8, MX, True), (BF16, BF16, False)])
def test_the_same_row_in_a_short_and_a_long_batch(T, hkv, group, kv, idx, pairs):
    """Both kernels round alike: a long batch's rows are bit for bit those of its
    parts, rows whose squares leave fp32's range among them."""
    c = base.Case(T, hkv, group, kv, idx, 64, pairs, q8=True, seed=31)
    for x in c.x.values():
        x[::7] *= 2.0 ** 70
        x[1::7] *= 2.0 ** -70
    q, iq = (t.clone() for t in c.run())
    caches = c.kv.buffer.clone(), c.idx.buffer.clone()
    c.kv.buffer.zero_(), c.idx.buffer.zero_()
    x, pos, slot = c.x, c.pos.cuda(), c.slot.cuda()
    for a in range(0, T, 600):
        s = slice(a, min(a + 600, T))
        got = c.op.run(x["q"][s], x["k"][s], x["v"][s], x["idx_q"][s], x["idx_k"][s], pos[s], slot[s])
        assert torch.equal(got[0], q[s]) and torch.equal(got[1], iq[s])
    assert torch.equal(c.kv.buffer, caches[0]) and torch.equal(c.idx.buffer, caches[1])
    assert c.op.dev_err.item() == 0


@pytest.mark.parametrize("T,group", [(2801, 60), (7500, 4)])
def test_in_place_and_captured(T, group):
    c = base.Case(T, 1, group, FP8, MX, 64, fused=False, seed=T)
    want = c.run()[0].clone()
    x, pos, slot = c.x, c.pos.cuda(), c.slot.cuda()
    kept = x["q"].clone()
    c.op.args.q_out = x["q"].data_ptr()  # (in place; the object's own rows stay as they were)
    args = (x["q"], x["k"], x["v"], x["idx_q"], x["idx_k"], pos, slot)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.op.run(*args)
    for _ in range(3):
        x["q"].copy_(kept)
        g.replay()
        assert torch.equal(x["q"], want)
