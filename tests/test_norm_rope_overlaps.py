"""Which overlaps of its tensors bsp_norm_rope_write refuses, on the host, before
anything is enqueued (no GPU needed; with a GPU the tests are left out: the
addresses are no one's)."""
import ctypes as C

import pytest
import torch

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="fake device addresses must never reach a GPU")
T, HQ, HKV = 4, 8, 2
SIZE = dict(q=T * HQ * 256, k=T * HKV * 256, v=T * HKV * 256, idx_q=T * HKV * 256, idx_k=T * HKV * 256, q_weight=256,
            k_weight=256, idx_q_weight=256, idx_k_weight=256, rope_table=100 * 64 * 4, positions=4 * T, slot=8 * T,
            q_out=T * HQ * 256, k_out=T * HKV * 256, idx_q_out=T * HKV * 256, dev_err=4)
AT = {n: (1 << 32) + i * (1 << 26) for i, n in enumerate(SIZE)}
OUT = ["q_out", "k_out", "idx_q_out", "dev_err"]
IN = [n for n in SIZE if n not in OUT]
REFUSED, LAUNCHED = 1, 4  # a launch fails without a device


@pytest.fixture(scope="module")
def bsp():
    from block_sparse_paged_score_gb300 import bsp
    bsp.lib()
    return bsp


def _status(bsp, kv_dtype=1, idx_dtype=2, stride=None, fields=(), **kw):
    kv, idx = bsp.KvCacheDesc(), bsp.IndexCacheDesc()
    assert bsp.lib().bsp_kv_cache_interleaved(kv_dtype, HKV, 1 << 40, 64, 0.5, 0.5, C.byref(kv)) == 0
    assert bsp.lib().bsp_index_cache_packed(idx_dtype, HKV, 1 << 41, 64, C.byref(idx)) == 0
    if stride:
        kv.id_stride_bytes = stride
    a = bsp.NormRopeArgs()
    for k, v in AT.items():
        setattr(a, k, v)
    a.q_stride, a.k_stride, a.v_stride, a.idx_q_stride, a.idx_k_stride = HQ * 128, 256, 256, 256, 256
    a.num_tokens, a.num_q_heads, a.num_kv_heads, a.num_idx_heads = T, HQ, HKV, HKV
    a.eps, a.rope_rows, a.rot_dim = 1e-6, 100, 64
    a.kv, a.idx = C.pointer(kv), C.pointer(idx)
    for k, v in kw.items():
        setattr(a, k, v)
    return bsp.lib().bsp_norm_rope_write(C.byref(a), None)


@pytest.mark.parametrize("out", OUT)
def test_an_output_on_an_input_or_another_output(bsp, out):
    assert _status(bsp) == LAUNCHED
    for other in SIZE:
        if other == out:
            continue
        # its first and its last 16 bytes (the smallest are 4 long), and right before and behind it
        last = AT[other] + (SIZE[other] - 1) // 16 * 16
        before, behind = AT[other] - -(-SIZE[out] // 16) * 16, AT[other] + -(-SIZE[other] // 16) * 16
        in_place = (out, other) in (("q_out", "q"), ("k_out", "k"), ("idx_q_out", "idx_q"))
        assert _status(bsp, **{out: AT[other]}) == (LAUNCHED if in_place else REFUSED), other
        if last != AT[other]:
            assert _status(bsp, **{out: last}) == REFUSED, other
        assert _status(bsp, **{out: before}) == LAUNCHED and _status(bsp, **{out: behind}) == LAUNCHED, other


@pytest.mark.parametrize("kv_dtype", [0, 1, 2])
@pytest.mark.parametrize("name", ["q_out", "k_out", "idx_q_out", "dev_err", "q", "v", "idx_k", "rope_table", "positions",
                                  "slot", "k_weight"])
def test_a_tensor_inside_a_cache(bsp, name, kv_dtype):
    n = 64 * bsp.kv_block_bytes(kv_dtype, HKV)
    behind = -(-SIZE[name] // 16) * 16
    for at in (1 << 40, (1 << 40) + n // 2, (1 << 40) + n - 16):
        assert _status(bsp, kv_dtype, **{name: at}) == REFUSED, at
    assert _status(bsp, kv_dtype, **{name: (1 << 40) + n}) == LAUNCHED
    assert _status(bsp, kv_dtype, **{name: (1 << 40) - behind}) == LAUNCHED
    n = 64 * HKV * 8704
    for at in (1 << 41, (1 << 41) + n // 2, (1 << 41) + n - 16):
        assert _status(bsp, kv_dtype, **{name: at}) == REFUSED, at
    assert _status(bsp, kv_dtype, **{name: (1 << 41) + n}) == LAUNCHED


def test_a_tensor_between_the_pages_of_a_cache_with_room(bsp):
    """One layer of a cache of several: what lies between its pages is another's."""
    for dtype, stride, page in ((1, 8 * 4096, HKV * 2048), (2, 16 * HKV * 8704, 2 * HKV * 8704)):
        for i in (0, 7, 50):  # (ids of K pages)
            at = (1 << 40) + i * stride
            assert _status(bsp, dtype, stride=stride, k_weight=at + page) == LAUNCHED, (dtype, i)
            assert _status(bsp, dtype, stride=stride, k_weight=at + page - 16) == REFUSED, (dtype, i)


def test_tensors_that_the_call_does_not_use(bsp):
    assert _status(bsp, rope_table=AT["q_out"], rot_dim=0) == LAUNCHED
    assert _status(bsp, slot=AT["q_out"], kv=None, idx=None, k=None, v=None, k_out=None, idx_k=None) == LAUNCHED
