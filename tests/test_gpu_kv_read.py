"""bsp_kv_page_read against the cache's bytes decoded in 64 bits: bf16 and MXFP4
values are exact, fp8 ones one rounding of e4m3 * scale."""
import numpy as np
import pytest
import torch

from plain64 import BF16, FP8, MX, bf16_to_f64, f64_to_bf16, idx_token, kv_token

pytestmark = pytest.mark.gpu
KS, VS = 0.0095, 0.0105


def _bytes(r, dtype, n):
    b = r.integers(0, 256, n, dtype=np.uint8)
    if dtype == BF16:  # finite values
        w = b.view(np.uint16)
        w[(w & 0x7F80) == 0x7F80] &= 0xBFFF
    elif dtype == FP8:
        b[(b & 127) == 127] -= 1
    else:
        f = b.reshape(-1, 8704)
        f[:, 8192:] = r.integers(100, 150, (f.shape[0], 512))
    return b


def _slots(r, blocks, T, order):
    if order == "random":
        s = r.integers(0, blocks * 128, T)
    else:  # a run that starts inside a page
        s = (5 + np.arange(T)) % (blocks * 128)
    s = s.astype(np.int64)
    if T > 3:
        s[T // 2], s[T - 1] = -1, -7
    return s


def _rounded(values, scale):
    """fp32 product of an e4m3 value and the fp32 scale, rounded to bf16 bits."""
    return f64_to_bf16((values.astype(np.float32) * np.float32(scale)))


@pytest.mark.parametrize("dtype", [BF16, FP8, MX])
@pytest.mark.parametrize("T,hkv,order", [(1, 1, "random"), (15, 2, "run"), (16, 1, "run"), (17, 4, "random"),
                                         (333, 2, "random"), (400, 1, "run")])
def test_k_and_v(dtype, T, hkv, order):
    from block_sparse_paged_score_gb300 import bsp
    r = np.random.default_rng(T * 10 + hkv)
    blocks = 4
    raw = _bytes(r, dtype, blocks * bsp.kv_block_bytes(dtype, hkv))
    kv = bsp.KvCache(dtype, hkv, blocks, KS, VS, buffer=torch.from_numpy(raw).cuda())
    slot = _slots(r, blocks, T, order)
    k, v, none = bsp.kv_page_read(kv, None, torch.from_numpy(slot).cuda())
    assert none is None
    k, v = (x.view(torch.int16).cpu().numpy().view(np.uint16) for x in (k, v))
    for t in range(T):
        ek, ev = (np.zeros((hkv, 128)),) * 2 if slot[t] < 0 else kv_token(raw, dtype, hkv, slot[t])
        if dtype == FP8:
            assert np.array_equal(k[t], _rounded(ek, KS)) and np.array_equal(v[t], _rounded(ev, VS)), t
        else:
            assert np.array_equal(bf16_to_f64(k[t]), ek) and np.array_equal(bf16_to_f64(v[t]), ev), t


@pytest.mark.parametrize("dtype", [BF16, FP8, MX])
@pytest.mark.parametrize("heads", [1, 3])
def test_index_keys(dtype, heads):
    from block_sparse_paged_score_gb300 import bsp
    r = np.random.default_rng(heads)
    blocks, T = 3, 70
    size = {BF16: 32768, FP8: 16896, MX: 8704}[dtype]
    raw = _bytes(r, dtype, blocks * heads * size)
    if dtype == FP8:
        raw.reshape(-1, size)[:, 16384:] = r.uniform(0.001, 3, (blocks * heads, 128)).astype(np.float32).view(np.uint8)
    idx = bsp.IndexCache(dtype, heads, blocks, buffer=torch.from_numpy(raw).cuda())
    slot = _slots(r, blocks, T, "random")
    got = bsp.kv_page_read(None, idx, torch.from_numpy(slot).cuda())[2].view(torch.int16).cpu().numpy().view(np.uint16)
    for t in range(T):
        for h in range(heads):
            if slot[t] < 0:
                assert not got[t, h].any()
                continue
            val, sc = idx_token(raw, dtype, heads, slot[t])
            want = _rounded(val[h], sc[h]) if dtype == FP8 else f64_to_bf16(val[h])
            assert np.array_equal(got[t, h], want), (t, h)


def test_slot_beyond_the_cache_reads_zeros_and_is_flagged():
    from block_sparse_paged_score_gb300 import bsp
    kv = bsp.KvCache(MX, 1, 2)
    kv.buffer.fill_(0x22)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    slot = torch.tensor([3, 256, 255, 1 << 40], device="cuda")
    k, v, _ = bsp.kv_page_read(kv, None, slot, dev_err=err)
    assert err.item() == 16
    assert (k[1] == 0).all() and (v[3] == 0).all() and (k[0] != 0).all() and (v[2] != 0).all()


def test_reads_back_what_the_writer_stored():
    from block_sparse_paged_score_gb300 import bsp
    kv, idx = bsp.KvCache(BF16, 2, 3), bsp.IndexCache(BF16, 2, 3)
    x = torch.randn(3, 50, 2, 128, device="cuda").bfloat16()
    slot = torch.randperm(3 * 128, device="cuda")[:50]
    bsp.kv_page_write(kv, idx, x[0], x[1], x[2], slot)
    for got, want in zip(bsp.kv_page_read(kv, idx, slot), x):
        assert torch.equal(got, want)


def test_rows_behind_the_last_token_are_left():
    from block_sparse_paged_score_gb300 import bsp
    kv = bsp.KvCache(FP8, 1, 1)
    k = torch.full((40, 1, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    bsp.kv_page_read(kv, None, torch.arange(33, device="cuda"), k=k, v=v)
    assert (k[33:] == 7).all() and (v[33:] == 7).all() and (k[:33] == 0).all()
