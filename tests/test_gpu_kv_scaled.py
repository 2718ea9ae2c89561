"""bsp_kv_scaled_write and bsp_kv_scaled_read against the definition run token
by token in 64 bits: bytes and scales are equal bit for bit (every rounding is
one e4m3 rounding of a value that fp32 holds exactly: x / s with s a power of
two, or a byte times a power of two)."""
import numpy as np
import pytest
import torch

import plain64_scaled as P
from plain64 import E4M3

pytestmark = pytest.mark.gpu


def make(rng, hkv, blocks, pow2=True):
    cache = rng.integers(0, 256, blocks * hkv * 32768, dtype=np.uint8)
    cache[(cache & 127) == 127] ^= 1
    scales = [(2.0 ** rng.integers(-9, -5, (blocks, hkv)) * (1 if pow2 else 1.3)).astype(np.float32) for _ in range(2)]
    return cache, scales


def rows(rng, T, hkv, spread=6):
    x = rng.standard_normal((T, hkv, 128)) * 2.0 ** rng.integers(-spread, 3, (T, 1, 1))
    return torch.from_numpy(x.astype(np.float32)).bfloat16()


def device_cache(cache, scales, hkv, blocks):
    from block_sparse_paged_score_gb300 import bsp
    c = [torch.from_numpy(x.copy()).cuda() for x in (cache, *scales)]
    return bsp.BlockScaledKvCache(hkv, blocks, buffer=c[0], k_scales=c[1], v_scales=c[2])


def check(cache, scales, hkv, blocks, k, v, slot, err_want=None):
    from block_sparse_paged_score_gb300 import bsp
    dev = device_cache(cache, scales, hkv, blocks)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bsp.kv_scaled_write(dev, k.cuda(), v.cuda(), torch.from_numpy(slot).cuda(), dev_err=err)
    want_c, want_s = cache.copy(), [s.copy() for s in scales]
    bits = P.scaled_write(want_c, want_s, hkv, P.bits_f64(k), P.bits_f64(v), slot, blocks)
    assert err.item() == bits and (err_want is None or bits == err_want)
    assert np.array_equal(dev.k_scales.cpu().numpy(), want_s[0])
    assert np.array_equal(dev.v_scales.cpu().numpy(), want_s[1])
    got = dev.buffer.cpu().numpy()
    # a NaN byte may change its sign
    same = (got == want_c) | (((got & 127) == 127) & ((want_c & 127) == 127))
    assert same.all(), np.argwhere(~same)[:5]
    return dev


def slots_of(blocks_list, starts, lens):
    """consecutive slots of sequences, each over its own blocks"""
    out = []
    for ids, at, n in zip(blocks_list, starts, lens):
        out += [ids[(at + i) // 128] * 128 + (at + i) % 128 for i in range(n)]
    return np.array(out, np.int64)


@pytest.mark.parametrize("hkv", [1, 2, 3])
@pytest.mark.parametrize("starts,lens", [((0,), (1,)), ((5,), (1,)), ((0, 127, 16, 15), (128, 1, 16, 17)),
                                         ((100, 3), (200, 300)), ((0, 0, 64), (127, 129, 64))])
def test_runs_of_any_start_and_length(hkv, starts, lens):
    rng = np.random.default_rng(hkv * 100 + sum(lens))
    per = [(a + n + 127) // 128 for a, n in zip(starts, lens)]
    blocks = sum(per) + 2
    ids = rng.permutation(blocks)
    cut = np.cumsum([0] + per)
    slot = slots_of([ids[a:b] for a, b in zip(cut, cut[1:])], starts, lens)
    cache, scales = make(rng, hkv, blocks)
    check(cache, scales, hkv, blocks, rows(rng, len(slot), hkv), rows(rng, len(slot), hkv), slot)


def test_many_tokens_take_the_long_grid():
    """64 requests of one token and one of 4900: the choice of tokens a CTA goes the other way."""
    rng = np.random.default_rng(4)
    starts, lens = [int(x) for x in rng.integers(1, 128, 64)] + [7], [1] * 64 + [4900]
    per = [(a + n + 127) // 128 for a, n in zip(starts, lens)]
    per[-1] += 1
    blocks = sum(per)
    ids = rng.permutation(blocks)
    cut = np.cumsum([0] + per)
    slot = slots_of([ids[a:b] for a, b in zip(cut, cut[1:])], starts, lens)
    slot[70] = -1  # a hole ends a run; what follows starts in the next block
    slot[71:] = slots_of([ids[cut[-2]:]], [128], [len(slot) - 71])
    cache, scales = make(rng, 1, blocks)
    check(cache, scales, 1, blocks, rows(rng, len(slot), 1), rows(rng, len(slot), 1), slot)


def test_pads_bad_slots_and_repeated_slots():
    rng = np.random.default_rng(9)
    cache, scales = make(rng, 2, 6)
    slot = np.array([-1, 3 * 128 + 9, 3 * 128 + 9, 3 * 128 + 8, -1, -7, 6 * 128, 2 ** 40, 128, 129, 128, 5 * 128 + 127, -1],
                    np.int64)
    check(cache, scales, 2, 6, rows(rng, len(slot), 2), rows(rng, len(slot), 2), slot, 16)


def test_tokens_in_any_order_within_a_run():
    rng = np.random.default_rng(10)
    cache, scales = make(rng, 1, 3)
    slot = np.concatenate([128 + rng.permutation(100) + 20, 256 + rng.permutation(128)]).astype(np.int64)
    check(cache, scales, 1, 3, rows(rng, 228, 1), rows(rng, 228, 1), slot)


@pytest.mark.parametrize("value", [0.0, 2.0 ** -133, 2.0 ** -62, 448.0 * 2.0 ** -60, 449.0, 448.0, 450.0, 3.3e38,
                                   float("inf"), float("nan")])
def test_extreme_rows(value):
    """A row of one value: the least scale's border, what saturates, what is not finite; into a new block and
    into one that holds values."""
    rng = np.random.default_rng(3)
    for slot in ([0], [130]):
        cache, scales = make(rng, 1, 2)
        x = torch.full((1, 1, 128), value).bfloat16()
        x[0, 0, ::3] = -x[0, 0, ::3]
        y = rows(rng, 1, 1)
        y[0, 0, 5] = value
        check(cache, scales, 1, 2, x, y, np.array(slot, np.int64))


def test_scales_that_are_no_powers_of_two_and_nan_bytes():
    """fp32 rounds old / s and the product, then e4m3 rounds: a value may differ from the definition's where
    that is within 2^-22 of a tie; these seeds hold none."""
    rng = np.random.default_rng(5)
    cache, scales = make(rng, 1, 4, pow2=False)
    cache[5::97] = 0x7F
    cache[9::97] = 0xFF
    k, v = rows(rng, 3, 1) * 100, rows(rng, 3, 1) * 100
    check(cache, scales, 1, 4, k, v, np.array([130, 131, 400], np.int64))


def test_a_block_filled_token_by_token_reads_as_written_at_once():
    """Growing scales are powers of two: bytes move by whole exponents, so only what became subnormal differs,
    by at most half a step of the last scale's subnormals, 2^-10 of it, for each time that the scale grew."""
    from block_sparse_paged_score_gb300 import bsp
    rng = np.random.default_rng(6)
    n = 128
    k, v = rows(rng, n, 2).cuda(), rows(rng, n, 2).cuda()
    slot = torch.arange(n, device="cuda")
    once, grown = (bsp.BlockScaledKvCache(2, 1) for _ in range(2))
    bsp.kv_scaled_write(once, k, v, slot)
    for t in range(n):
        bsp.kv_scaled_write(grown, k[t:t + 1], v[t:t + 1], slot[t:t + 1])
    assert torch.equal(once.k_scales, grown.k_scales) and torch.equal(once.v_scales, grown.v_scales)
    for a, b, s in zip(bsp.kv_scaled_read(once, slot), bsp.kv_scaled_read(grown, slot), (once.k_scales, once.v_scales)):
        # nine scales at most (2^-6 .. 2^2 of spread 6): each growth rounds once
        assert ((a.float() - b.float()).abs() <= 9 * 2.0 ** -10 * s[0][None, :, None]).all()


def test_strided_rows():
    rng = np.random.default_rng(8)
    from block_sparse_paged_score_gb300 import bsp
    row = rows(rng, 40, 7).cuda()
    k, v = row[:, 1:3], row[:, 4:6]
    slot = torch.arange(40, device="cuda") + 100
    a, b = (bsp.BlockScaledKvCache(2, 2) for _ in range(2))
    bsp.kv_scaled_write(a, k, v, slot)
    bsp.kv_scaled_write(b, k.contiguous(), v.contiguous(), slot)
    assert torch.equal(a.buffer, b.buffer) and torch.equal(a.k_scales, b.k_scales)


@pytest.mark.parametrize("T,hkv", [(1, 1), (15, 2), (16, 1), (333, 3), (2000, 1)])
def test_read(T, hkv):
    """e4m3 * scale is one fp32 product of 4 and 24 significant bits, then one bf16 rounding: with a power of
    two as scale both are exact, else off by at most 2^-8 + 2^-24 of the value."""
    from block_sparse_paged_score_gb300 import bsp
    rng = np.random.default_rng(T)
    blocks = T // 128 + 2
    for pow2 in (True, False):
        cache, scales = make(rng, hkv, blocks, pow2)
        cache[1::53] = 0x7F
        dev = device_cache(cache, scales, hkv, blocks)
        slot = rng.permutation(blocks * 128)[:T].astype(np.int64)
        if T > 4:
            slot[2], slot[4] = -1, blocks * 128
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        k, v = bsp.kv_scaled_read(dev, torch.from_numpy(slot).cuda(), dev_err=err)
        assert err.item() == (16 if T > 4 else 0)
        for side, got in ((0, P.bits_f64(k)), (1, P.bits_f64(v))):
            for t, s in enumerate(slot):
                for h in range(hkv):
                    if not 0 <= s < blocks * 128:
                        assert (got[t, h] == 0).all()
                        continue
                    want = E4M3[cache[P.addresses(hkv, s // 128, s % 128, h, side)]] * float(scales[side][s // 128, h])
                    tol = 0 if pow2 else (2.0 ** -8 + 2.0 ** -24) * np.abs(want)
                    ok = (np.abs(got[t, h] - want) <= tol) | (np.isnan(want) & np.isnan(got[t, h]))
                    assert ok.all(), (t, h, side)


def test_guard_bands_and_an_empty_call():
    from block_sparse_paged_score_gb300 import bsp
    rng = np.random.default_rng(12)
    hkv, blocks, band = 2, 3, 4096
    n = blocks * hkv * 32768
    buf = torch.full((n + 2 * band,), 0xA5, dtype=torch.uint8, device="cuda")
    sc = torch.full((2, blocks * hkv + 32), 7.0, device="cuda")
    c = bsp.BlockScaledKvCache(hkv, blocks, buffer=buf[band:band + n], k_scales=sc[0, 16:-16].view(blocks, hkv),
                               v_scales=sc[1, 16:-16].view(blocks, hkv))
    k, v = rows(rng, 300, hkv).cuda(), rows(rng, 300, hkv).cuda()
    bsp.kv_scaled_write(c, k[:0], v[:0], torch.empty(0, dtype=torch.int64, device="cuda"))
    assert (buf == 0xA5).all()
    bsp.kv_scaled_write(c, k, v, torch.arange(300, device="cuda") + 84)
    assert (buf[:band] == 0xA5).all() and (buf[-band:] == 0xA5).all()
    assert (sc[:, :16] == 7).all() and (sc[:, -16:] == 7).all()
    out = torch.full((2, 300 + 8, hkv, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    bsp.kv_scaled_read(c, torch.arange(300, device="cuda") + 84, k=out[0, 4:-4], v=out[1, 4:-4])
    assert (out[:, :4] == 3).all() and (out[:, -4:] == 3).all()
