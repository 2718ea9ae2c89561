"""bsp_dense_pa_decode_fp8 against the definition in 64 bits.

Tolerances, for a row with a = sum p |v| / sum p: weights rounded to f16, 2^-11
of each; logits as fp32 sums of 128 products (2^-17 of sum |q k| at most, which
these inputs keep below 2^6, so 2^-11 of a weight, in either direction and in
the sum again: 2^-10); a bf16 query's parts, within the same; the output's
rounding, 2^-8 of it."""
import numpy as np
import pytest
import torch

import plain64 as R
import plain64_scaled as P

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


def problem(seed, n, q_len, hkv, group, lens, q8, nb=None, extra=3):
    rng = np.random.default_rng(seed)
    nb = nb or max(1, -(-max(lens) // 128))
    blocks = n * nb + extra
    cache = rng.integers(0, 256, blocks * hkv * 32768, dtype=np.uint8)
    cache = P.e4m3(rng.standard_normal(cache.size) * 60)
    scales = [2.0 ** rng.integers(-8, -4, (blocks, hkv)).astype(np.float32) for _ in range(2)]
    scales = [s.astype(np.float32) for s in scales]
    table = rng.permutation(blocks)[:n * nb].reshape(n, nb).astype(np.int32)
    x = rng.standard_normal((n * q_len, hkv * group, 128))
    if q8:
        q = torch.from_numpy(P.e4m3(x))
        q64 = R.E4M3[q.numpy()]
    else:
        q = torch.from_numpy(x.astype(np.float32)).bfloat16()
        q64 = P.bits_f64(q)
    row_len, row_seq = [], []
    for s in range(n):
        for j in range(q_len):
            row_len += [max(0, lens[s] - (q_len - 1 - j))] * hkv
            row_seq += [s] * hkv
    return dict(cache=cache, scales=scales, table=table, q=q, q64=q64, q8=q8, hkv=hkv, group=group, q_len=q_len,
                blocks=blocks, row_len=np.array(row_len, np.int32), row_seq=np.array(row_seq, np.int32))


def expected(p, scale=SCALE):
    return R.dense_attention(lambda b, side, h: P.block_values(p["cache"], p["scales"], p["hkv"], b, h, side),
                             p["table"], p["q64"], p["row_seq"], p["row_len"], p["hkv"], p["group"], scale)


def attend(p, scale=SCALE, per_tensor=None, err=None, **kw):
    from block_sparse_paged_score_gb300 import bsp
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    if per_tensor is None:
        c = bsp.BlockScaledKvCache(p["hkv"], p["blocks"], buffer=t(p["cache"]), k_scales=t(p["scales"][0]),
                                   v_scales=t(p["scales"][1]))
    else:
        c = bsp.KvCache(bsp.FP8_E4M3, p["hkv"], p["blocks"], *per_tensor, buffer=t(p["cache"]))
    own = err if err is not None else torch.zeros(1, dtype=torch.int32, device="cuda")
    out = bsp.dense_pa_decode_fp8(c, p["q"].cuda(), bsp.FP8_E4M3 if p["q8"] else bsp.BF16, p["hkv"] * p["group"],
                                  t(p["table"]), t(p["row_seq"]), t(p["row_len"]), p["q_len"], sm_scale=scale,
                                  dev_err=own, **kw)
    assert err is not None or own.item() == 0
    return out


def close(got, o, a):
    got = P.bits_f64(got)
    tol = (2.0 ** -11 + 2.0 ** -10) * a + 2.0 ** -8 * np.abs(o) + 1e-30
    bad = ~(np.abs(got - o) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], o[bad][:4])


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("hkv,group", [(1, 1), (2, 2), (1, 4), (3, 8), (1, 16)])
@pytest.mark.parametrize("q_len,lens", [(1, (1, 128, 0, 129, 1000)), (2, (1, 2, 300)), (4, (127, 3, 513)),
                                        (8, (5, 1025, 8))])
def test_heads_lengths_and_types(q8, hkv, group, q_len, lens):
    p = problem(len(lens) * 100 + q_len, len(lens), q_len, hkv, group, lens, q8)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = attend(p, err=err)
    assert err.item() == 0
    close(got, *expected(p))


@pytest.mark.parametrize("q_len,group", [(1, 16), (4, 16), (3, 16), (8, 16), (5, 4)])
def test_long_contexts_that_are_cut(q_len, group):
    p = problem(7, 2, q_len, 1, group, (40000, 33333), False)
    close(attend(p), *expected(p))


def test_more_sequences_than_ctas():
    rng = np.random.default_rng(1)
    lens = [int(x) for x in rng.integers(0, 300, 700)]
    p = problem(8, 700, 1, 1, 4, lens, True)
    close(attend(p), *expected(p))


@pytest.mark.parametrize("scale", [-0.1, 0.0, 3.0])
def test_scales_of_the_softmax(scale):
    """(|z| reaches some hundreds at scale 3: sum |q k| scale stays below 2^11, so the logits' part is 2^-5 of
    those weights at worst; the rows' values then lie on one or two keys, whose errors cancel in the quotient --
    the bound below counts it in full)"""
    p = problem(9, 2, 2, 1, 8, (200, 333), False)
    o, a = expected(p, scale)
    got = P.bits_f64(attend(p, scale))
    z = 2.0 ** -17 * np.abs(scale) * 128 * 4 * 28 / 4  # sum |q k| <= 128 * 4 * 28 of these inputs
    assert (np.abs(got - o) <= (2.0 ** -11 + 2 * z) * a + 2.0 ** -8 * np.abs(o) + 1e-30).all()


def test_per_tensor_scales():
    from block_sparse_paged_score_gb300 import bsp  # noqa: F401
    p = problem(10, 3, 1, 2, 4, (500, 1, 130), False)
    p["scales"] = [np.full((p["blocks"], 2), s, np.float32) for s in (0.0095, 0.0105)]
    close(attend(p, per_tensor=(0.0095, 0.0105)), *expected(p))


def test_block_scales_far_apart():
    """The blocks' V scales span 2^100: a row's reference counts them, so each block's share is right; K scales
    spread so that some blocks' logits are flat."""
    p = problem(11, 1, 1, 1, 16, (128 * 12,), False)
    rng = np.random.default_rng(2)
    p["scales"][1] = (2.0 ** rng.integers(-60, 40, p["scales"][1].shape)).astype(np.float32)
    p["scales"][0] = (2.0 ** rng.integers(-40, -5, p["scales"][0].shape)).astype(np.float32)
    close(attend(p), *expected(p))


def test_what_no_row_sees_may_be_anything():
    """NaN bytes and scales behind the lengths; NaN in V's byte of a token that only later rows of the group see."""
    p = problem(12, 2, 4, 1, 4, (130, 255), False, nb=3)
    o, a = expected(p)
    cache, table = p["cache"], p["table"]
    for s, n in ((0, 130), (1, 255)):
        for t in range(n, 3 * 128):
            for side in (0, 1):
                cache[P.addresses(1, table[s, t // 128], t % 128, 0, side)] = 0x7F if t % 2 else 0xFF
        p["scales"][0][table[s, 2]] = np.nan
        p["scales"][1][table[s, 2]] = np.nan
    close(attend(p), o, a)
    # the third query token of sequence 0 sees tokens up to 128, the fourth 129
    at = P.addresses(1, table[0, 1], 1, 0, 1)[7]
    cache[at] = 0x7F
    got = P.bits_f64(attend(p))
    assert np.isnan(got[3, :, 7]).all()
    o[3, :, 7] = 0
    got[3, :, 7] = 0
    assert (np.abs(got - o) <= (2.0 ** -11 + 2.0 ** -10) * a + 2.0 ** -8 * np.abs(o)).all()


def test_nan_keys_queries_and_scales_give_nan_rows():
    p = problem(13, 3, 1, 1, 4, (200, 200, 200), False)
    p["cache"][P.addresses(1, p["table"][0, 1], 3, 0, 0)[5]] = 0x7F
    p["q"][1, 2, 9] = float("inf")
    p["scales"][1][p["table"][2, 0]] = -1.0
    got = P.bits_f64(attend(p))
    assert np.isnan(got[0]).all() and np.isnan(got[1, 2]).all() and np.isnan(got[2]).all()
    assert np.isfinite(got[1, [0, 1, 3]]).all()


def test_zero_scales():
    """A block of V scale 0 holds zeros (its scale counts as 2^-60), a block of K scale 0 has logits of 0."""
    p = problem(14, 1, 1, 1, 2, (384,), True)
    p["scales"][1][p["table"][0, 1]] = 0
    p["scales"][0][p["table"][0, 2]] = 0
    close(attend(p), *expected(p))


def test_bad_blocks_are_left_out():
    p = problem(15, 2, 1, 1, 4, (384, 256), False)
    q = {**p, "table": p["table"].copy()}
    q["table"][0, 1], q["table"][1, 0] = p["blocks"], -1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = P.bits_f64(attend(q, err=err))
    assert err.item() == 2
    # the same without those tokens
    r = {**p, "table": np.array([[p["table"][0, 0], p["table"][0, 2]], [p["table"][1, 1], 0]], np.int32),
         "row_len": np.array([256, 128], np.int32)}
    o, a = expected(r)
    assert (np.abs(got - o) <= (2.0 ** -11 + 2.0 ** -10) * a + 2.0 ** -8 * np.abs(o)).all()


def test_rows_of_other_sequences_are_flagged():
    p = problem(16, 2, 2, 1, 4, (300, 300), False)
    p["row_seq"][1] = 1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    attend(p, err=err)
    assert err.item() == 4


@pytest.mark.parametrize("big", [2.0 ** 20, 2.0 ** 90])
def test_huge_logits(big):
    """Logits past 2^28, and past 2^90: the largest one takes the row."""
    p = problem(17, 1, 1, 1, 4, (300,), False)
    p["scales"][0][:] = big
    o, a = expected(p)
    close(attend(p), o, a)


def test_the_same_bits_twice_and_guard_bands():
    p = problem(18, 5, 3, 1, 16, (5000, 0, 7777, 1, 300), False)
    n = p["q"].shape[0]
    buf = torch.full((n + 4, 16, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    first = attend(p, out=buf[2:-2]).clone()
    assert (buf[:2] == 9).all() and (buf[-2:] == 9).all()
    assert torch.equal(first, attend(p))


def test_captured_and_on_a_side_stream():
    from block_sparse_paged_score_gb300 import bsp
    p = problem(19, 3, 1, 1, 8, (3000, 10, 700), True)
    want = attend(p)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    c = bsp.BlockScaledKvCache(1, p["blocks"], buffer=t(p["cache"]), k_scales=t(p["scales"][0]), v_scales=t(p["scales"][1]))
    q, table, rs, rl = p["q"].cuda(), t(p["table"]), t(p["row_seq"]), t(p["row_len"])
    ws = bsp.dense_pa_fp8_workspace(3, 1, 8, 1)
    out = torch.empty_like(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    bsp.dense_pa_decode_fp8(c, q, bsp.FP8_E4M3, 8, table, rs, rl, 1, sm_scale=SCALE, out=out, ws=ws, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bsp.dense_pa_decode_fp8(c, q, bsp.FP8_E4M3, 8, table, rs, rl, 1, sm_scale=SCALE, out=out, ws=ws)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
