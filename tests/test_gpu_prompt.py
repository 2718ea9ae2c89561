"""bsp_prompt_attention against the definition in 64 bits.

Tolerances, for a row with a = sum p |v| / sum p: weights rounded to bf16, 2^-8
of each; logits as fp32 sums of 128 products (2^-17 of sum |q k| scale at most,
which these inputs keep below 2^5, so 2^-12 of a weight, and in the sum again:
2^-11); the output's rounding, 2^-8 of it."""
import numpy as np
import pytest
import torch

import plain64_scaled as P

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


def problem(seed, nq, nk, hkv, group, pad=0):
    rng = np.random.default_rng(seed)
    cu_q, cu_k = np.cumsum([0] + list(nq)), np.cumsum([0] + list(nk))
    f = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).bfloat16().cuda()  # noqa: E731
    return dict(q=f(cu_q[-1] + pad, hkv * group, 128), k=f(cu_k[-1] + pad, hkv, 128), v=f(cu_k[-1] + pad, hkv, 128),
                cu_q=cu_q, cu_k=cu_k)


def attend(p, scale=SCALE, dev_err=None, **kw):
    from block_sparse_paged_score_gb300 import bsp
    i = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()  # noqa: E731
    err = dev_err if dev_err is not None else torch.zeros(1, dtype=torch.int32, device="cuda")
    out = bsp.prompt_attention(p["q"], p["k"], p["v"], i(p["cu_q"]), i(p["cu_k"]), sm_scale=scale, dev_err=err, **kw)
    assert dev_err is not None or err.item() == 0
    return out


def expected(p, scale=SCALE):
    return P.prompt(P.bits_f64(p["q"]), P.bits_f64(p["k"]), P.bits_f64(p["v"]), p["cu_q"], p["cu_k"], scale)


def close(got, o, a, extra=0.0):
    got = P.bits_f64(got)
    live = ~np.isnan(a)
    tol = (2.0 ** -8 + 2.0 ** -11 + extra) * a + 2.0 ** -8 * np.abs(o) + 1e-30
    bad = live & ~(np.abs(got - o) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], o[bad][:4])


@pytest.mark.parametrize("hkv,group", [(1, 1), (1, 2), (3, 1), (2, 4), (1, 8), (2, 16)])
@pytest.mark.parametrize("nq", [(1,), (1, 2, 3), (127, 128, 129), (17, 0, 256, 0, 5), (300, 1, 64)])
def test_packed_prompts(hkv, group, nq):
    p = problem(sum(nq) + group, nq, nq, hkv, group)
    close(attend(p), *expected(p))


@pytest.mark.parametrize("group", [1, 4, 16])
def test_chunks_over_their_contexts(group):
    nq, nk = (1, 20, 100, 3, 130), (1000, 20, 228, 515, 4000)
    p = problem(5, nq, nk, 2, group)
    close(attend(p), *expected(p))


def test_rows_without_keys_are_zero():
    p = problem(6, (5, 300, 7), (2, 0, 300), 1, 8)
    got = attend(p)
    assert (got[:3] == 0).all() and (got[5:305] == 0).all()
    close(got, *expected(p))


def test_no_keys_at_all():
    p = problem(7, (5, 9), (0, 0), 1, 4)
    assert (attend(p) == 0).all()


@pytest.mark.parametrize("group", [1, 16])
def test_one_long_prompt(group):
    p = problem(8, (2500,), (2500,), 1, group)
    close(attend(p), *expected(p))


def test_few_rows_over_long_keys():
    p = problem(9, (3, 1), (30000, 20001), 1, 16)
    close(attend(p), *expected(p))


def test_many_short_prompts():
    rng = np.random.default_rng(10)
    nq = [int(x) for x in rng.integers(0, 60, 500)]
    p = problem(10, nq, nq, 1, 4)
    close(attend(p), *expected(p))


def test_rows_behind_the_last_sequence_are_left():
    p = problem(11, (40, 90), (40, 90), 1, 8, pad=37)
    out = torch.full((167 + 8, 8, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    got = attend(p, out=out[4:-4])
    assert (out[:4] == 5).all() and (out[4 + 130:] == 5).all()
    close(got, *expected(p))
    assert (attend(p)[130:] == 0).all()


def test_what_no_row_sees_may_be_anything():
    """The next sequence's keys, the rows behind the last one, and keys that are later than the query."""
    for group in (1, 4, 16):
        p = problem(12, (100, 70, 200), (100, 70, 200), 2, group, pad=50)
        o, a = expected(p)
        p["k"][370:], p["v"][370:] = float("nan"), float("inf")
        p["k"][100:170], p["v"][100:170] = float("nan"), float("nan")
        p["k"][170 + 150:370] = float("inf")
        p["v"][170 + 150:370] = float("-inf")
        got = P.bits_f64(attend(p))
        rows = np.r_[0:100, 170:170 + 150]
        tol = (2.0 ** -8 + 2.0 ** -11) * a + 2.0 ** -8 * np.abs(o)
        assert (np.abs(got - o)[rows] <= tol[rows]).all()
        assert np.isnan(got[100:170]).all() and np.isnan(got[320:370]).all()


def test_an_infinite_value_reaches_the_rows_that_see_it():
    p = problem(13, (300,), (300,), 1, 4)
    o, a = expected(p)
    p["v"][140, 0, 3], p["v"][200, 0, 4] = float("inf"), float("nan")
    got = P.bits_f64(attend(p))
    assert (got[140:, :, 3] == np.inf).all() and np.isnan(got[200:, :, 4]).all()
    got[140:, :, 3], got[200:, :, 4] = o[140:, :, 3], o[200:, :, 4]
    assert (np.abs(got - o) <= (2.0 ** -8 + 2.0 ** -11) * a + 2.0 ** -8 * np.abs(o)).all()


@pytest.mark.parametrize("scale", [-0.1, 0.0, 2.0])
def test_scales(scale):
    """(sum |q k| stays below 128 * 5 * 5 / 4 of these inputs: fp32 logits are off by 2^-17 of that times the scale)"""
    p = problem(14, (260,), (260,), 1, 4)
    close(attend(p, scale), *expected(p, scale), extra=2 * 2.0 ** -17 * abs(scale) * 800)


@pytest.mark.parametrize("big", [2.0 ** 12, 2.0 ** 50])
def test_huge_logits(big):
    """Logits past 2^24 and past 2^100: the largest takes the row (q and k have few bits, so that the order of
    the logits is the same in fp32)."""
    p = problem(15, (200,), (200,), 1, 2)
    for n in "qk":
        p[n] = ((p[n].float() * 4).round() / 4 * big).bfloat16()
    o, a = expected(p)
    got = P.bits_f64(attend(p))
    assert (np.abs(got - o) <= (2.0 ** -8 + 2.0 ** -11) * a + 2.0 ** -8 * np.abs(o)).all()


def test_growing_logits_move_the_reference():
    """Keys whose logits grow along the prompt, 12 binades a block: every block moves the rows' references."""
    p = problem(16, (64,), (1200,), 1, 8)
    ramp = torch.linspace(0, 12, 1200, device="cuda")[:, None, None]
    p["q"][:] = (0.1 * p["q"].float() + 1).bfloat16()
    p["k"][:] = (0.1 * p["k"].float() + ramp).bfloat16()
    close(attend(p), *expected(p), extra=2 * 2.0 ** -17 * 200)


def test_strides_and_views():
    from block_sparse_paged_score_gb300 import bsp
    p = problem(17, (30, 200), (30, 200), 2, 4)
    row = torch.zeros(230, 20, 128, dtype=torch.bfloat16, device="cuda")
    row[:, 1:9], row[:, 10:12], row[:, 15:17] = p["q"], p["k"], p["v"]
    cu = torch.tensor([0, 30, 230], dtype=torch.int32, device="cuda")
    got = bsp.prompt_attention(row[:, 1:9], row[:, 10:12], row[:, 15:17], cu)
    assert torch.equal(got, attend(p))


def test_bad_offsets_are_cut():
    p = problem(18, (50, 60), (50, 60), 1, 4)
    o, a = expected(p)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for cu_q, cu_k in (((-5, 50, 110), (-1, 50, 110)), ((0, 50, 200), (0, 50, 2 ** 31 - 1))):
        err.zero_()
        got = attend({**p, "cu_q": cu_q, "cu_k": cu_k}, dev_err=err)
        assert err.item() == 32
        close(got, o, a)
    err.zero_()
    attend({**p, "cu_q": (0, 80, 50), "cu_k": (60, 20, 110)}, dev_err=err)
    assert err.item() == 32
    attend(p, dev_err=err.zero_())
    assert err.item() == 0


def test_the_same_bits_twice_captured_and_on_a_side_stream():
    from block_sparse_paged_score_gb300 import bsp
    p = problem(19, (700, 3, 1100), (700, 9000, 1100), 1, 16)
    want = attend(p)
    assert torch.equal(want, attend(p))
    cu_q, cu_k = (torch.from_numpy(p[n].astype(np.int32)).cuda() for n in ("cu_q", "cu_k"))
    ws, out = bsp.prompt_attention_workspace(want.shape[0], 3, 1, 16), torch.empty_like(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    bsp.prompt_attention(p["q"], p["k"], p["v"], cu_q, cu_k, out=out, ws=ws, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bsp.prompt_attention(p["q"], p["k"], p["v"], cu_q, cu_k, out=out, ws=ws)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
