"""Prompt attention and the block-scaled cache's operators at their edges: scales
that are no numbers, many sequences, addresses past 32 bits, calls at once,
workspaces that graphs share, guard bands, drawn problems.  Tolerances as in the
operators' own tests."""
import numpy as np
import pytest
import torch

import plain64_scaled as P
import test_gpu_dense_pa_fp8 as D
import test_gpu_prompt as A

pytestmark = pytest.mark.gpu


def equal(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("q_len,group", [(2, 4), (4, 16)])
@pytest.mark.parametrize("side,value", [(0, np.nan), (0, np.inf), (1, np.nan), (1, np.inf), (1, -1.0)])
def test_a_scale_that_is_no_number_reaches_the_rows_that_see_its_block(side, value, q_len, group):
    """the last query token alone sees the last block"""
    p = D.problem(21, 2, q_len, 1, group, (257, 200), False, nb=3)
    o, a = D.expected(p)
    p["scales"][side][p["table"][0, 2]] = value
    got = P.bits_f64(D.attend(p))
    hit = q_len - 1
    if value != np.inf:
        assert np.isnan(got[hit]).all()
    rest = np.arange(2 * q_len) != hit
    tol = (2.0 ** -11 + 2.0 ** -10) * a + 2.0 ** -8 * np.abs(o) + 1e-30
    assert (np.abs(got - o) <= tol)[rest].all()


@pytest.mark.parametrize("group", [2, 16])
def test_more_sequences_than_threads(group):
    rng = np.random.default_rng(5)
    nq = rng.integers(0, 4, 1500)
    nk = nq + np.where(rng.integers(0, 9, 1500) == 0, rng.integers(0, 300, 1500), 0)
    p = A.problem(22, nq, nk, 1, group)
    A.close(A.attend(p), *A.expected(p))


@pytest.mark.parametrize("hkv,group", [(16, 8), (40, 1)])
def test_many_heads(hkv, group):
    nq, nk = (40, 1, 150), (40, 700, 300)
    p = A.problem(23, nq, nk, hkv, group)
    A.close(A.attend(p), *A.expected(p))


@pytest.mark.parametrize("power", [70, -70])
def test_values_far_from_one(power):
    """V times a power of two gives the output times it, bit for bit, also where later
    logits are up to e^20 times the first block's: nothing overflows on the way"""
    p = A.problem(27, (300, 1, 40), (300, 3000, 1500), 2, 8)
    ramp = torch.linspace(0, 1, len(p["k"]), device="cuda")[:, None]
    p["k"][..., 0] = (ramp * 20 * 128 ** 0.5).bfloat16()
    p["q"][..., 0] = 1
    want = A.attend(p)
    A.close(want, *A.expected(p))
    p["v"] = p["v"] * 2.0 ** power
    assert equal(A.attend(p), want * 2.0 ** power)


def test_shares_that_are_lengthened_to_fit_the_units():
    """some tokens of each request, three units a head, over more keys than L2 holds"""
    nk = (13000, 12000, 14001, 13000, 13100, 12900, 13000, 13333)
    p = A.problem(26, (33, 40, 33, 47, 33, 33, 35, 33), nk, 4, 16)
    A.close(A.attend(p), *A.expected(p))


def test_a_cache_past_32_bits():
    """Write, read and attention in the last of 131100 blocks (4.3 GB) give what a
    small cache with the same tokens gives."""
    from block_sparse_paged_score_gb300 import bsp
    nb, last = 131100, 8
    far = bsp.BlockScaledKvCache(1, nb, buffer=torch.empty(nb * 32768, dtype=torch.uint8, device="cuda"))
    near = bsp.BlockScaledKvCache(1, last)
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(700, 1, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
    slot = torch.arange(700, device="cuda") + 128
    q = torch.randn(3, 4, 128, generator=g, device="cuda").bfloat16()
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    got = []
    for c, first in ((far, nb - last), (near, 0)):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        for part in (slice(0, 690), slice(690, 700)):
            bsp.kv_scaled_write(c, k[part], v[part], slot[part] + first * 128, dev_err=err)
        rk, rv = bsp.kv_scaled_read(c, slot + first * 128, dev_err=err)
        table = (torch.arange(1, 7, dtype=torch.int32, device="cuda") + first).view(1, 6)
        o = bsp.dense_pa_decode_fp8(c, q, bsp.BF16, 4, table, i(0, 0, 0), i(698, 699, 700), 3, dev_err=err)
        assert err.item() == 0
        got.append((rk, rv, o, c.k_scales[first:first + last], c.v_scales[first:first + last],
                    c.buffer[(first + 1) * 32768:(first + 6) * 32768]))
    for x, y in zip(*got):
        assert equal(x, y)


def test_rows_past_32_bits():
    """K and V rows 128 KB apart, 5.2 GB in all, attend like dense ones."""
    from block_sparse_paged_score_gb300 import bsp
    n, stride = 40000, 65536
    g = torch.Generator(device="cuda").manual_seed(2)
    rows = torch.empty(n, stride, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.randn(n, 2, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
    fk, fv = rows[:, :256].view(n, 2, 128), rows[:, 65280:].view(n, 2, 128)
    fk.copy_(k), fv.copy_(v)
    q = torch.randn(5, 8, 128, generator=g, device="cuda").bfloat16()
    cu_q, cu_k = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ((0, 2, 5), (0, 20, n)))
    assert equal(bsp.prompt_attention(q, fk, fv, cu_q, cu_k), bsp.prompt_attention(q, k, v, cu_q, cu_k))


def calls():
    """a prompt attention and a dense attention whose units are cut, as functions of a workspace"""
    from block_sparse_paged_score_gb300 import bsp
    p, d = A.problem(24, (400, 3, 900), (1400, 9000, 900), 2, 4), D.problem(25, 3, 2, 2, 4, (9000, 77, 20000), False)
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    i = lambda x: t(np.asarray(x, np.int32))  # noqa: E731
    cu_q, cu_k = i(p["cu_q"]), i(p["cu_k"])
    c = bsp.BlockScaledKvCache(2, d["blocks"], buffer=t(d["cache"]), k_scales=t(d["scales"][0]), v_scales=t(d["scales"][1]))
    q, table, seq, lens = d["q"].cuda(), t(d["table"]), t(d["row_seq"]), t(d["row_len"])
    return (lambda ws, out: bsp.prompt_attention(p["q"], p["k"], p["v"], cu_q, cu_k, out=out, ws=ws),
            lambda: bsp.prompt_attention_workspace(len(p["q"]), 3, 2, 4), lambda: torch.zeros_like(p["q"])), \
           (lambda ws, out: bsp.dense_pa_decode_fp8(c, q, bsp.BF16, 8, table, seq, lens, 2, out=out, ws=ws),
            lambda: bsp.dense_pa_fp8_workspace(len(lens), 2, 4, 2), lambda: torch.zeros_like(q))


def test_calls_that_know_only_per_tensor_scales_give_nan():
    from block_sparse_paged_score_gb300 import bsp
    c = bsp.BlockScaledKvCache(1, 2)
    x = torch.ones(20, 1, 128, dtype=torch.bfloat16, device="cuda")
    slot = torch.arange(20, device="cuda")
    bsp.kv_scaled_write(c, x, x, slot)
    k, v = bsp.kv_scaled_read(c, slot)
    assert equal(k, x) and equal(v, x)
    k, v, _ = bsp.kv_page_read(c, None, slot)
    assert k.isnan().all() and v.isnan().all()
    i = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    table = i(0, 1).view(1, 2)
    kv = bsp.KvCache(bsp.FP8_E4M3, 1, 2, c.desc.k_scale, c.desc.v_scale, buffer=c.buffer)
    assert bsp.dense_pa_decode_fp8(kv, x[:1], bsp.BF16, 1, table, i(0), i(20), 1).isnan().all()
    assert equal(bsp.dense_pa_decode_fp8(c, x[:1], bsp.BF16, 1, table, i(0), i(20), 1), x[:1])


def test_calls_at_once():
    """both operators on four streams, each with its own workspace"""
    both = calls()
    want = [call(ws(), out()) for call, ws, out in both]
    streams = [torch.cuda.Stream() for _ in range(4)]
    mine = [(both[n % 2], both[n % 2][1](), both[n % 2][2]()) for n in range(4)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, ((call, _, _), ws, out) in zip(streams, mine):
            with torch.cuda.stream(s):
                call(ws, out)
    torch.cuda.synchronize()
    for n, (_, _, out) in enumerate(mine):
        assert equal(out, want[n % 2])


def test_graphs_that_share_a_workspace():
    """two captured calls of the same operator and one workspace, replayed in turn on
    one stream; what the workspace holds does not count"""
    for call, ws, out in calls():
        want = call(ws(), out())
        w, o = ws(), [out(), out()]
        torch.cuda.synchronize()
        graphs = []
        for x in o:
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                call(w, x)
        for n in range(6):
            w.fill_(0xFF if n % 2 else 0x7F)
            o[n % 2].zero_()
            graphs[n % 2].replay()
            graphs[n % 2].replay()
            assert equal(o[n % 2], want)


def test_outputs_and_workspaces_stay_in_their_bounds():
    for call, ws, out in calls():
        want, w, o = call(ws(), out()), ws(), out()
        gw = torch.full((w.numel() + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
        go = torch.full((o.numel() * 2 + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
        inner = go[4096:-4096].view(torch.bfloat16).view(o.shape)
        call(gw[4096:-4096], inner)
        assert equal(inner, want)
        for x in (gw, go):
            assert (x[:4096] == 0xA5).all() and (x[-4096:] == 0xA5).all()


@pytest.mark.parametrize("seed", range(12))
def test_drawn_prompts(seed):
    rng = np.random.default_rng(100 + seed)
    hkv, group = int(rng.integers(1, 4)), int(rng.choice([1, 2, 4, 8, 16]))
    n = int(rng.integers(1, 7))
    nq = rng.integers(0, int(rng.choice([3, 40, 300])), n) + (rng.integers(0, 3, n) > 0)
    if not nq.any():
        nq[0] = 1
    nk = np.maximum(nq + rng.integers(-20, int(rng.choice([1, 200, 2000])), n), 0)
    p = A.problem(200 + seed, nq, nk, hkv, group, pad=int(rng.integers(0, 5)))
    scale = float(rng.choice([128 ** -0.5, -0.05, 0.0, 0.02]))
    A.close(A.attend(p, scale), *A.expected(p, scale))


@pytest.mark.parametrize("seed", range(12))
def test_drawn_decode_batches(seed):
    rng = np.random.default_rng(300 + seed)
    hkv, group, q_len = int(rng.integers(1, 4)), int(rng.choice([1, 2, 4, 8, 16])), int(rng.integers(1, 9))
    n = int(rng.integers(1, 9))
    lens = rng.integers(0, int(rng.choice([4, 130, 1500, 6000])), n).tolist()
    lens[0] = max(lens[0], 1)
    p = D.problem(400 + seed, n, q_len, hkv, group, lens, bool(rng.integers(0, 2)))
    scale = float(rng.choice([128 ** -0.5, -0.05, 0.0, 0.02]))
    D.close(D.attend(p, scale), *D.expected(p, scale))
