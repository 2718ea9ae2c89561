"""bsp_norm_rope_write against its definition in 64 bits.

Error of the fp32 row before its one rounding, u = 2^-24: the mean of 128
squares is off by at most 13u (8 products and sums in a lane, 4 shuffle adds,
one scaling), so its inverse root by 7u, and by 4u of the root itself; two
products and the weight's sum add 4u; the rotation two products and a sum, 3u
of |a c| + |b s| <= 2 hypot(a, b).  Together under 32u hypot(a, b) = 2^-19
hypot(a, b).  A rounding adds half a step: 2^-8 |y| for bf16; max(2^-4 |y|,
2^-10) for e4m3; a quarter, a half or one below 2, 4 and 6 for e2m1."""
import numpy as np
import pytest
import torch

from plain64 import BF16, FP8, MX, bf16_to_f64, idx_token, kv_token, norm_rope, E4M3

pytestmark = pytest.mark.gpu
KS, VS = 0.0095, 0.0105
SLACK = 2.0 ** -19


class Case:
    def __init__(self, T, hkv, group, kv, idx, rot, pairs=False, q8=False, weight=True, offset=0.0, pads=0, seed=0,
                 fused=True, scale=2.0, eps=1e-6):
        from block_sparse_paged_score_gb300 import bsp, step
        g = torch.Generator().manual_seed(seed)
        hq = hkv * group
        sizes = [hq * 128, hkv * 128, hkv * 128, hkv * 128, hkv * 128]
        row = (torch.randn(T, sum(sizes) + 64, generator=g) * scale * (0.05 + torch.rand(T, 1, generator=g))).bfloat16().cuda()
        parts = torch.split(row[:, :sum(sizes)], sizes, 1)
        if not fused:
            parts = [p.contiguous() for p in parts]
        self.x = dict(zip(("q", "k", "v", "idx_q", "idx_k"), (p.view(T, -1, 128) for p in parts)))
        self.w = {n: ((1 - offset + 0.3 * torch.randn(128, generator=g)).bfloat16().cuda() if weight else None)
                  for n in ("q", "k", "idx_q", "idx_k")}
        self.pos = torch.randint(0, 5000, (T,), generator=g, dtype=torch.int32)
        self.blocks = 2 + T // 128
        self.slot = torch.randperm(self.blocks * 128, generator=g)[:T]
        if pads:
            self.pos[T - pads:], self.slot[T - pads:] = -1, -1
        self.rope = step.rope_table(5000, rot, 1e6) if rot else None
        self.T, self.hkv, self.hq, self.kvt, self.idxt = T, hkv, hq, kv, idx
        self.rot, self.pairs, self.q8, self.offset, self.eps = rot, pairs, q8, offset, eps
        self.kv, self.idx = bsp.KvCache(kv, hkv, self.blocks, KS, VS), bsp.IndexCache(idx, hkv, self.blocks)
        qt = bsp.FP8_E4M3 if q8 else bsp.BF16
        self.op = step.NormRopeWrite(self.kv, self.idx, hq, T, q_weight=self.w["q"], k_weight=self.w["k"],
                                     idx_q_weight=self.w["idx_q"], idx_k_weight=self.w["idx_k"], weight_offset=offset,
                                     eps=eps, rope_table=self.rope, rope_pairs=pairs, q_dtype=qt, idx_q_dtype=qt)

    def run(self):
        x = self.x
        return self.op.run(x["q"], x["k"], x["v"], x["idx_q"], x["idx_k"], self.pos.cuda(), self.slot.cuda())

    def want(self, name):
        x = bf16_to_f64(self.x[name].contiguous().view(torch.int16).cpu().numpy().view(np.uint16))
        w = self.w[name]
        w = None if w is None else bf16_to_f64(w.view(torch.int16).cpu().numpy().view(np.uint16))
        rope = None if self.rope is None else self.rope.cpu().numpy()
        return norm_rope(x, w, self.offset, self.eps, rope, self.rot, self.pairs, self.pos.numpy())


def _near(got, want, tol, what):
    bad = np.abs(got - want) > tol
    assert not bad.any(), (what, np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


def _check_queries(c, got, name):
    y, mag = c.want(name)
    if c.q8:
        v = E4M3[got.cpu().numpy()]
        y = np.clip(y, -448, 448)
        _near(v, y, np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10) + SLACK * mag, name)
    else:
        v = bf16_to_f64(got.view(torch.int16).cpu().numpy().view(np.uint16))
        _near(v, y, 2.0 ** -8 * np.abs(y) + SLACK * mag, name)


def _check_mx(row_bytes, y, mag, what):
    """One head's 64 + 4 bytes."""
    data, sc = row_bytes
    for g in range(4):
        s = slice(32 * g, 32 * g + 32)
        amax, slack = np.abs(y[s]).max(), SLACK * mag[s].max()
        lo, hi = max(amax - slack, 0), amax + slack
        e = [(-127 if a == 0 else int(np.clip(np.floor(np.log2(a)) - 2, -127, 127))) for a in (lo, hi)]
        assert int(sc[g]) - 127 in e, (what, g, sc[g], e)
        unit = 2.0 ** (int(sc[g]) - 127)
        z = np.clip(y[s] / unit, -6, 6)
        half = np.where(np.abs(z) < 2, 0.25, np.where(np.abs(z) < 4, 0.5, 1.0))
        _near(data[s] / unit, z, half + SLACK * mag[s] / unit, (what, g))


def _check_caches(c):
    raw, iraw = c.kv.buffer.cpu().numpy(), c.idx.buffer.cpu().numpy()
    k, kmag = c.want("k")
    ik, imag = c.want("idx_k")
    v = bf16_to_f64(c.x["v"].contiguous().view(torch.int16).cpu().numpy().view(np.uint16))
    size = {BF16: 32768, FP8: 16896, MX: 8704}[c.idxt]
    for t in range(c.T):
        s = int(c.slot[t])
        if s < 0:
            continue
        blk, o = divmod(s, 128)
        gk, gv = kv_token(raw, c.kvt, c.hkv, s)
        gi, gs = idx_token(iraw, c.idxt, c.hkv, s)
        for h in range(c.hkv):
            what = (t, h)
            if c.kvt == MX:
                for side, got, want, mag in ((0, gk, k, kmag), (1, gv, v, np.zeros_like(v))):
                    f = (blk * 2 * c.hkv + side * c.hkv + h) * 8704
                    _check_mx((got[h], raw[f + 8192 + 4 * o:f + 8196 + 4 * o]), want[t, h], mag[t, h], (what, side))
            elif c.kvt == FP8:
                zk, zv = np.clip(k[t, h] / np.float32(KS), -448, 448), np.clip(v[t, h] / np.float32(VS), -448, 448)
                half = lambda z: np.maximum(2.0 ** -4 * np.abs(z), 2.0 ** -10)  # noqa: E731
                _near(gk[h], zk, half(zk) + SLACK * (kmag[t, h] / KS + np.abs(zk)), (what, "k"))
                _near(gv[h], zv, half(zv) + SLACK * np.abs(zv), (what, "v"))
            else:
                _near(gk[h], k[t, h], 2.0 ** -8 * np.abs(k[t, h]) + SLACK * kmag[t, h], (what, "k"))
                assert np.array_equal(gv[h], v[t, h]), (what, "v")
            y, mag = ik[t, h], imag[t, h]
            if c.idxt == MX:
                f = (blk * c.hkv + h) * size
                _check_mx((gi[h], iraw[f + 8192 + 4 * o:f + 8196 + 4 * o]), y, mag, (what, "idx"))
            elif c.idxt == FP8:
                amax = np.abs(y).max()
                assert abs(gs[h] - (amax / 448 if amax else 1.0)) <= 2.0 ** -18 * max(mag.max() / 448, 2.0 ** -126), what
                z = y / gs[h]
                # amax / scale may exceed 448 by the scale's own error; the cast saturates
                _near(gi[h], np.clip(z, -448, 448), np.maximum(2.0 ** -4 * np.abs(z), 2.0 ** -10) + SLACK * (mag / gs[h] + np.abs(z)), (what, "idx"))
            else:
                _near(gi[h], y, 2.0 ** -8 * np.abs(y) + SLACK * mag, (what, "idx"))


@pytest.mark.parametrize("kv,idx", [(BF16, BF16), (FP8, FP8), (MX, MX), (FP8, MX), (MX, BF16)])
@pytest.mark.parametrize("T,hkv,group,rot,pairs,q8", [(1, 1, 4, 128, True, False), (7, 2, 8, 64, False, True),
                                                      (65, 1, 16, 96, False, False), (130, 4, 1, 16, True, True),
                                                      (33, 1, 2, 0, False, False), (40, 3, 3, 128, False, True)])
def test_queries_and_caches(kv, idx, T, hkv, group, rot, pairs, q8):
    c = Case(T, hkv, group, kv, idx, rot, pairs, q8, pads=3 if T > 8 else 0, seed=T + kv, offset=float(T % 2),
             fused=T != 65)
    q, iq = c.run()
    assert c.op.dev_err.item() == 0
    _check_queries(c, q, "q")
    _check_queries(c, iq, "idx_q")
    _check_caches(c)


def test_no_weights_and_long_batches():
    c = Case(1500, 2, 4, FP8, FP8, 64, weight=False, pads=20)
    q, iq = c.run()
    _check_queries(c, q, "q")
    _check_queries(c, iq, "idx_q")
    _check_caches(c)


def test_pad_rows_are_zero_and_store_nothing():
    c = Case(20, 1, 4, FP8, FP8, 64, pads=20)
    c.slot[3] = 5  # a pad row is not cached whatever its slot
    q, iq = c.run()
    assert not q.any() and not iq.any() and not c.kv.buffer.any() and not c.idx.buffer.any()


def test_a_slot_of_minus_one_with_a_position_is_normed_but_not_cached():
    c = Case(20, 1, 4, FP8, MX, 64)
    c.slot[:] = -1
    q, iq = c.run()
    _check_queries(c, q, "q")
    assert not c.kv.buffer.any() and not c.idx.buffer.any()


def test_positions_past_the_table_and_slots_past_the_cache_are_flagged():
    c = Case(9, 1, 4, MX, MX, 64)
    c.pos[2] = 5000
    q, _ = c.run()
    assert c.op.dev_err.item() == 64 and not q[2].any() and q[3].any()
    c = Case(9, 1, 4, MX, MX, 64)
    c.slot[4] = c.blocks * 128
    c.run()
    assert c.op.dev_err.item() == 16


def test_rows_of_zeros_and_large_rows():
    c = Case(6, 1, 2, MX, FP8, 64, eps=1e-6)
    for x in c.x.values():
        x[0] = 0
        x[1] *= 2.0 ** 40
        x[2] *= 2.0 ** -60
    q, iq = c.run()
    _check_queries(c, q, "q")
    _check_queries(c, iq, "idx_q")
    _check_caches(c)


def test_v_is_stored_as_the_page_writer_stores_it():
    from block_sparse_paged_score_gb300 import bsp
    for kv in (BF16, FP8, MX):
        c = Case(77, 2, 2, kv, BF16, 64)
        c.run()
        other = bsp.KvCache(kv, 2, c.blocks, KS, VS)
        v = c.x["v"].contiguous()
        bsp.kv_page_write(other, None, v, v, None, c.slot.cuda())
        slot = c.slot.cuda()
        assert torch.equal(bsp.kv_page_read(c.kv, None, slot)[1], bsp.kv_page_read(other, None, slot)[1])


def test_parts_alone_in_place_and_outside_their_buffers():
    """Queries alone, in place; rows behind the last token stay as they were."""
    import ctypes as C
    from block_sparse_paged_score_gb300 import bsp
    c = Case(11, 1, 4, FP8, FP8, 64, fused=False)
    want = c.run()[0].clone()
    q = torch.cat([c.x["q"], torch.full_like(c.x["q"], 3.0)])
    a = bsp.NormRopeArgs()
    C.memmove(C.byref(a), C.byref(c.op.args), C.sizeof(a))
    a.q = a.q_out = q.data_ptr()
    a.q_stride = 4 * 128
    for f in ("k", "v", "idx_q", "idx_k", "idx_q_out", "slot"):
        setattr(a, f, None)
    a.kv = a.idx = None
    pos = c.pos.cuda()
    a.positions = pos.data_ptr()
    bsp.norm_rope_write(a)
    torch.cuda.synchronize()
    assert torch.equal(q[:11], want) and (q[11:] == 3).all()


def test_captured_and_replayed_on_another_stream():
    c = Case(64, 1, 16, MX, MX, 64, q8=True)
    x, pos, slot = c.x, c.pos.cuda(), c.slot.cuda()
    args = (x["q"], x["k"], x["v"], x["idx_q"], x["idx_k"], pos, slot)
    q, iq = (t.clone() for t in c.op.run(*args))
    kept = c.kv.buffer.clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = c.op.run(*args)
    c.kv.buffer.zero_()
    out[0].zero_()
    with torch.cuda.stream(s):
        s.wait_stream(torch.cuda.default_stream())
        g.replay()
    s.synchronize()
    assert torch.equal(out[0], q) and torch.equal(out[1], iq) and torch.equal(c.kv.buffer, kept)


@pytest.mark.parametrize("kv,idx", [(BF16, BF16), (FP8, FP8), (MX, MX)])
@pytest.mark.parametrize("hkv,group,rot,pairs,q8", [(1, 3, 64, False, True), (3, 1, 128, True, False)])
def test_batches_long_enough_for_a_half_warp_a_token(kv, idx, hkv, group, rot, pairs, q8):
    c = Case(3801, hkv, group, kv, idx, rot, pairs, q8, pads=9, seed=kv)
    q, iq = c.run()
    assert c.op.dev_err.item() == 0
    _check_queries(c, q, "q")
    _check_queries(c, iq, "idx_q")
    _check_caches(c)


def test_the_same_row_in_a_short_and_a_long_batch():
    """Both kernels round alike: a long batch's rows are bit for bit those of its parts."""
    c = Case(4000, 1, 4, MX, FP8, 64, q8=True, seed=31)
    q, iq = (t.clone() for t in c.run())
    kv, idx = c.kv.buffer.clone(), c.idx.buffer.clone()
    c.kv.buffer.zero_(), c.idx.buffer.zero_()
    x, pos, slot = c.x, c.pos.cuda(), c.slot.cuda()
    for a in range(0, 4000, 700):
        s = slice(a, min(a + 700, 4000))
        got = c.op.run(x["q"][s], x["k"][s], x["v"][s], x["idx_q"][s], x["idx_k"][s], pos[s], slot[s])
        assert torch.equal(got[0], q[s]) and torch.equal(got[1], iq[s])
    assert torch.equal(c.kv.buffer, kv) and torch.equal(c.idx.buffer, idx)


@pytest.mark.parametrize("T", [30, 4100])
def test_without_a_kv_cache_without_an_index_cache_and_keys_as_rows(T):
    from block_sparse_paged_score_gb300 import step
    c = Case(T, 2, 2, FP8, MX, 64, seed=T)
    q, iq = (t.clone() for t in c.run())
    x, pos, slot = c.x, c.pos.cuda(), c.slot.cuda()
    kv, idx = c.kv.buffer.clone(), c.idx.buffer.clone()
    w = dict(q_weight=c.w["q"], k_weight=c.w["k"], idx_q_weight=c.w["idx_q"], idx_k_weight=c.w["idx_k"],
             rope_table=c.rope)
    c.kv.buffer.zero_(), c.idx.buffer.zero_()
    a = step.NormRopeWrite(None, c.idx, c.hq, T, **w)
    got = a.run(x["q"], None, None, x["idx_q"], x["idx_k"], pos, slot)
    assert torch.equal(got[0], q) and torch.equal(got[1], iq)
    assert not c.kv.buffer.any() and torch.equal(c.idx.buffer, idx)
    c.idx.buffer.zero_()
    b = step.NormRopeWrite(c.kv, None, c.hq, T, **w)
    k_out = torch.full((T + 1, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    b.args.k_out = k_out.data_ptr()
    got = b.run(x["q"], x["k"], x["v"], None, None, pos, slot)
    assert torch.equal(got[0], q) and got[1] is None
    assert torch.equal(c.kv.buffer, kv) and not c.idx.buffer.any()
    y, mag = c.want("k")
    _near(bf16_to_f64(k_out[:T].view(torch.int16).cpu().numpy().view(np.uint16)), y, 2.0 ** -8 * np.abs(y) + SLACK * mag, "k")
    assert (k_out[T:] == 7).all()


def test_no_tokens():
    c = Case(5, 1, 4, MX, FP8, 64)
    x, pos, slot = c.x, c.pos.cuda(), c.slot.cuda()
    q, iq = c.op.run(x["q"][:0], x["k"][:0], x["v"][:0], x["idx_q"][:0], x["idx_k"][:0], pos[:0], slot[:0])
    assert q.shape == (0, 4, 128) and iq.shape == (0, 1, 128)
    assert not c.kv.buffer.any() and not c.idx.buffer.any()
