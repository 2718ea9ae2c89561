"""bsp_dense_pa_decode against softmax(scale q K^T) V in 64 bits.

Tolerance.  With a = sum p |v| / sum p of an output element: a softmax weight
is rounded to at most 2^-11 relative (f16; in two bf16 parts, 2^-17, where V's
scales are beyond f16, and V's values are exact either way), a logit is off by at most
e = 2^-18 * scale * sum |q k| (fp32 sums of at most 512 exact products, and
the split of a bf16 query into two e4m3 parts, 2^-18 of its row's largest
value), which moves a weight and the sum by e each, and the exponentials, the
sums and the merges add less than 2^-13.  Together under (2^-11 + 2^-13 + 2 e) a,
and the bf16 output adds half a step, 2^-8 |o|.  Below the range of f16 a weight
is off by an absolute 2^-25, where the row's largest is at least 2^7: at most
2^-32 of the largest weight, times a value of at most 6 * 2^(the largest scale
of its 32 dims) = top, for each of n tokens; exponentials below 2^-126 and
outputs below bf16's normal range are less than that: n 2^-32 top + 2^-133."""
import math

import numpy as np
import pytest
import torch

from plain64 import E4M3, MX, bf16_to_f64, dense_attention, mx_field

pytestmark = pytest.mark.gpu
SCALE = 1 / math.sqrt(128)


class Case:
    def __init__(self, lens, hkv=1, group=16, q_len=1, q8=True, seed=0, spread=2, q_scale=1.0, width=None, pad_bytes=0):
        from block_sparse_paged_score_gb300 import bsp
        r = np.random.default_rng(seed)
        n = len(lens)
        self.lens, self.hkv, self.group, self.q_len, self.q8 = lens, hkv, group, q_len, q8
        width = width or max(1, max(-(-x // 128) for x in lens))
        self.blocks = n * width + 1
        self.stride = 2 * hkv * 8704 + pad_bytes
        raw = r.integers(0, 256, self.blocks * self.stride, dtype=np.uint8)
        f = raw.reshape(self.blocks, self.stride)[:, :2 * hkv * 8704].reshape(self.blocks, 2 * hkv, 8704)
        f[:, :, 8192:] = 126 + r.integers(-spread, spread + 1, (self.blocks, 2 * hkv, 512))
        self.raw, self.fields = raw, f
        self.table = r.permutation(self.blocks)[:n * width].reshape(n, width).astype(np.int32)
        tokens = n * q_len
        q = (r.standard_normal((tokens, hkv * group, 128)) * q_scale).astype(np.float32)
        qt = torch.from_numpy(q)
        self.q_t = qt.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if q8 else qt.bfloat16()
        self.q = E4M3[self.q_t.numpy()] if q8 else bf16_to_f64(self.q_t.view(torch.int16).numpy().view(np.uint16))
        self.row_len = np.array([max(0, lens[s] - (q_len - 1 - j)) for s in range(n) for j in range(q_len)
                                 for _ in range(hkv)], np.int32)
        self.row_seq = np.repeat(np.arange(n), q_len * hkv).astype(np.int32)
        self.bsp = bsp

    def device(self):
        c = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        self.buf = c(self.raw)
        kv = self.bsp.KvCache(MX, self.hkv, self.blocks if self.stride == 2 * self.hkv * 8704 else 1, buffer=self.buf)
        kv.desc.id_stride_bytes, kv.desc.num_blocks = self.stride, self.blocks
        self.kv, self.dq, self.dtable = kv, self.q_t.cuda(), c(self.table)
        self.dseq, self.dlen = c(self.row_seq), c(self.row_len)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        return self

    def call(self, out=None, ws=None, stream=None):
        b = self.bsp
        return b.dense_pa_decode(self.kv, self.dq, b.FP8_E4M3 if self.q8 else b.BF16, self.hkv * self.group, self.dtable,
                                 self.dseq, self.dlen, self.q_len, out=out, ws=ws, dev_err=self.err, stream=stream)

    def want(self):
        o, a = dense_attention(lambda b, side, h: mx_field(self.fields[b, side * self.hkv + h]), self.table, self.q,
                               self.row_seq, self.row_len, self.hkv, self.group, SCALE)
        return o, a

    def logit_slack(self):
        top = 2.0 ** (self.fields[:, :self.hkv, 8192:].max() - 127.0)
        return 2.0 ** -18 * SCALE * np.abs(self.q).sum(-1).max() * 6 * top

    def floor(self, r):
        """n 2^-32 top + 2^-133 of row r: [128]"""
        s, h, n = int(self.row_seq[r]), r % self.hkv, int(min(self.row_len[r], 128 * self.table.shape[1]))
        ids = [b for b in self.table[s, :-(-n // 128)] if 0 <= b < self.blocks]
        if not ids:
            return np.zeros(128)
        sc = self.fields[ids, self.hkv + h, 8192:].reshape(-1, 4)[:n].astype(np.float64)
        return n * 2.0 ** -32 * 6 * np.repeat(2.0 ** (sc.max(0) - 127), 32) + 2.0 ** -133

    def check(self, got):
        o, a = self.want()
        g = bf16_to_f64(got.view(torch.int16).cpu().numpy().view(np.uint16))
        tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 2.0 ** -13 + 2 * self.logit_slack()) * a
        for r in range(len(self.row_len)):
            t, h = divmod(r, self.hkv)
            tol[t, h * self.group:(h + 1) * self.group] += self.floor(r)
        bad = ~(np.abs(g - o) <= tol)
        assert not bad.any(), (np.argwhere(bad)[:5], g[bad][:5], o[bad][:5], tol[bad][:5], bad.sum())


def _close(c):
    c.device()
    out = c.call()
    torch.cuda.synchronize()
    assert c.err.item() == 0
    c.check(out)
    return out


EDGES = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 300, 383, 385, 500]


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("group", [1, 2, 4, 8, 16])
def test_lengths_around_every_tile(group, q8):
    _close(Case(EDGES, group=group, q8=q8, seed=group))


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("q_len", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("hkv,group", [(1, 16), (2, 8), (4, 2), (3, 1)])
def test_query_groups(hkv, group, q_len, q8):
    _close(Case([3, 40, 129, 700, 8], hkv, group, q_len, q8, seed=q_len))


@pytest.mark.parametrize("lens", [[0], [0, 0, 0], [0, 5, 0, 1300, 0], [1]])
def test_rows_that_see_nothing_are_zero(lens):
    c = Case(lens, q_len=4, width=11)
    out = _close(c)
    for s, n in enumerate(lens):
        if n == 0:
            assert not out[4 * s:4 * s + 4].any()


@pytest.mark.parametrize("n,length", [(1, 1000), (1, 20000), (2, 40001), (7, 3000), (150, 200), (700, 40), (1300, 3)])
def test_batches_from_one_sequence_to_more_than_the_grid(n, length):
    r = np.random.default_rng(n)
    lens = [int(x) for x in r.integers(max(1, length // 2), length + 1, n)]
    lens[0] = length
    _close(Case(lens, group=4, q8=True, seed=n))


@pytest.mark.parametrize("q_len,q8", [(1, True), (4, True), (8, False), (2, False)])
def test_long_and_short_sequences_side_by_side(q_len, q8):
    _close(Case([30000, 1, 900, 128, 0, 5000, 2, 129], q_len=q_len, q8=q8, seed=5))


def test_more_key_heads():
    _close(Case([1500, 700, 64], hkv=4, group=16, q_len=2, seed=3))


@pytest.mark.parametrize("q8", [True, False])
def test_sharp_and_flat_logits(q8):
    _close(Case([2000, 37, 515], seed=6, q_scale=16.0, q8=q8))
    _close(Case([2000, 37, 515], seed=7, q_scale=1e-3 if not q8 else 0.05, q8=q8))


def test_constant_values_come_back():
    """Weights sum to one: V of one value everywhere gives that value."""
    c = Case([5000, 3, 129], seed=8)
    c.fields[:, c.hkv:, :8192] = 0x55  # 3.0
    c.fields[:, c.hkv:, 8192:] = 127
    out = _close(c)
    assert (out.float() - 3).abs().max() <= 3 * 2.0 ** -8


@pytest.mark.parametrize("spread", [10, 30, 60])
@pytest.mark.parametrize("q_len", [1, 4])
def test_scales_of_wide_range_in_v(spread, q_len):
    """V scales from 2^-spread to 2^spread beside one another; K's are ordinary."""
    c = Case([700, 128, 31, 3001], q_len=q_len, seed=spread)
    r = np.random.default_rng(spread)
    c.fields[:, c.hkv:, 8192:] = 127 + r.integers(-spread, spread + 1, c.fields[:, c.hkv:, 8192:].shape)
    _close(c)


def test_scales_that_grow_and_fall_along_the_context():
    c = Case([4000, 4000], seed=2)
    for s in range(2):
        for i, b in enumerate(c.table[s]):
            e = 100 + 2 * i if s == 0 else 160 - 2 * i
            c.fields[b, 1, 8192:] = e
    _close(c)


def test_groups_of_zeros_have_the_smallest_scale():
    c = Case([900, 300], seed=4)
    z = np.random.default_rng(1).random((c.blocks, 2, 128, 4)) < 0.3
    f = c.fields
    data = f[:, :, :8192].reshape(c.blocks, 2, 128, 4, 16)
    data[z] = 0
    f[:, :, :8192] = data.reshape(c.blocks, 2, 8192)
    sc = f[:, :, 8192:].reshape(c.blocks, 2, 128, 4)
    sc[z] = 0
    f[:, :, 8192:] = sc.reshape(c.blocks, 2, 512)
    _close(c)


@pytest.mark.parametrize("q_len", [1, 4])
def test_bytes_past_the_length_are_never_used(q_len):
    """NaN scales and the widest ones in every place at or past a row's length."""
    lens = [1, 77, 128, 200, 1025, 31]
    c = Case(lens, q_len=q_len, seed=9)
    want = _close(c).clone()
    f = c.fields
    for s, n in enumerate(lens):
        for i, b in enumerate(c.table[s]):
            lo = max(0, min(128, n - 128 * i))
            d = f[b].reshape(2, 8704)
            d[:, 64 * lo:8192] = 0x7F
            d[:, 8192 + 4 * lo:] = 255
    c.device()
    assert torch.equal(c.call(), want)


def test_a_table_wider_than_the_contexts_and_a_padded_cache():
    c = Case([300, 5, 777], seed=10, width=40, pad_bytes=96)
    want = _close(c).clone()
    for s, n in enumerate(c.lens):  # entries past a context are never read
        c.table[s, -(-n // 128):] = -1 if s else 1 << 30
    c.device()
    assert torch.equal(c.call(), want) and c.err.item() == 0


def test_lengths_past_the_table_are_clamped():
    c = Case([256, 100], seed=11, width=2)
    want = _close(c).clone()
    c.row_len[0] = 2 ** 31 - 1
    c.device()
    assert torch.equal(c.call(), want) and c.err.item() == 0


def test_bad_block_ids_are_flagged_and_left_out():
    c = Case([1000, 600, 300], seed=12, q_len=2)
    c.table[0, 3], c.table[1, 1], c.table[1, 4] = c.blocks, -1, 2 ** 31 - 1
    c.device()
    got = c.call()
    assert c.err.item() == 2
    keep = lambda b, side, h: mx_field(c.fields[b, side])  # noqa: E731
    # the same rows with the bad blocks' tokens taken out
    for s in range(2):
        ids = [int(b) for b in c.table[s] if 0 <= b < c.blocks]
        for j in range(2):
            row = 2 * s + j
            n = int(c.row_len[row])
            toks = [(b, t) for i, b in enumerate(c.table[s]) for t in range(128) if i * 128 + t < n and b in ids]
            k = np.stack([keep(b, 0, 0)[t] for b, t in toks])
            v = np.stack([keep(b, 1, 0)[t] for b, t in toks])
            z = c.q[row] @ k.T * SCALE
            p = np.exp(z - z.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            g = bf16_to_f64(got[row].view(torch.int16).cpu().numpy().view(np.uint16))
            o, a = p @ v, p @ np.abs(v)
            assert (np.abs(g - o) <= 2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 2.0 ** -13 + 2 * c.logit_slack()) * a + c.floor(row)).all()


def test_a_row_that_names_another_sequence_is_flagged():
    c = Case([300, 400], q_len=2)
    c.row_seq[1] = 1
    c.device()
    out = c.call()
    torch.cuda.synchronize()
    assert c.err.item() == 4
    c.row_seq[1] = 0  # computed with the first row's sequence
    c.check(out)


def test_a_last_group_of_fewer_tokens():
    c = Case([500, 900], q_len=4, seed=13)
    c.device()
    want = c.call().clone()
    c.dq, c.dseq, c.dlen = c.dq[:6], c.dseq[:6], c.dlen[:6]
    assert torch.equal(c.call(), want[:6])


def test_same_bits_again_rows_behind_untouched_and_dirty_workspaces():
    c = Case([30000, 1, 900, 12000], q_len=2, seed=14).device()
    rows = len(c.row_len)
    ws = c.bsp.dense_pa_workspace(rows, 1, 16, 2)
    out = torch.full((rows + 3, 16, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    ws.fill_(0xFF)  # NaN, and counts of -1
    first = c.call(out=out, ws=ws).clone()
    assert (first[rows:] == 9).all()
    for fill in (0, 0x3C):
        ws.fill_(fill)
        out.fill_(9.0)
        assert torch.equal(c.call(out=out, ws=ws), first)
    c.check(first[:rows])


def test_two_streams_and_a_replayed_capture():
    a, b = Case([20000, 300], q_len=1, seed=15).device(), Case([9000, 40, 7000], q_len=3, seed=16).device()
    wa, wb = a.call().clone(), b.call().clone()
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    out_a, out_b = torch.zeros_like(wa), torch.zeros_like(wb)
    wsa = a.bsp.dense_pa_workspace(2, 1, 16, 1)
    wsb = b.bsp.dense_pa_workspace(9, 1, 16, 3)
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga, stream=sa):
        a.call(out=out_a, ws=wsa)
    with torch.cuda.graph(gb, stream=sb):
        b.call(out=out_b, ws=wsb)
    for _ in range(20):
        with torch.cuda.stream(sa):
            ga.replay()
        with torch.cuda.stream(sb):
            gb.replay()
    torch.cuda.synchronize()
    assert torch.equal(out_a, wa) and torch.equal(out_b, wb)
    # a captured call serves other lengths
    a.row_len[:] = [777, 0]
    a.dlen.copy_(torch.from_numpy(a.row_len))
    torch.cuda.synchronize()
    with torch.cuda.stream(sa):
        ga.replay()
    sa.synchronize()
    a.check(out_a)


def test_offsets_past_32_bits():
    """Blocks at the far end of a cache of more than 4 GiB."""
    blocks = (1 << 32) // (2 * 8704) + 40
    c = Case([700, 90], seed=17)
    c.device()
    big = torch.empty(blocks * 2 * 8704, dtype=torch.uint8, device="cuda")
    n = c.blocks
    big[(blocks - n) * 2 * 8704:] = c.buf
    c.kv = c.bsp.KvCache(MX, 1, blocks, buffer=big)
    c.dtable = c.dtable + (blocks - n)
    out = c.call()
    torch.cuda.synchronize()
    assert c.err.item() == 0
    c.check(out)


def _tolerance(c, o, a):
    tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 2.0 ** -13 + 2 * c.logit_slack()) * a
    for r in range(len(c.row_len)):
        t, h = divmod(r, c.hkv)
        tol[t, h * c.group:(h + 1) * c.group] += c.floor(r)
    return tol


def _f64(out):
    return bf16_to_f64(out.view(torch.int16).cpu().numpy().view(np.uint16))


@pytest.mark.parametrize("byte", [9, 40, 109, 110, 134, 135, 180])
@pytest.mark.parametrize("q_len", [1, 2, 4])
def test_one_scale_in_v(byte, q_len):
    """On both sides of what f16 holds (bytes 110 to 134)."""
    c = Case([900, 70], q_len=q_len, seed=byte)
    c.fields[:, c.hkv:, 8192:] = byte
    _close(c)


@pytest.mark.parametrize("q_len,group", [(1, 16), (2, 16), (4, 16), (8, 16), (3, 4)])
@pytest.mark.parametrize("q8", [True, False])
def test_logits_that_grow_along_the_context(q_len, group, q8):
    """Every few blocks some row's maximum passes its reference."""
    c = Case([2500, 1800, 400], group=group, q_len=q_len, q8=q8, seed=21)
    for s in range(3):
        for i, b in enumerate(c.table[s]):
            c.fields[b, 0, 8192:] = 118 + min(i, 12)
    _close(c)


@pytest.mark.parametrize("side", [0, 1])
def test_a_nan_reaches_only_the_rows_that_see_it(side):
    """A scale byte of 255 in K (the whole row) or in one group of V, in the last
    two tokens of four rows of growing length."""
    lens = [130, 700, 3]
    c = Case(lens, q_len=4, seed=22)
    o, a = c.want()
    tol = _tolerance(c, o, a)
    for s, n in enumerate(lens):
        for t in (n - 1, n - 2):
            c.fields[c.table[s, t // 128], side, 8192 + 4 * (t % 128) + 1] = 255
    c.device()
    g = _f64(c.call())
    for s in range(3):
        for j in range(4):
            r = 4 * s + j
            hit = j >= 2  # row j sees tokens below n - 3 + j
            dims = np.zeros(128, bool)
            if hit:
                dims[slice(None) if side == 0 else slice(32, 64)] = True
            assert np.isnan(g[r][:, dims]).all(), (s, j)
            assert (np.abs(g[r] - o[r]) <= tol[r])[:, ~dims].all(), (s, j)


@pytest.mark.parametrize("scale", [-0.07, 0.0, 0.3])
def test_other_logit_scales(scale):
    c = Case([700, 129, 4000], q_len=2, seed=23).device()
    b = c.bsp
    got = _f64(b.dense_pa_decode(c.kv, c.dq, b.FP8_E4M3, 16, c.dtable, c.dseq, c.dlen, 2, sm_scale=scale))
    o, a = dense_attention(lambda blk, side, h: mx_field(c.fields[blk, side * c.hkv + h]), c.table, c.q, c.row_seq,
                           c.row_len, c.hkv, c.group, scale)
    tol = _tolerance(c, o, a) + 2 * (abs(scale) / SCALE) * c.logit_slack() * a
    assert (np.abs(got - o) <= tol).all()


def test_calls_of_other_sizes_in_one_workspace_one_after_another():
    cases = [Case([9000, 40], q_len=4, seed=24).device(), Case([300, 12000, 5], q_len=1, seed=25).device(),
             Case([5000], q_len=2, group=8, q8=False, seed=26).device()]
    ws = torch.empty(max(c.bsp.dense_pa_workspace_bytes(len(c.row_len), 1, c.group, c.q_len) for c in cases),
                     dtype=torch.uint8, device="cuda")
    want = [c.call().clone() for c in cases]
    for _ in range(3):
        for c, w in zip(cases, want):
            assert torch.equal(c.call(ws=ws), w)


def test_no_rows():
    c = Case([300], seed=27).device()
    c.dq, c.dseq, c.dlen = c.dq[:0], c.dseq[:0], c.dlen[:0]
    assert c.call().shape == (0, 16, 128) and c.err.item() == 0


def test_many_short_requests():
    """More units than CTAs, and groups than a CTA has threads."""
    r = np.random.default_rng(28)
    _close(Case([int(x) for x in r.integers(0, 400, 1500)], group=16, seed=28))
    _close(Case([int(x) for x in r.integers(0, 300, 700)], group=8, q_len=4, seed=29))


def test_a_cache_of_no_blocks():
    c = Case([300, 0], q_len=2, seed=30).device()
    c.kv.desc.num_blocks = 0
    assert not c.call().any() and c.err.item() == 2
