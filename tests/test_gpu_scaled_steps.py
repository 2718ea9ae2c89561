"""A layer without an indexer over a block-scaled 8-bit cache, run as a serving
loop would: new prompts, chunks over their contexts, decode tokens, each step
against the same in 64 bits from the rows it was given and the bytes that the
cache held.  Tolerances as in the tests of the single operators: bytes and
scales are equal bit for bit from the step's own bf16 rows, the attentions
within their weights' roundings."""
import numpy as np
import pytest
import torch

import plain64_scaled as P
from plain64 import E4M3, dense_attention, norm_rope

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5
HKV, GROUP, N, NB, BT = 2, 4, 5, 64, 12


class Layer:
    def __init__(self, seed):
        from block_sparse_paged_score_gb300 import bsp, step
        self.g = torch.Generator().manual_seed(seed)
        self.cache = bsp.BlockScaledKvCache(HKV, NB)
        self.w = {k: (1 + 0.1 * torch.randn(128, generator=self.g)).bfloat16().cuda() for k in ("q_weight", "k_weight")}
        self.rope = step.rope_table(2000, 64, 1e5)
        self.free = torch.randperm(NB, generator=self.g).int().cuda()
        self.head = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ctx = torch.zeros(N, dtype=torch.int32, device="cuda")
        self.table = torch.full((N, BT), -1, dtype=torch.int32, device="cuda")
        self.norm = dict(rope_table=self.rope, block_table=self.table, **self.w)

    def rows(self, T):
        """q, k, v as the parts of one projection's rows"""
        x = torch.randn(T, (GROUP + 2) * HKV, 128, generator=self.g).bfloat16().cuda()
        return x.split([GROUP * HKV, HKV, HKV], 1)

    def bytes(self):
        return self.cache.buffer.cpu().numpy(), [self.cache.k_scales.cpu().numpy(), self.cache.v_scales.cpu().numpy()]

    def step(self, st, new, x, contexts=True, stream=None):
        """one step, its norms and its write checked; (output, lengths, offsets)"""
        cache, scales = self.bytes()
        new_d = torch.tensor(new, dtype=torch.int32, device="cuda")
        out = st.run(self.ctx if contexts else None, new_d, self.free, self.head, *x, stream=stream)
        torch.cuda.synchronize()
        t = st.tables
        assert st.dev_err.item() == 0
        T = x[0].shape[0]
        pos = t.query_abs_pos.cpu().numpy()[:T]
        k_out = P.bits_f64(st.norm.k_out[:T])
        y, _ = norm_rope(P.bits_f64(x[1]), P.bits_f64(self.w["k_weight"]), 0.0, 1e-6, self.rope.cpu().numpy(), 64, False, pos)
        assert np.abs(k_out - y).max() <= 2.0 ** -8 * np.abs(y).max() * 1.01
        P.scaled_write(cache, scales, HKV, k_out, P.bits_f64(x[2]), t.slot.cpu().numpy()[:T], NB)
        got, got_s = self.bytes()
        assert np.array_equal(got, cache) and all(np.array_equal(a, b) for a, b in zip(got_s, scales))
        self.ctx, self.head = t.seq_lens.clone(), self.head + t.blocks_taken
        return out, t.seq_lens.cpu().numpy(), t.cu_tokens.cpu().numpy()

    def tokens(self, lens):
        """K and V of the first lens[s] tokens of each request, from the cache's bytes"""
        cache, scales = self.bytes()
        table = self.table.cpu().numpy()
        kv = []
        for side in (0, 1):
            seqs = []
            for s, n in enumerate(lens):
                b = [np.stack([P.block_values(cache, scales, HKV, table[s, i], h, side) for h in range(HKV)], 1)
                     for i in range(-(-n // 128))]
                seqs.append(np.concatenate(b + [np.zeros((0, HKV, 128))])[:n])
            kv.append(np.concatenate(seqs))
        return kv


def near(got, o, a, weight, extra=0.0):
    tol = (weight + extra) * a + 2.0 ** -8 * np.abs(o) + 1e-30
    bad = ~(np.abs(got - o) <= tol) & ~np.isnan(a)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], o[bad][:4])


@pytest.mark.parametrize("side_stream", [False, True])
def test_prompts_chunks_and_decode_tokens(side_stream):
    from block_sparse_paged_score_gb300 import bsp, step
    la = Layer(4)
    hq = HKV * GROUP
    stream = torch.cuda.Stream() if side_stream else None
    torch.cuda.synchronize()
    first = step.ScaledPromptStep(la.cache, hq, N, 900, BT, **la.norm)
    chunk = step.ScaledPromptStep(la.cache, hq, N, 700, BT, key_capacity=2200, **la.norm)
    decode = {ql: step.ScaledDecodeStep(la.cache, hq, N, ql, BT, q_dtype=qt, **la.norm)
              for ql, qt in ((1, bsp.FP8_E4M3), (3, bsp.BF16))}
    torch.cuda.synchronize()  # (made on this stream, used on another)

    # new prompts, one of a token, one of none yet, and three pad rows
    new = [300, 1, 0, 128, 257]
    x = la.rows(sum(new) + 3)
    out, lens, cu = la.step(first, new, x, contexts=False, stream=stream)
    q, k = P.bits_f64(first.norm.q_out[:len(x[0])]), P.bits_f64(first.norm.k_out[:len(x[0])])
    o, a = P.prompt(q, k, P.bits_f64(x[2]), cu, cu, SCALE)
    near(P.bits_f64(out), o, a, 2.0 ** -8, 2.0 ** -11)

    # chunks over them: the empty request begins, one sits out
    new = [100, 250, 33, 0, 300]
    x = la.rows(sum(new))
    out, lens, cu = la.step(chunk, new, x, stream=stream)
    seen = np.where(np.array(new) > 0, lens, 0)
    k, v = la.tokens(seen)
    k, v = [P.bits_f64(torch.from_numpy(t).float().bfloat16()) for t in (k, v)]  # as read back
    o, a = P.prompt(P.bits_f64(chunk.norm.q_out[:len(x[0])]), k, v, cu, np.cumsum([0, *seen]), SCALE)
    near(P.bits_f64(out), o, a, 2.0 ** -8, 2.0 ** -11)

    # decode tokens, of several lengths and types, one request sitting out each time
    for i in range(8):
        ql = (1, 3)[i % 2]
        st = decode[ql]
        new = [ql] * N
        new[i % N] = 0
        x = la.rows(N * ql)
        out, lens, cu = la.step(st, new, x, stream=stream)
        assert not out[(N - 1) * ql:].any()
        q = E4M3[st.norm.q_out.cpu().numpy()] if ql == 1 else P.bits_f64(st.norm.q_out)
        cache, scales = la.bytes()
        req, pos = st.tables.query_req_id.cpu().numpy(), st.tables.query_abs_pos.cpu().numpy()
        o, a = dense_attention(lambda b, side, h: P.block_values(cache, scales, HKV, b, h, side), la.table.cpu().numpy(),
                               q, np.repeat(req, HKV), np.repeat(pos + 1, HKV), HKV, GROUP, SCALE)
        near(P.bits_f64(out), o, a, 2.0 ** -11, 2.0 ** -10)


def test_steps_captured_and_replayed():
    """A chunk and a decode step captured once and replayed with new lengths in the
    same buffers give what eager steps give."""
    from block_sparse_paged_score_gb300 import step
    outs = []
    for captured in (False, True):
        la = Layer(9)
        hq = HKV * GROUP
        chunk = step.ScaledPromptStep(la.cache, hq, N, 400, BT, key_capacity=1500, **la.norm)
        dec = step.ScaledDecodeStep(la.cache, hq, N, 2, BT, **la.norm)
        new = torch.zeros(N, dtype=torch.int32, device="cuda")
        xc, xd = [t.clone() for t in la.rows(400)], [t.clone() for t in la.rows(2 * N)]
        got, graphs = [], {}
        for i, lens in enumerate(([90, 0, 100, 1, 30], [2] * N, [100, 129, 0, 7, 64], [2] * N, [2, 0, 2, 2, 2])):
            st, x = (dec, xd) if max(lens) <= 2 else (chunk, xc)
            new.copy_(torch.tensor(lens, dtype=torch.int32))
            for t in x:
                t.copy_(torch.randn(t.shape, generator=la.g))
            if captured and st not in graphs:
                kept = [t.clone() for t in (la.cache.buffer, la.cache.k_scales, la.cache.v_scales, la.table)]
                st.run(la.ctx, new, la.free, la.head, *x)  # (loads the kernels)
                graphs[st] = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graphs[st]):
                    st.run(la.ctx, new, la.free, la.head, *x)
                for t, old in zip((la.cache.buffer, la.cache.k_scales, la.cache.v_scales, la.table), kept):
                    t.copy_(old)
            graphs[st].replay() if captured else st.run(la.ctx, new, la.free, la.head, *x)
            la.ctx.copy_(st.tables.seq_lens)
            la.head += st.tables.blocks_taken
            assert st.dev_err.item() == 0
            got.append((st.out[:st.tables.cu_tokens[-1]].clone(), la.cache.buffer.clone(), la.cache.k_scales.clone()))
        outs.append(got)
    for a, b in zip(*outs):
        assert all(torch.equal(s.view(torch.uint8), t.view(torch.uint8)) for s, t in zip(a, b))


def test_key_capacity_and_free_blocks_that_run_out_show_in_the_error_word():
    from block_sparse_paged_score_gb300 import step
    la = Layer(2)
    st = step.ScaledPromptStep(la.cache, HKV * GROUP, N, 400, BT, key_capacity=350, **la.norm)
    new = torch.tensor([300, 50, 0, 0, 0], dtype=torch.int32, device="cuda")
    st.run(la.ctx, new, la.free, la.head, *la.rows(350))
    assert st.dev_err.item() == 0
    st.run(st.tables.seq_lens.clone(), new, la.free, st.tables.blocks_taken.clone(), *la.rows(350))
    assert st.dev_err.item() == 32  # the keys do not fit: cut
    with pytest.raises(ValueError, match="contexts"):
        st.run(None, new, la.free, la.head, *la.rows(350))
