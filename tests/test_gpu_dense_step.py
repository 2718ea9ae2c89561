"""The operators in a run: tables -> norm, rotation and write -> row lengths ->
dense attention over several steps of a small batch, against the same in 64
bits from the bytes the cache holds; and the same tables, norms and writes in
front of the indexer's score -> select -> attend."""
import math

import numpy as np
import pytest
import torch

from plain64 import FP8, MX, bf16_to_f64, dense_attention, mx_field, norm_rope

pytestmark = pytest.mark.gpu


def test_steps_of_a_dense_layer():
    from block_sparse_paged_score_gb300 import bsp, step
    hkv, group, n, ql, nb = 2, 4, 5, 3, 64
    g = torch.Generator().manual_seed(3)
    kv = bsp.KvCache(MX, hkv, nb)
    w = {k: (1 + 0.1 * torch.randn(128, generator=g)).bfloat16().cuda() for k in ("q_weight", "k_weight")}
    rope = step.rope_table(2000, 64, 1e5)
    st = step.DenseStep(kv, hkv * group, n, ql, 8, q_dtype=bsp.BF16, rope_table=rope, **w)
    free = torch.randperm(nb, generator=g).int().cuda()
    head = torch.zeros(1, dtype=torch.int32, device="cuda")
    ctx = torch.zeros(n, dtype=torch.int32, device="cuda")
    for i in range(60):
        # a request that sits out, in turn; the others bring ql tokens
        new = torch.full((n,), ql, dtype=torch.int32)
        new[i % n] = 0
        x = [torch.randn(n * ql, h, 128, generator=g).bfloat16().cuda() for h in (hkv * group, hkv, hkv)]
        before = kv.buffer.clone()
        out = st.run(ctx, new.cuda(), free, head, *x)
        t = st.tables
        ctx, head = t.seq_lens.clone(), head + t.blocks_taken
        live = (n - 1) * ql
        assert not out[live:].any() and st.norm.dev_err.item() == 0 and t.dev_err.item() == 0
        if i % 19:
            continue
        # the attention from the cache's own bytes
        f = kv.buffer.cpu().numpy().reshape(nb, 2 * hkv, 8704)
        pos, req = t.query_abs_pos.cpu().numpy(), t.query_req_id.cpu().numpy()
        q = bf16_to_f64(x[0].view(torch.int16).cpu().numpy().view(np.uint16))
        qw = bf16_to_f64(w["q_weight"].view(torch.int16).cpu().numpy().view(np.uint16))
        y, _ = norm_rope(q, qw, 0.0, 1e-6, rope.cpu().numpy(), 64, False, pos)
        got_q = bf16_to_f64(st.norm.q_out.view(torch.int16).cpu().numpy().view(np.uint16))
        assert np.abs(got_q - y).max() <= 2.0 ** -8 * np.abs(y).max() * 1.01
        o, a = dense_attention(lambda b, side, h: mx_field(f[b, side * hkv + h]), t.block_table.cpu().numpy(), got_q,
                               np.repeat(req, hkv), np.repeat(pos + 1, hkv), hkv, group, 1 / math.sqrt(128))
        gd = bf16_to_f64(out.view(torch.int16).cpu().numpy().view(np.uint16))
        # the dense attention's own bound, with logits of |q k| <= 128 * 16 * 16
        assert (np.abs(gd - o) <= 2.0 ** -8 * np.abs(o) + 2.0 ** -10 * a).all()
        # only the step's slots changed
        changed = (kv.buffer != before).view(nb, 2 * hkv, 8704)[:, 0, :8192].reshape(nb * 128, 64).any(1)
        slots = t.slot[:live]
        assert changed.sum() <= live and not changed[torch.isin(torch.arange(nb * 128, device="cuda"), slots, invert=True)].any()


def test_tables_and_norms_in_front_of_the_indexer():
    """A layer with an indexer: whatever the tables and the fused writer give,
    selecting every page attends like the rows written one by one."""
    from block_sparse_paged_score_gb300 import bsp, step
    n, ql, nb, group = 3, 2, 40, 16
    g = torch.Generator().manual_seed(5)
    kv, idx = bsp.KvCache(FP8, 1, nb, 0.01, 0.01), bsp.IndexCache(FP8, 1, nb)
    rope = step.rope_table(3000, 64, 1e5)
    w = {k: (1 + 0.1 * torch.randn(128, generator=g)).bfloat16().cuda()
         for k in ("q_weight", "k_weight", "idx_q_weight", "idx_k_weight")}
    free = torch.randperm(nb, generator=g).int().cuda()
    ctx0 = torch.tensor([300, 17, 900], dtype=torch.int32)
    total = int(ctx0.sum())
    # the contexts in one chunk, then a decode step
    tables = step.StepTables(n, 10, total, nb)
    op = step.NormRopeWrite(kv, idx, group, total, rope_table=rope, idx_q_dtype=bsp.FP8_E4M3, **w)
    row = lambda T: [torch.randn(T, h, 128, generator=g).bfloat16().cuda() for h in (group, 1, 1, 1, 1)]  # noqa: E731
    t = tables.run(torch.zeros(n, dtype=torch.int32, device="cuda"), ctx0.cuda(), free)
    op.run(*row(total), t.query_abs_pos, t.slot)
    taken, lens = t.blocks_taken.clone(), t.seq_lens.clone()
    small = step.StepTables(n, 10, n * ql, nb, block_table=t.block_table)
    x = row(n * ql)
    new = torch.full((n,), ql, dtype=torch.int32, device="cuda")
    t = small.run(lens, new, free, taken)
    q, iq = op.run(*x, t.query_abs_pos, t.slot)
    row_seq, row_len = bsp.row_lengths_prefill(t.query_req_id, t.query_abs_pos, 1)
    assert torch.equal(torch.stack([row_seq, row_len]), torch.stack(bsp.row_lengths_decode(t.seq_lens, ql, 1)))
    scores = bsp.index_score(idx, iq, bsp.FP8_E4M3, t.block_table, row_seq, row_len, ql, 80)
    _, sbt, sctx = bsp.topk_select(scores, row_seq, row_len, t.block_table, FP8, 80)
    assert torch.equal(sctx, row_len)  # every page selected
    out = bsp.sparse_pa_decode(kv, q, bsp.BF16, group, sbt, sctx, 80)
    # the same attention over the rows read back from the cache
    for s in range(n):
        L = int(t.seq_lens[s])
        p = torch.arange(L, device="cuda")
        slots = t.block_table[s, p // 128].long() * 128 + p % 128
        k, v, _ = bsp.kv_page_read(kv, None, slots)
        for j in range(ql):
            seen = int(row_len[s * ql + j])
            z = q[s * ql + j].double() @ k[:seen, 0].double().T / math.sqrt(128)
            o = torch.softmax(z, -1) @ v[:seen, 0].double()
            # K and V read back are rounded to bf16 once more, 2^-9 each of a value: a logit moves by at most
            # l = 2^-9 scale sum |q k|, a weight and the sum by l each, V by 2^-9; the call itself by 2^-11 (f16
            # weights) and 2^-8 of the output
            l = 2.0 ** -9 * float((q[s * ql + j].double().abs() @ k[:seen, 0].double().abs().T).max()) / math.sqrt(128)
            a = torch.softmax(z, -1) @ v[:seen, 0].double().abs()
            tol = 2.0 ** -8 * o.abs() + (2 * l + 2.0 ** -9 + 2.0 ** -10) * a
            assert ((out[s * ql + j].double() - o).abs() <= tol).all()
    assert small.dev_err.item() == 0 and op.dev_err.item() == 0
