"""bsp_step_tables against the definition, request by request: every output is
a whole number and has to be equal."""
import numpy as np
import pytest
import torch

from plain64 import step_tables

pytestmark = pytest.mark.gpu

OUT = ("block_table", "seq_lens", "cu_tokens", "blocks_taken", "slot", "query_req_id", "query_abs_pos")


def _case(seed, n, width, ctx_hi, new_hi, extra_free=20, zeros=True):
    r = np.random.default_rng(seed)
    ctx, new = r.integers(0, ctx_hi + 1, n).astype(np.int32), r.integers(0 if zeros else 1, new_hi + 1, n).astype(np.int32)
    have = -(-ctx // 128)
    fresh = -(-(ctx + new) // 128) - have
    ids = r.permutation(int(have.sum() + fresh.sum()) + extra_free + 3).astype(np.int32)
    table = np.full((n, width), -1, np.int32)
    at = 0
    for s in range(n):
        table[s, :min(have[s], width)] = ids[at:at + min(have[s], width)]
        at += min(have[s], width)
    return ctx, new, table, ids[at:].copy(), len(ids)


def _run(ctx, new, table, free, head, capacity, num_blocks):
    from block_sparse_paged_score_gb300 import step
    t = step.StepTables(len(ctx), table.shape[1], capacity, num_blocks, block_table=torch.from_numpy(table).cuda())
    g = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    for x in (t.slot, t.query_req_id, t.query_abs_pos, t.seq_lens, t.cu_tokens, t.blocks_taken):
        x.fill_(-77)
    h = None if head is None else torch.tensor([head], dtype=torch.int32, device="cuda")
    t.run(g(ctx), g(new), g(free), h)
    torch.cuda.synchronize()
    return t


def _check(ctx, new, table, free, head, capacity, num_blocks):
    t = _run(ctx, new, table, free, head, capacity, num_blocks)
    want, err = step_tables(ctx, new, table, free, head or 0, capacity, num_blocks)
    for k in OUT:
        assert np.array_equal(getattr(t, k).cpu().numpy(), want[k]), k
    assert t.dev_err.item() == err
    return t


# sizes around a thread's 4 requests, a warp's 128, the tile's 1024 and two tiles
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 127, 128, 129, 1023, 1024, 1025, 2500])
@pytest.mark.parametrize("new_hi", [1, 4, 300])
def test_every_output(n, new_hi):
    ctx, new, table, free, nb = _case(n * 7 + new_hi, n, 9, 700, new_hi)
    _check(ctx, new, table, free, 3, int(new.sum()) + 5, nb)


def test_one_long_chunk_spans_many_ctas():
    ctx, new = np.array([5, 130, 0], np.int32), np.array([1, 40000, 77], np.int32)
    table = np.full((3, 400), -1, np.int32)
    table[0, 0], table[1, :2] = 900, (901, 902)
    free = np.random.default_rng(0).permutation(800).astype(np.int32)
    _check(ctx, new, table, free, None, 40100, 1000)


@pytest.mark.parametrize("capacity", [0, 1, 3])
def test_no_new_tokens_and_pad_rows(capacity):
    ctx, new, table, free, nb = _case(1, 6, 4, 300, 0)
    _check(ctx, new, table, free, 0, capacity, nb)


def test_no_requests():
    _check(np.zeros(0, np.int32), np.zeros(0, np.int32), np.zeros((0, 4), np.int32), np.arange(4, dtype=np.int32), 0, 5, 4)


def test_negative_lengths_count_as_zero():
    ctx, new, table, free, nb = _case(2, 5, 5, 300, 9)
    ctx[1], new[2] = -5, -9
    table[1] = -1
    _check(ctx, new, table, free, 0, 40, nb)


@pytest.mark.parametrize("fault", ["capacity", "width", "free", "head", "free id", "table id"])
def test_a_step_that_does_not_fit_is_flagged_and_has_no_slots(fault):
    ctx, new, table, free, nb = _case(3, 40, 9, 700, 300, zeros=False)
    head, cap = 2, int(new.sum()) + 4
    if fault == "capacity":
        cap = int(new.sum()) - 7
    elif fault == "width":
        table = table[:, :6].copy()
    elif fault == "free":
        free = free[:20].copy()
    elif fault == "head":
        head = -4
    elif fault == "free id":
        free[10], free[15] = nb, -3
    else:
        s = int(np.flatnonzero((ctx > 128) & (ctx % 128 != 0))[0])
        table[s, ctx[s] // 128] = nb + 5
    t = _check(ctx, new, table, free, head, cap, nb)
    assert t.dev_err.item() == (2 if fault.endswith(" id") else 32)


def test_positions_past_the_table_at_the_largest_lengths():
    top = 2 ** 31 - 1
    ctx, new = np.array([top - 3, 10], np.int32), np.array([3, 2], np.int32)
    table = np.full((2, 2), 1, np.int32)
    t = _check(ctx, new, table, np.arange(4, dtype=np.int32), 0, 8, 4)
    assert t.query_abs_pos.cpu().tolist()[:5] == [top - 3, top - 2, top - 1, 10, 11]


def test_a_second_step_continues_the_first_and_a_captured_one_replays():
    from block_sparse_paged_score_gb300 import step
    n, cap, nb = 33, 33 * 70 + 2, 600
    r = np.random.default_rng(9)
    free = r.permutation(nb).astype(np.int32)
    t = step.StepTables(n, 12, cap, nb)
    ctx = torch.zeros(n, dtype=torch.int32, device="cuda")
    new = torch.zeros(n, dtype=torch.int32, device="cuda")
    fr, head = torch.from_numpy(free).cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    t.run(ctx, new, fr, head)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        t.run(ctx, new, fr, head)
        ctx.copy_(t.seq_lens)
        head += t.blocks_taken
    table, c, h = np.full((n, 12), -1, np.int32), np.zeros(n, np.int32), 0
    for i in range(6):
        m = r.integers(0, 71, n).astype(np.int32)
        new.copy_(torch.from_numpy(m))
        g.replay()
        want, err = step_tables(c, m, table, free, h, cap, nb)
        torch.cuda.synchronize()
        for k in OUT:
            assert np.array_equal(getattr(t, k).cpu().numpy(), want[k]), (i, k)
        table, c, h = want["block_table"], want["seq_lens"], h + int(want["blocks_taken"][0])
        assert head.item() == h
    assert t.dev_err.item() == 0
