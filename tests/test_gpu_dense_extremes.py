"""bsp_dense_pa_decode at the ends of its inputs' ranges."""
import math

import numpy as np
import pytest
import torch

from test_gpu_dense_pa import Case, _f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("q_len", [1, 2, 4])
def test_a_query_that_is_not_finite_gives_nan_in_its_row_alone(value, q_len):
    """Every logit of such a row is infinite or NaN, whatever the keys hold, so
    softmax has no value there: all of the row is NaN (zeros where it sees nothing)."""
    c = Case([700, 1, 0, 129], q_len=q_len, q8=False, seed=31)
    # keys of 0 and of 0.5 in the dims that are hit, and ordinary ones
    for b in range(c.blocks):
        c.fields[b, 0, :8192].reshape(128, 64)[:, 0] = 0x10
    c.device()
    want = c.call().clone()
    hit = []
    for i, (tok, head, dim) in enumerate([(0, 3, 0), (q_len, 0, 1), (2 * q_len, 7, 77), (4 * q_len - 1, 15, 127)]):
        c.dq[tok, head, dim] = -value if i % 2 else value
        hit.append((tok, head))
    got = c.call()
    assert c.err.item() == 0
    for t in range(4 * q_len):
        for h in range(16):
            if (t, h) in hit and c.row_len[t] > 0:
                assert got[t, h].isnan().all(), (t, h)
            else:
                assert torch.equal(got[t, h], want[t, h]), (t, h)


@pytest.mark.parametrize("byte", [127, 200, 215, 230, 239])
@pytest.mark.parametrize("q8,q_len", [(True, 1), (False, 2), (True, 4)])
@pytest.mark.parametrize("code", [0xFF, 0x77])  # -6 and 6
def test_equal_logits_of_any_size_average_the_values(byte, q8, q_len, code):
    """Keys and queries of one value: 128 equal products sum exactly, so the logits of
    a row are the same number, bit for bit, and no error of theirs enters.  Sums of
    up to 8e36, logits of up to 1e36 in units of ln 2: well inside fp32."""
    c = Case([1, 77, 300, 2500], q_len=q_len, q8=q8, seed=byte)
    c.fields[:, 0, :8192], c.fields[:, 0, 8192:] = code, byte
    c.q_t = torch.full_like(c.q_t, 0x40 if byte > 235 else 0x7E) if q8 else torch.full_like(c.q_t, 2.0 if byte > 235 else 448.0)
    c.q[:] = 2.0 if byte > 235 else 448.0
    c.device()
    got = _f64(c.call())
    assert c.err.item() == 0
    o, a = c.want()
    tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 2.0 ** -13) * a
    for r in range(len(c.row_len)):
        tol[r] += c.floor(r)
    assert (np.abs(got - o) <= tol).all(), (got[0, 0, :4], o[0, 0, :4])


def test_a_context_of_two_to_the_31_minus_one_tokens():
    """The last block's last token is not seen.  Every token seen has the logit 0
    and the value 1; weights of 2^7 and their sums over a share of the blocks are
    exact in fp32, so the mean is off by bf16's half step and the join's roundings."""
    from block_sparse_paged_score_gb300 import bsp
    n = 4096  # blocks that the context goes through again and again, and the last one
    kv = bsp.KvCache(bsp.MXFP4, 1, n + 1)
    f = kv.buffer.view(n + 1, 2, 8704)
    f[:, :, 8192:] = 127
    f[:, 1, :8192] = 0x22  # V: 1
    f[n, 0, 127 * 64:8192], f[n, 1, 127 * 64:8192] = 0x77, 0xFF  # the unseen token: a logit of 70, V -6
    table = (torch.arange(1 << 24, dtype=torch.int32, device="cuda") % n)[None]
    table[0, -1] = n
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.ones(1, 16, 128, dtype=torch.bfloat16, device="cuda")
    one = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")  # noqa: E731
    out = bsp.dense_pa_decode(kv, q, bsp.BF16, 16, table, one(0), one(2 ** 31 - 1), 1, dev_err=err)
    assert err.item() == 0
    assert (out.float() - 1).abs().max() <= 2.0 ** -8
