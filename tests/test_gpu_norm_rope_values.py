"""bsp_norm_rope_write once more, with comparisons that a NaN does not pass, and
on rows whose squares leave fp32's range.  Tolerances are those derived in
test_gpu_norm_rope."""
import numpy as np
import pytest
import torch

import test_gpu_norm_rope as base
from plain64 import BF16, FP8, MX

pytestmark = pytest.mark.gpu


def _near(got, want, tol, what):
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


@pytest.fixture(autouse=True)
def strict(monkeypatch):
    monkeypatch.setattr(base, "_near", _near)


def _check(c):
    q, iq = c.run()
    assert c.op.dev_err.item() == 0
    base._check_queries(c, q, "q")
    base._check_queries(c, iq, "idx_q")
    base._check_caches(c)


@pytest.mark.parametrize("kv,idx", [(BF16, BF16), (FP8, FP8), (MX, MX), (FP8, MX), (MX, BF16)])
@pytest.mark.parametrize("T,hkv,group,rot,pairs,q8", [(7, 2, 8, 64, False, True), (65, 1, 16, 96, False, False),
                                                      (130, 4, 1, 16, True, True), (33, 1, 2, 0, False, False),
                                                      (3801, 1, 3, 64, False, True), (3801, 2, 1, 128, True, False)])
def test_values(kv, idx, T, hkv, group, rot, pairs, q8):
    _check(base.Case(T, hkv, group, kv, idx, rot, pairs, q8, pads=3, seed=T + kv, offset=float(T % 2), fused=T != 65))


@pytest.mark.parametrize("T", [6, 4000])
def test_rows_of_zeros_and_large_rows(T):
    c = base.Case(T, 1, 2, MX, FP8, 64, eps=1e-6)
    for x in c.x.values():
        x[0] = 0
        x[1] *= 2.0 ** 40
        x[2] *= 2.0 ** -60
    _check(c)


@pytest.mark.parametrize("kv,idx", [(BF16, BF16), (FP8, FP8), (MX, MX)])
@pytest.mark.parametrize("T,rot,pairs,q8,eps", [(12, 64, False, False, 1e-6), (12, 128, True, True, 0.0),
                                                (4000, 64, False, True, 0.0), (4000, 32, True, False, 1e-6)])
def test_rows_whose_squares_leave_fp32(kv, idx, T, rot, pairs, q8, eps):
    """Rows of 2^-100 to 2^120 times normal ones, among ordinary rows; without an
    epsilon the small ones are normed to 1 as well."""
    c = base.Case(T, 1, 4, kv, idx, rot, pairs, q8, seed=T + rot, eps=eps)
    r = np.random.default_rng(T)
    for name, x in c.x.items():
        for t in range(T):
            if r.random() < 0.5 and t < 200:
                x[t] *= 2.0 ** int(r.integers(-100, 121))
    _check(c)


def test_rows_that_are_not_finite_are_not_finite_alone():
    c = base.Case(40, 1, 4, BF16, BF16, 64, seed=3)
    want = [t.clone() for t in c.run()]
    c.x["q"][5, 1, 3], c.x["q"][7, 0, 100], c.x["idx_q"][9, 0, 64] = float("nan"), float("inf"), -float("inf")
    got = c.run()
    for g, w, hit in ((got[0], want[0], [(5, 1), (7, 0)]), (got[1], want[1], [(9, 0)])):
        for t in range(40):
            for h in range(g.shape[1]):
                assert g[t, h].isnan().any() if (t, h) in hit else torch.equal(g[t, h], w[t, h]), (t, h)
