"""DenseStep's error word: what any call of the step finds is in it."""
import types

import pytest
import torch

from block_sparse_paged_score_gb300 import bsp, step


def test_every_call_of_the_step_has_the_steps_error_word(monkeypatch):
    seen = []

    class Lib:
        def __getattr__(self, name):
            def call(*a):
                if name == "bsp_dense_pa_decode":
                    seen.append(a[-2])
                elif name in ("bsp_step_tables", "bsp_norm_rope_write"):
                    seen.append(a[0]._obj.dev_err)
                return 4096 if name.endswith("_bytes") else 0
            return call

    stream = types.SimpleNamespace(device=torch.device("cpu"), cuda_stream=0)
    monkeypatch.setattr(bsp, "lib", lambda *a: Lib())
    monkeypatch.setattr(bsp, "_ptr", lambda t: None if t is None else t.data_ptr())
    kv = types.SimpleNamespace(desc=bsp.KvCacheDesc(), num_kv_heads=1, num_blocks=4,
                               buffer=torch.zeros(16, dtype=torch.uint8))
    st = step.DenseStep(kv, 4, 2, 1, 3, device="cpu", rope_table=torch.zeros(8, 64))
    i = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    x = [torch.zeros(2, h, 128, dtype=torch.bfloat16) for h in (4, 1, 1)]
    st.run(i(0, 0), i(1, 1), i(0, 1), None, *x, stream=stream)
    assert seen == [st.dev_err.data_ptr()] * 3
    assert st.tables.dev_err is st.dev_err and st.norm.dev_err is st.dev_err
    # on their own they have one each, or the caller's
    word = torch.zeros(1, dtype=torch.int32)
    a, b = step.StepTables(2, 3, 2, 4, device="cpu"), step.StepTables(2, 3, 2, 4, device="cpu", dev_err=word)
    assert a.dev_err is not word and b.dev_err is word and b.args.dev_err == word.data_ptr()
    b = step.NormRopeWrite(kv, None, 4, 2, device="cpu", dev_err=word)
    assert b.dev_err is word and b.args.dev_err == word.data_ptr()


@pytest.mark.gpu
def test_a_free_list_that_runs_out_shows_in_the_steps_error_word():
    kv = bsp.KvCache(bsp.MXFP4, 1, 4)
    st = step.DenseStep(kv, 4, 2, 1, 3, q_dtype=bsp.BF16, rope_table=step.rope_table(8, 64))
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    x = [torch.zeros(2, h, 128, dtype=torch.bfloat16, device="cuda") for h in (4, 1, 1)]
    st.run(i(0, 0), i(1, 1), i(2, 3), None, *x)
    assert st.dev_err.item() == 0
    st.run(i(0, 0), i(1, 1), i(2), None, *x)
    assert st.dev_err.item() == 32 | 2  # no block for the second request's token, and none to attend to
