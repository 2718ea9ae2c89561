"""The steps over a block-scaled cache: every call has the step's error word and
the step's buffers, and the arguments that do not go together are refused."""
import contextlib
import types

import pytest
import torch

from block_sparse_paged_score_gb300 import bsp, step


@pytest.fixture
def calls(monkeypatch):
    seen = []

    class Lib:
        def __getattr__(self, name):
            def call(*a):
                if name in ("bsp_dense_pa_decode_fp8", "bsp_kv_scaled_write", "bsp_kv_scaled_read"):
                    seen.append((name, a[-2]))
                elif name in ("bsp_step_tables", "bsp_norm_rope_write", "bsp_prompt_attention"):
                    seen.append((name, a[0]._obj.dev_err))
                return 16 if name.endswith("_bytes") else 0
            return call

    monkeypatch.setattr(bsp, "lib", lambda *a: Lib())
    monkeypatch.setattr(bsp, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    return seen


def pieces():
    cache = bsp.BlockScaledKvCache(1, 4, buffer=torch.zeros(64, dtype=torch.uint8), k_scales=torch.zeros(4, 1),
                                   v_scales=torch.zeros(4, 1))
    i = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    x = [torch.zeros(2, h, 128, dtype=torch.bfloat16) for h in (4, 1, 1)]
    stream = types.SimpleNamespace(device=torch.device("cpu"), cuda_stream=0)
    return cache, i, x, stream, dict(device="cpu", rope_table=torch.zeros(8, 64))


def test_every_call_of_a_step_has_the_steps_error_word(calls):
    cache, i, x, stream, kw = pieces()
    head = ["bsp_step_tables", "bsp_norm_rope_write", "bsp_kv_scaled_write"]
    for st, ctx, rest in ((step.ScaledPromptStep(cache, 4, 2, 2, 3, **kw), None, ["bsp_prompt_attention"]),
                          (step.ScaledPromptStep(cache, 4, 2, 2, 3, key_capacity=9, **kw), i(0, 0),
                           ["bsp_kv_scaled_read", "bsp_prompt_attention"]),
                          (step.ScaledDecodeStep(cache, 4, 2, 1, 3, **kw), i(0, 0), ["bsp_dense_pa_decode_fp8"])):
        calls.clear()
        st.tables.seq_lens.zero_(), st.tables.block_table.zero_()
        st.run(ctx, i(1, 1), i(0, 1), None, *x, stream=stream)
        assert calls == [(name, st.dev_err.data_ptr()) for name in head + rest]


def test_slots_of_the_keys(calls):
    cache, i, x, stream, kw = pieces()
    st = step.ScaledPromptStep(cache, 4, 3, 2, 2, key_capacity=300, block_table=i(3, -1, 7, 5, 2, 0).view(3, 2), **kw)
    st.tables.seq_lens.copy_(i(5, 130, 128))
    slot = st._key_slots(i(0, 1, 128))  # the first request has no new tokens
    assert st.cu_k.tolist() == [0, 0, 130, 258]
    want = [7 * 128 + t for t in range(128)] + [5 * 128, 5 * 128 + 1] + [2 * 128 + t for t in range(128)]
    assert slot.tolist() == want + [-1] * 42 and slot.dtype is torch.int64
    st.tables.seq_lens.copy_(i(130, 0, 300))  # no block for two tokens; past the capacity and the table
    slot = st._key_slots(i(1, 1, 1))
    assert slot.tolist()[:130] == [3 * 128 + t for t in range(128)] + [-1, -1] and len(slot) == 300
    assert slot.tolist()[130:] == [2 * 128 + t for t in range(128)] + [t for t in range(42)]


def test_contexts_need_a_key_capacity(calls):
    cache, i, x, stream, kw = pieces()
    for cap, ctx in ((0, i(0, 0)), (4, None)):
        st = step.ScaledPromptStep(cache, 4, 2, 2, 3, key_capacity=cap, **kw)
        calls.clear()
        with pytest.raises(ValueError, match="contexts"):
            st.run(ctx, i(1, 1), i(0, 1), None, *x, stream=stream)
        assert not calls
    with pytest.raises(ValueError, match="keys"):
        step.NormRopeWrite(cache, None, 4, 2, device="cpu", k_out_heads=1)
