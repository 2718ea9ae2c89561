"""Where a call's own outputs and workspaces come from: the memory pool of the
stream it runs on (a stand-in library and stream; no GPU needed)."""
import contextlib
import types

import pytest
import torch

from block_sparse_paged_score_gb300 import bsp


class Lib:
    def __getattr__(self, name):
        return lambda *a: 4096 if name.endswith("_bytes") else 0

    def bsp_kv_page_read(self, kv, idx, slot, n, k, v, idx_k, *a):
        return int(bool(k) != bool(v))


class Stream:
    device, cuda_stream = torch.device("cpu"), 0


@pytest.fixture
def made(monkeypatch):
    """The stream that was current at each allocation (None: torch's)."""
    current, out = [None], []

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    def counted(make):
        return lambda *a, **k: (out.append(current[-1]), make(*a, **k))[1]

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", counted(torch.empty))
    monkeypatch.setattr(torch, "zeros", counted(torch.zeros))
    monkeypatch.setattr(bsp, "lib", lambda *a: Lib())
    monkeypatch.setattr(bsp, "_Current", Stream)
    for name in ("_ptr", "_io_ptr"):
        monkeypatch.setattr(bsp, name, lambda t: None if t is None else t.data_ptr())
    return out


def _i(*shape):
    return torch.ones(shape, dtype=torch.int32)


BUF = torch.ones(16, dtype=torch.uint8)
KV = types.SimpleNamespace(desc=bsp.KvCacheDesc(), num_kv_heads=1, buffer=BUF)
IDX = types.SimpleNamespace(desc=bsp.IndexCacheDesc(), num_heads=1, buffer=BUF)
Q = torch.ones(2, 4, 128, dtype=torch.bfloat16)
CALLS = {
    "dense_pa_decode": (2, lambda s: bsp.dense_pa_decode(KV, Q, bsp.BF16, 4, _i(1, 3), _i(2), _i(2), 2, stream=s)),
    "kv_page_read": (3, lambda s: bsp.kv_page_read(KV, IDX, torch.ones(2, dtype=torch.int64), stream=s)),
    "cast_e4m3": (1, lambda s: bsp.cast_e4m3(Q, stream=s)),
    "row_lengths_decode": (2, lambda s: bsp.row_lengths_decode(_i(2), 1, 1, stream=s)),
    "row_lengths_prefill": (2, lambda s: bsp.row_lengths_prefill(_i(2), _i(2), 1, stream=s)),
    "index_score": (1, lambda s: bsp.index_score(IDX, Q, bsp.BF16, _i(1, 3), _i(2), _i(2), 1, 8, stream=s)),
    "index_score_prefill": (1, lambda s: bsp.index_score_prefill(IDX, Q, bsp.FP8_E4M3, _i(1, 3), _i(2), _i(2), _i(2), 1,
                                                                 1, 8, stream=s)),
    "topk_select": (3, lambda s: bsp.topk_select(torch.ones(2, 8), _i(2), _i(2), _i(1, 3), bsp.FP8_E4M3, 4, stream=s)),
    "sparse_pa_decode": (2, lambda s: bsp.sparse_pa_decode(KV, Q, bsp.BF16, 4, _i(2, 4), _i(2), 4, stream=s)),
    "sparse_pa_decode_noalloc": (1, lambda s: bsp.sparse_pa_decode_noalloc(KV, Q, bsp.BF16, 4, _i(2, 4), _i(2), 4,
                                                                           stream=s)),
    "sparse_pa_prefill": (1, lambda s: bsp.sparse_pa_prefill(KV, Q, bsp.BF16, 4, _i(2, 4), _i(2), 4, stream=s)),
}


@pytest.mark.parametrize("name", CALLS)
def test_buffers_come_from_the_pool_of_the_stream_of_the_call(made, name):
    n, call = CALLS[name]
    side = Stream()
    for stream in (side, None):
        made.clear()
        call(stream)
        assert made == [stream] * n, name


@pytest.mark.parametrize("name", ["decode_workspace", "dense_pa_workspace"])
def test_a_workspace_for_a_stream_comes_from_its_pool(made, name):
    make, args = getattr(bsp, name), (2, 1, 4) + ((1,) if name == "dense_pa_workspace" else ())
    side = Stream()
    make(*args, device="cpu", stream=side)
    make(*args, device="cpu")
    assert made == [side, None]


def test_a_read_of_no_tokens_into_given_rows(made):
    """Empty tensors have no address: a given k beside an empty v is not a missing one."""
    k = torch.ones(4, 1, 128, dtype=torch.bfloat16)
    got = bsp.kv_page_read(KV, IDX, torch.ones(0, dtype=torch.int64), k=k, stream=Stream())
    assert got[0] is k and got[1].shape == got[2].shape == (0, 1, 128)
