"""A cache on another device than the stream is refused before the library is
called (stand-in stream and caches; no GPU needed)."""
import types

import pytest
import torch

from block_sparse_paged_score_gb300 import bsp, step


class Stream:
    device, cuda_stream = torch.device("cpu"), 0


def _cache(desc, device, **kw):
    return types.SimpleNamespace(desc=desc(), buffer=torch.zeros(16, dtype=torch.uint8, device=device), num_blocks=1, **kw)


KV = {d: _cache(bsp.KvCacheDesc, d, num_kv_heads=1) for d in ("cpu", "meta")}
IDX = {d: _cache(bsp.IndexCacheDesc, d, num_heads=1) for d in ("cpu", "meta")}


@pytest.fixture(autouse=True)
def calls(monkeypatch):
    made = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: (made.append(name), 4096 if name.endswith("_bytes") else 0)[1]

    monkeypatch.setattr(bsp, "lib", lambda *a: Lib())
    return made


def _dense(kv):
    one = torch.zeros(1, dtype=torch.int32)
    return bsp.dense_pa_decode(kv, torch.zeros(1, 4, 128, dtype=torch.bfloat16), bsp.BF16, 4, one[None], one, one, 1,
                               out=torch.zeros(1, 4, 128, dtype=torch.bfloat16), ws=torch.zeros(4096, dtype=torch.uint8),
                               stream=Stream())


def _read(kv, idx):
    x = lambda: torch.zeros(1, 1, 128, dtype=torch.bfloat16)  # noqa: E731
    return bsp.kv_page_read(kv, idx, torch.zeros(1, dtype=torch.int64), k=kv and x(), v=kv and x(), idx_k=idx and x(),
                            stream=Stream())


def test_caches_on_the_device_of_the_stream_pass(calls):
    _dense(KV["cpu"]), _read(KV["cpu"], IDX["cpu"]), _read(None, IDX["cpu"]), _read(KV["cpu"], None)
    step.NormRopeWrite(KV["cpu"], IDX["cpu"], 4, 2, device="cpu")
    assert calls.count("bsp_dense_pa_decode") == 1 and calls.count("bsp_kv_page_read") == 3


def test_caches_elsewhere_are_refused(calls):
    for call in (lambda: _dense(KV["meta"]), lambda: _read(KV["meta"], None), lambda: _read(None, IDX["meta"]),
                 lambda: _read(KV["cpu"], IDX["meta"]),
                 lambda: step.NormRopeWrite(KV["meta"], IDX["cpu"], 4, 2, device="cpu"),
                 lambda: step.NormRopeWrite(KV["cpu"], IDX["meta"], 4, 2, device="cpu"),
                 lambda: step.NormRopeWrite(None, IDX["meta"], 4, 2, device="cpu")):
        with pytest.raises(ValueError, match="cache is on meta"):
            call()
    assert not calls
