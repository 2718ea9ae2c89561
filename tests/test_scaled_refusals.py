"""What the block-scaled cache's calls and the prompt attention refuse, on the
host, before anything is enqueued (no GPU needed: the addresses are never
dereferenced; with a GPU the tests that use them are left out, as a case that
should have been refused would launch)."""
import ctypes as C
import types

import pytest
import torch

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake device addresses must never reach a GPU")
BASE, STEP = 1 << 32, 1 << 28
T, HQ, HKV, BLOCKS = 6, 8, 2, 64
CACHE, CACHE_BYTES = 1 << 40, BLOCKS * HKV * 32768
REFUSED, UNSUPPORTED, WORKSPACE, LAUNCHED = 1, 2, 3, 4  # a launch fails without a device


@pytest.fixture(scope="module")
def bsp():
    from block_sparse_paged_score_gb300 import bsp
    bsp.lib()
    return bsp


def at(names):
    return {n: BASE + i * STEP for i, n in enumerate(names)}


def cache(bsp, dtype=1):
    kv = bsp.KvCacheDesc()
    assert bsp.lib().bsp_kv_cache_interleaved(dtype, HKV, CACHE, BLOCKS, 0.5, 0.5, C.byref(kv)) == 0
    return kv


@pytest.fixture()
def write(bsp):
    ptr = at(["ks", "vs", "k", "v", "slot", "dev_err"])

    def status(dtype=1, ks_stride=256, vs_stride=256, tokens=T, scales=True, **kw):
        a = {**ptr, **kw}
        s = bsp.KvScalesDesc(a["ks"], a["vs"])
        return bsp.lib().bsp_kv_scaled_write(C.byref(cache(bsp, dtype)), C.byref(s) if scales else None, a["k"], ks_stride,
                                             a["v"], vs_stride, a["slot"], tokens, a["dev_err"], None)

    status.ptr = ptr
    return status


@no_gpu
def test_write(bsp, write):
    n0, p = bsp.launch_count(), write.ptr
    for n in ("ks", "vs", "k", "v", "slot"):
        assert write(**{n: None}) == REFUSED, n
        assert write(**{n: p[n] + 2}) == REFUSED, n
    assert write(scales=False) == REFUSED
    assert write(dtype=0) == UNSUPPORTED and write(dtype=2) == UNSUPPORTED
    assert write(tokens=-1) == REFUSED and write(tokens=0) == 0
    assert write(ks_stride=248) == REFUSED and write(vs_stride=260) == REFUSED
    assert write(vs_stride=(1 << 32) + 8) == UNSUPPORTED
    for n in ("ks", "vs", "k", "v", "slot", "dev_err"):  # in the cache's pages
        assert write(**{n: CACHE + 4096}) == REFUSED, n
    assert write(ks=p["vs"] + 4 * BLOCKS * HKV - 4) == REFUSED  # the scales in each other, in an input, under dev_err
    assert write(ks=p["k"] + T * 512 - 16) == REFUSED and write(dev_err=p["slot"] + 40) == REFUSED
    assert write(dev_err=p["vs"] + 8) == REFUSED
    assert write(ks=p["k"] + 5 * 2 * 640 + 512, ks_stride=640) == LAUNCHED  # right behind the last row
    assert write() == LAUNCHED and write(dev_err=None) == LAUNCHED
    assert bsp.launch_count() == n0


@no_gpu
def test_read(bsp):
    p = at(["ks", "vs", "k", "v", "slot", "dev_err"])

    def status(dtype=1, tokens=T, **kw):
        a = {**p, **kw}
        return bsp.lib().bsp_kv_scaled_read(C.byref(cache(bsp, dtype)), C.byref(bsp.KvScalesDesc(a["ks"], a["vs"])),
                                            a["slot"], tokens, a["k"], a["v"], a["dev_err"], None)

    for n in ("ks", "vs", "k", "v", "slot"):
        assert status(**{n: None}) == REFUSED, n
        assert status(**{n: p[n] + 2}) == REFUSED, n
    assert status(dtype=0) == UNSUPPORTED and status(tokens=-1) == REFUSED and status(tokens=0) == 0
    assert status(k=CACHE) == REFUSED and status(v=p["k"] + 512) == REFUSED and status(k=p["slot"]) == REFUSED
    assert status(v=p["ks"]) == REFUSED and status(dev_err=p["k"]) == REFUSED
    assert status() == LAUNCHED and status(dev_err=None) == LAUNCHED


@no_gpu
def test_dense_attention(bsp):
    p = at(["ks", "vs", "q", "table", "seq", "len", "out", "ws", "dev_err"])

    def status(dtype=1, q_dtype=0, heads=HQ, stride=4, rows=T * HKV, group=1, scale=0.1, ws_bytes=1 << 27, scales=True, **kw):
        a = {**p, **kw}
        s = bsp.KvScalesDesc(a["ks"], a["vs"])
        return bsp.lib().bsp_dense_pa_decode_fp8(C.byref(cache(bsp, dtype)), C.byref(s) if scales else None, a["q"], q_dtype,
                                                 heads, a["table"], stride, a["seq"], a["len"], rows, group,
                                                 C.c_float(scale), a["out"], a["ws"], ws_bytes, a["dev_err"], None)

    for n in ("ks", "vs", "q", "table", "seq", "len", "out"):
        assert status(**{n: None}) == REFUSED, n
        assert status(**{n: p[n] + 2}) == REFUSED, n
    assert status(dtype=0) == UNSUPPORTED and status(dtype=2) == UNSUPPORTED and status(q_dtype=2) == UNSUPPORTED
    assert status(dtype=0, scales=False) == UNSUPPORTED
    assert status(heads=6) == UNSUPPORTED and status(heads=7) == REFUSED and status(rows=T * HKV - 1) == REFUSED
    assert status(group=9) == UNSUPPORTED and status(group=0) == UNSUPPORTED and status(stride=0) == REFUSED
    for x in (float("inf"), float("nan")):
        assert status(scale=x) == REFUSED
    assert status(rows=0) == 0
    assert status(out=p["q"]) == REFUSED and status(out=CACHE) == REFUSED and status(dev_err=p["len"]) == REFUSED
    if bsp.dense_pa_fp8_workspace_bytes(T * HKV, HKV, HQ // HKV, 1):
        assert status(ws=None) == WORKSPACE and status(ws_bytes=16) == WORKSPACE and status(ws=p["ws"] + 8) == WORKSPACE
        assert status(ws=p["q"]) == REFUSED and status(ws=p["out"]) == REFUSED
    assert status() == LAUNCHED and status(scales=False) == LAUNCHED and status(q_dtype=1) == LAUNCHED


@no_gpu
def test_prompt_attention(bsp):
    p = at(["q", "k", "v", "cu_q", "cu_k", "out", "ws", "dev_err"])

    def status(**kw):
        a = bsp.PromptAttentionArgs()
        for n, x in p.items():
            setattr(a, n, x)
        a.q_stride, a.k_stride, a.v_stride = HQ * 128, HKV * 128, HKV * 128
        a.num_tokens, a.num_keys, a.num_q_heads, a.num_kv_heads, a.num_seqs = 300, 400, HQ, HKV, 3
        a.sm_scale, a.ws_bytes = 0.1, 1 << 27
        for n, x in kw.items():
            setattr(a, n, x)
        return bsp.lib().bsp_prompt_attention(C.byref(a), None)

    n0 = bsp.launch_count()
    for n in ("q", "k", "v", "cu_q", "cu_k", "out"):
        assert status(**{n: None}) == REFUSED, n
        assert status(**{n: p[n] + 2}) == REFUSED, n
    for n in ("num_tokens", "num_keys", "num_seqs"):
        assert status(**{n: -1}) == REFUSED, n
    assert status(num_tokens=0) == 0 and status(num_seqs=0) == 0
    assert status(num_q_heads=0) == REFUSED and status(num_kv_heads=0) == REFUSED and status(num_q_heads=7) == REFUSED
    assert status(num_q_heads=6) == UNSUPPORTED and status(num_q_heads=64, q_stride=64 * 128) == UNSUPPORTED
    assert status(num_seqs=(1 << 20) + 1) == UNSUPPORTED and status(num_tokens=1 << 30) == UNSUPPORTED
    for n in ("q_stride", "k_stride", "v_stride"):
        assert status(**{n: 64}) == REFUSED and status(**{n: HQ * 128 + 4}) == REFUSED, n
        assert status(**{n: (1 << 32) + 8}) == UNSUPPORTED, n
    for x in (float("inf"), float("nan")):
        assert status(sm_scale=x) == REFUSED
    for n in ("q", "k", "v", "cu_q", "cu_k"):
        assert status(out=p[n]) == REFUSED and status(dev_err=p[n] + 4) == REFUSED, n
    if bsp.prompt_attention_workspace_bytes(300, 3, HKV, HQ // HKV):
        assert status(ws=None) == WORKSPACE and status(ws_bytes=16) == WORKSPACE and status(ws=p["ws"] + 8) == WORKSPACE
        assert status(ws=p["q"]) == REFUSED and status(ws=p["out"]) == REFUSED
    assert bsp.lib().bsp_prompt_attention(None, None) == REFUSED
    assert status() == LAUNCHED and status(cu_k=p["cu_q"]) == LAUNCHED
    assert bsp.launch_count() == n0


class Stream:
    device, cuda_stream = torch.device("cpu"), 0


@pytest.fixture()
def calls(monkeypatch, bsp):
    made = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: (made.append(name), 4096 if name.endswith("_bytes") else 0)[1]

    monkeypatch.setattr(bsp, "lib", lambda *a: Lib())
    return made


def scaled(bsp, device):
    c = object.__new__(bsp.BlockScaledKvCache)
    c.desc, c.scales, c.num_kv_heads, c.num_blocks = bsp.KvCacheDesc(), bsp.KvScalesDesc(), 1, 1
    c.buffer = torch.zeros(16, dtype=torch.uint8, device=device)
    return c


def test_binding(bsp, calls):
    x = lambda *s: torch.zeros(*s, 1, 128, dtype=torch.bfloat16)  # noqa: E731
    slot, cu = torch.zeros(3, dtype=torch.int64), torch.tensor([0, 3], dtype=torch.int32)
    here, there, s = scaled(bsp, "cpu"), scaled(bsp, "meta"), Stream()
    one = torch.zeros(1, dtype=torch.int32)
    bsp.kv_scaled_write(here, x(3), x(3), slot, stream=s)
    bsp.kv_scaled_read(here, slot, k=x(3), v=x(3), stream=s)
    bsp.prompt_attention(x(3), x(3), x(3), cu, out=x(3), ws=torch.zeros(4096, dtype=torch.uint8), stream=s)
    made = list(calls)
    for c in (lambda: bsp.kv_scaled_write(there, x(3), x(3), slot, stream=s),
              lambda: bsp.kv_scaled_read(there, slot, k=x(3), v=x(3), stream=s),
              lambda: bsp.kv_scaled_write(types.SimpleNamespace(desc=bsp.KvCacheDesc(), buffer=here.buffer, num_kv_heads=1),
                                          x(3), x(3), slot, stream=s),
              lambda: bsp.kv_scaled_write(here, x(2), x(3), slot, stream=s),
              lambda: bsp.kv_scaled_write(here, x(3), x(3).float(), slot, stream=s),
              lambda: bsp.kv_scaled_write(here, x(3), x(3), slot.int(), stream=s),
              lambda: bsp.kv_scaled_read(here, slot, k=x(2), v=x(3), stream=s),
              lambda: bsp.dense_pa_decode_fp8(there, x(1), 0, 1, one[None], one, one, 1, out=x(1),
                                              ws=torch.zeros(4096, dtype=torch.uint8), stream=s),
              lambda: bsp.prompt_attention(x(3), x(2), x(3), cu, out=x(3), stream=s),
              lambda: bsp.prompt_attention(x(3).float(), x(3), x(3), cu, out=x(3), stream=s),
              lambda: bsp.prompt_attention(x(3), x(3), x(3), cu.long(), out=x(3), stream=s),
              lambda: bsp.prompt_attention(x(3), x(3), x(3), cu, cu[:1], out=x(3), stream=s),
              lambda: bsp.prompt_attention(x(3), x(3), x(3), cu, out=x(2), stream=s),
              lambda: bsp.prompt_attention(x(3)[:, 0], x(3), x(3), cu, out=x(3), stream=s)):
        with pytest.raises(ValueError):
            c()
    assert [c for c in calls if not c.endswith("_bytes")] == [c for c in made if not c.endswith("_bytes")]
    with pytest.raises(ValueError):  # scales of too few elements, and of another type
        bsp.BlockScaledKvCache(1, 2, buffer=torch.zeros(65536, dtype=torch.uint8), k_scales=torch.zeros(1))
