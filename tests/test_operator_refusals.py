"""What the step-table, norm-and-rotation, cache-read and dense-attention calls
refuse, on the host, before anything is enqueued (no GPU needed: the addresses
are never dereferenced; with a GPU the tests are left out, as a case that
should have been refused would launch)."""
import ctypes as C

import pytest
import torch

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="fake device addresses must never reach a GPU")
BASE = 1 << 32


@pytest.fixture(scope="module")
def bsp():
    from block_sparse_paged_score_gb300 import bsp
    bsp.lib()
    return bsp


def _addresses(names, step=1 << 26):
    return {n: BASE + i * step for i, n in enumerate(names)}


def _caches(bsp, kv_dtype, idx_dtype, hkv=1):
    kv, idx = bsp.KvCacheDesc(), bsp.IndexCacheDesc()
    assert bsp.lib().bsp_kv_cache_interleaved(kv_dtype, hkv, 1 << 40, 64, 0.5, 0.5, C.byref(kv)) == 0
    assert bsp.lib().bsp_index_cache_packed(idx_dtype, hkv, 1 << 41, 64, C.byref(idx)) == 0
    return kv, idx


def test_step_tables(bsp):
    ptrs = _addresses(["context_lens", "new_lens", "block_table", "free_blocks", "free_head", "seq_lens", "cu_tokens",
                       "blocks_taken", "slot", "query_req_id", "query_abs_pos", "dev_err"])

    def status(**kw):
        a = bsp.StepTablesArgs()
        for k, v in ptrs.items():
            setattr(a, k, v)
        a.num_seqs, a.bt_stride, a.num_free, a.token_capacity, a.num_blocks = 8, 16, 100, 64, 200
        for k, v in kw.items():
            setattr(a, k, v)
        return bsp.lib().bsp_step_tables(C.byref(a), None)

    n0 = bsp.launch_count()
    for k in ("context_lens", "new_lens", "block_table", "free_blocks", "seq_lens", "cu_tokens", "blocks_taken", "slot",
              "query_req_id", "query_abs_pos"):
        assert status(**{k: None}) == 1, k
    for k in ("num_seqs", "num_free", "token_capacity", "num_blocks"):
        assert status(**{k: -1}) == 1, k
    assert status(bt_stride=0) == 1
    assert status(num_seqs=65537) == 2
    assert status(slot=ptrs["slot"] + 4) == 1  # misaligned
    assert status(seq_lens=ptrs["context_lens"]) == 1  # in place
    assert status(blocks_taken=ptrs["free_head"]) == 1
    assert status(query_abs_pos=ptrs["slot"] + 8 * 63) == 1  # an output inside another
    assert bsp.lib().bsp_step_tables(None, None) == 1
    assert bsp.launch_count() == n0


def test_norm_rope_write(bsp):
    kv, idx = _caches(bsp, bsp.FP8_E4M3, bsp.MXFP4, 2)
    ptrs = _addresses(["q", "k", "v", "idx_q", "idx_k", "q_weight", "k_weight", "idx_q_weight", "idx_k_weight",
                       "rope_table", "positions", "slot", "q_out", "k_out", "idx_q_out", "dev_err"])

    def status(**kw):
        a = bsp.NormRopeArgs()
        for k, v in ptrs.items():
            setattr(a, k, v)
        a.q_stride, a.k_stride, a.v_stride, a.idx_q_stride, a.idx_k_stride = 1024, 256, 256, 256, 256
        a.num_tokens, a.num_q_heads, a.num_kv_heads, a.num_idx_heads = 4, 8, 2, 2
        a.eps, a.rope_rows, a.rot_dim = 1e-6, 100, 64
        a.kv, a.idx = C.pointer(kv), C.pointer(idx)
        for k, v in kw.items():
            setattr(a, k, v)
        return bsp.lib().bsp_norm_rope_write(C.byref(a), None)

    n0 = bsp.launch_count()
    for k in ("q_out", "idx_q_out", "q", "idx_q", "k", "v", "idx_k", "slot", "positions", "rope_table"):
        assert status(**{k: None}) == 1, k
    assert status(kv=None) == 1 and status(idx=None) == 1
    for k in ("q_stride", "k_stride", "v_stride", "idx_q_stride", "idx_k_stride"):
        assert status(**{k: 64}) == 1 and status(**{k: 1028}) == 1, k
    for k in ("q", "k", "v", "idx_q", "idx_k", "q_out", "k_out", "rope_table", "q_weight"):
        assert status(**{k: ptrs[k] + 8}) == 1, k  # misaligned
    assert status(num_tokens=-1) == 1 and status(num_q_heads=0) == 1
    assert status(num_kv_heads=1) == 1 and status(num_idx_heads=4) == 1  # not the caches'
    assert status(rot_dim=24) == 2 and status(rot_dim=144) == 2 and status(rot_dim=-16) == 2
    assert status(rope_rows=0) == 1
    assert status(eps=-1.0) == 1 and status(eps=float("nan")) == 1 and status(weight_offset=float("nan")) == 1
    assert status(q_out_dtype=bsp.MXFP4) == 2 and status(idx_q_out_dtype=7) == 2
    assert status(q_out=ptrs["q"], q_out_dtype=bsp.FP8_E4M3) == 1  # e4m3 in place
    assert status(q_out=ptrs["q"], q_stride=2048) == 1  # in place of strided rows
    assert status(q_out=ptrs["q"] + 256) == 1
    assert status(k_out=ptrs["v"]) == 1 and status(idx_q_out=ptrs["q_out"] + 512) == 1
    assert bsp.lib().bsp_norm_rope_write(None, None) == 1
    assert status(num_tokens=0) == 0
    assert bsp.launch_count() == n0


def test_kv_page_read(bsp):
    kv, idx = _caches(bsp, bsp.BF16, bsp.FP8_E4M3)
    L, p = bsp.lib(), _addresses(["slot", "k", "v", "ik", "err"])

    def status(kv_=C.byref(kv), idx_=C.byref(idx), slot=p["slot"], n=5, k=p["k"], v=p["v"], ik=p["ik"]):
        return L.bsp_kv_page_read(kv_, idx_, slot, n, k, v, ik, p["err"], None)

    n0 = bsp.launch_count()
    assert status(n=-1) == 1 and status(k=None) == 1 and status(v=None) == 1
    assert status(kv_=None) == 1 and status(idx_=None) == 1 and status(slot=None) == 1
    assert status(k=p["k"] + 2) == 1 and status(ik=p["ik"] + 8) == 1 and status(slot=p["slot"] + 4) == 1
    assert status(n=0) == 0 and status(k=None, v=None, ik=None, kv_=None, idx_=None) == 0
    assert bsp.launch_count() == n0


def test_dense_pa_decode(bsp):
    L = bsp.lib()
    mx, _ = _caches(bsp, bsp.MXFP4, bsp.MXFP4, 2)
    fp8, _ = _caches(bsp, bsp.FP8_E4M3, bsp.MXFP4, 2)
    p = _addresses(["q", "bt", "seq", "len", "out", "ws", "err"])

    def status(kv=mx, q=p["q"], qt=bsp.FP8_E4M3, hq=32, bt=p["bt"], stride=8, seq=p["seq"], ln=p["len"], rows=16,
               group=4, scale=0.1, out=p["out"], ws=p["ws"], nbytes=1 << 30):
        return L.bsp_dense_pa_decode(C.byref(kv) if kv is not None else None, q, qt, hq, bt, stride, seq, ln, rows,
                                     group, scale, out, ws, nbytes, p["err"], None)

    n0 = bsp.launch_count()
    assert status(kv=None) == 1 and status(kv=fp8) == 2
    for f, v in (("k_base", (1 << 40) + 16), ("id_stride_bytes", mx.id_stride_bytes + 16)):
        odd = bsp.KvCacheDesc()
        C.memmove(C.byref(odd), C.byref(mx), C.sizeof(odd))
        setattr(odd, f, v)
        assert status(kv=odd) == 2, f
    assert status(qt=bsp.MXFP4) == 2
    for k in ("q", "bt", "seq", "ln", "out"):
        assert status(**{k: None}) == 1, k
    assert status(q=p["q"] + 8) == 1 and status(out=p["out"] + 8) == 1 and status(ln=p["len"] + 2) == 1
    assert status(hq=31) == 1 and status(hq=6) == 2 and status(hq=64) == 2 and status(hq=0) == 1
    assert status(rows=15) == 1 and status(rows=-2) == 1 and status(stride=0) == 1
    assert status(group=0) == 2 and status(group=9) == 2
    assert status(scale=float("inf")) == 1 and status(scale=float("nan")) == 1
    assert status(rows=0) == 0
    need = bsp.dense_pa_workspace_bytes(16, 2, 16, 4)
    if need:
        assert status(ws=None) == 3 and status(nbytes=need - 1) == 3 and status(ws=p["ws"] + 4) == 3
    assert bsp.dense_pa_workspace_bytes(16, 2, 3, 4) == 0 and bsp.dense_pa_workspace_bytes(16, 2, 16, 9) == 0
    assert bsp.launch_count() == n0


def test_the_binding_refuses_other_dtypes_devices_and_strides(bsp):
    cpu, other = torch.device("cpu"), torch.device("cuda", 1)
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    assert bsp._dense("x", x, torch.bfloat16, cpu, 4 * 2 * 128) == x.data_ptr() and bsp._dense("x", None, None, cpu) is None
    with pytest.raises(ValueError, match="dtype"):
        bsp._dense("x", x, torch.int32, cpu)
    with pytest.raises(ValueError, match="contiguous"):
        bsp._dense("x", x[:, ::2], torch.bfloat16, cpu)
    with pytest.raises(ValueError, match="needed"):
        bsp._dense("x", x, torch.bfloat16, cpu, 4 * 2 * 128 + 1)
    with pytest.raises(ValueError, match="stream"):
        bsp._dense("x", x, torch.bfloat16, other)
    wide = torch.zeros(4, 4, 128, dtype=torch.bfloat16)
    assert bsp._head_rows("x", wide[:, 1:3], 4, 2, cpu) == (wide.data_ptr() + 256, 512)
    assert bsp._head_rows("x", wide[2:3, :1], 1, 1, cpu)[1] == 128 and bsp._head_rows("x", None, 4, 2, cpu) == (None, 0)
    with pytest.raises(ValueError, match="side by side"):
        bsp._head_rows("x", wide[:, ::2], 4, 2, cpu)
    with pytest.raises(ValueError, match="bf16"):
        bsp._head_rows("x", torch.zeros(4, 4, 64, dtype=torch.bfloat16), 4, 4, cpu)
    with pytest.raises(ValueError, match="bf16"):
        bsp._head_rows("x", x, 4, 3, cpu)
    with pytest.raises(ValueError, match="stream"):
        bsp._head_rows("x", x, 4, 2, other)
