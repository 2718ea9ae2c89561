"""ctypes binding of libbsp (include/bsp.h).

Argument marshalling only: every step runs in the library's CUDA kernels.
Tensors are torch CUDA tensors; the stream is torch's current stream unless
one is given.  Outputs and workspaces that a call makes itself come from its
stream's memory pool; whoever uses such an output on another stream orders the
two, as for any tensor made on a side stream.  A call whose library is missing
raises -- there is no CPU fallback.
"""
import ctypes as C
import math
import os

import torch

from . import build as _build

BF16, FP8_E4M3, MXFP4 = 0, 1, 2
FORCE_TAIL = 1
REUSE_SELECTION = 2  # decode step: attend with another layer's sparse_bt / sparse_ctx
SELECT_BLOCKS = 4  # top-k: 128-token blocks are the unit of selection
DEVERR = {1: "page id", 2: "block id", 4: "group sequence", 8: "timeout", 16: "slot", 32: "capacity", 64: "position"}
STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "workspace too small", 4: "CUDA error"}


class BspError(RuntimeError):
    def __init__(self, fn, status):
        super().__init__(f"{fn}: {STATUS.get(status, status)} (status {status})")
        self.status = status


class KvCacheDesc(C.Structure):
    _fields_ = [("dtype", C.c_int32), ("num_kv_heads", C.c_int32), ("k_base", C.c_void_p), ("v_base", C.c_void_p),
                ("id_stride_bytes", C.c_int64), ("num_ids", C.c_int64), ("num_blocks", C.c_int64),
                ("k_scale", C.c_float), ("v_scale", C.c_float)]


class IndexCacheDesc(C.Structure):
    _fields_ = [("dtype", C.c_int32), ("num_heads", C.c_int32), ("base", C.c_void_p),
                ("block_stride_bytes", C.c_int64), ("num_blocks", C.c_int64)]


class DecodeStepArgs(C.Structure):
    _fields_ = [("kv", C.POINTER(KvCacheDesc)), ("idx", C.POINTER(IndexCacheDesc)),
                ("k_new", C.c_void_p), ("v_new", C.c_void_p), ("idx_k_new", C.c_void_p), ("slot", C.c_void_p),
                ("num_new_tokens", C.c_int32),
                ("q", C.c_void_p), ("q_dtype", C.c_int32), ("q_cast", C.c_void_p), ("num_q_heads", C.c_int32),
                ("idx_q", C.c_void_p), ("idx_q_dtype", C.c_int32), ("idx_q_cast", C.c_void_p),
                ("seq_lens", C.c_void_p), ("num_seqs", C.c_int32), ("q_len", C.c_int32),
                ("block_table", C.c_void_p), ("bt_stride", C.c_int32), ("max_pages", C.c_int32),
                ("k_pages", C.c_int32), ("flags", C.c_int32), ("sm_scale", C.c_float),
                ("row_seq", C.c_void_p), ("row_len", C.c_void_p), ("scores", C.c_void_p), ("topk_idx", C.c_void_p),
                ("sparse_bt", C.c_void_p), ("sparse_ctx", C.c_void_p), ("out", C.c_void_p), ("ws", C.c_void_p),
                ("ws_bytes", C.c_size_t), ("dev_err", C.c_void_p), ("sel_counters", C.c_void_p)]


class StepTablesArgs(C.Structure):
    _fields_ = [("context_lens", C.c_void_p), ("new_lens", C.c_void_p), ("num_seqs", C.c_int32),
                ("bt_stride", C.c_int32), ("block_table", C.c_void_p), ("free_blocks", C.c_void_p),
                ("free_head", C.c_void_p), ("num_free", C.c_int32), ("token_capacity", C.c_int32),
                ("num_blocks", C.c_int64), ("seq_lens", C.c_void_p), ("cu_tokens", C.c_void_p),
                ("blocks_taken", C.c_void_p), ("slot", C.c_void_p), ("query_req_id", C.c_void_p),
                ("query_abs_pos", C.c_void_p), ("dev_err", C.c_void_p)]


class NormRopeArgs(C.Structure):
    _fields_ = [("q", C.c_void_p), ("k", C.c_void_p), ("v", C.c_void_p), ("idx_q", C.c_void_p),
                ("idx_k", C.c_void_p), ("q_stride", C.c_int64), ("k_stride", C.c_int64), ("v_stride", C.c_int64),
                ("idx_q_stride", C.c_int64), ("idx_k_stride", C.c_int64), ("num_tokens", C.c_int32),
                ("num_q_heads", C.c_int32), ("num_kv_heads", C.c_int32), ("num_idx_heads", C.c_int32),
                ("q_weight", C.c_void_p), ("k_weight", C.c_void_p), ("idx_q_weight", C.c_void_p),
                ("idx_k_weight", C.c_void_p), ("weight_offset", C.c_float), ("eps", C.c_float),
                ("rope_table", C.c_void_p), ("rope_rows", C.c_int64), ("rot_dim", C.c_int32),
                ("rope_pairs", C.c_int32), ("positions", C.c_void_p), ("slot", C.c_void_p), ("q_out", C.c_void_p),
                ("k_out", C.c_void_p), ("idx_q_out", C.c_void_p), ("q_out_dtype", C.c_int32),
                ("idx_q_out_dtype", C.c_int32), ("kv", C.POINTER(KvCacheDesc)), ("idx", C.POINTER(IndexCacheDesc)),
                ("dev_err", C.c_void_p)]


_lib = None
SYMBOLS = {
    "bsp_kv_cache_interleaved": [C.c_int32, C.c_int32, C.c_void_p, C.c_int64, C.c_float, C.c_float,
                                 C.POINTER(KvCacheDesc)],
    "bsp_index_cache_packed": [C.c_int32, C.c_int32, C.c_void_p, C.c_int64, C.POINTER(IndexCacheDesc)],
    "bsp_kv_page_write": [C.POINTER(KvCacheDesc), C.POINTER(IndexCacheDesc), C.c_void_p, C.c_void_p, C.c_void_p,
                          C.c_void_p, C.c_int32, C.c_void_p, C.c_void_p],
    "bsp_cast_e4m3": [C.c_void_p, C.c_void_p, C.c_int64, C.c_void_p],
    "bsp_row_lengths_decode": [C.c_void_p, C.c_int32, C.c_int32, C.c_int32, C.c_void_p, C.c_void_p, C.c_void_p],
    "bsp_row_lengths_prefill": [C.c_void_p, C.c_void_p, C.c_int32, C.c_int32, C.c_void_p, C.c_void_p, C.c_void_p],
    "bsp_index_score": [C.POINTER(IndexCacheDesc), C.c_void_p, C.c_int32, C.c_void_p, C.c_int32, C.c_void_p,
                        C.c_void_p, C.c_int32, C.c_int32, C.c_int32, C.c_void_p, C.c_void_p, C.c_void_p],
    "bsp_index_score_prefill": [C.POINTER(IndexCacheDesc), C.c_void_p, C.c_int32, C.c_void_p, C.c_int32, C.c_void_p,
                                C.c_void_p, C.c_int32, C.c_void_p, C.c_int32, C.c_int32, C.c_int32, C.c_void_p,
                                C.c_void_p, C.c_void_p],
    "bsp_topk_select": [C.c_void_p, C.c_int32, C.c_int32, C.c_void_p, C.c_void_p, C.c_void_p, C.c_int32, C.c_int32,
                        C.c_int32, C.c_int32, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p],
    "bsp_sparse_pa_decode": [C.POINTER(KvCacheDesc), C.c_void_p, C.c_int32, C.c_int32, C.c_void_p, C.c_void_p,
                             C.c_int32, C.c_int32, C.c_float, C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p,
                             C.c_void_p],
    "bsp_sparse_pa_decode_noalloc": [C.POINTER(KvCacheDesc), C.c_void_p, C.c_int32, C.c_int32, C.c_void_p,
                                     C.c_void_p, C.c_int32, C.c_int32, C.c_float, C.c_void_p, C.c_void_p,
                                     C.c_void_p],
    "bsp_sparse_pa_prefill": [C.POINTER(KvCacheDesc), C.c_void_p, C.c_int32, C.c_int32, C.c_void_p, C.c_void_p,
                              C.c_int32, C.c_int32, C.c_float, C.c_void_p, C.c_void_p, C.c_void_p],
    "bsp_sparse_pa_decode_workspace_bytes": [C.c_int32, C.c_int32, C.c_int32],
    "bsp_sparse_pa_decode_splits": [C.c_int32, C.c_int32, C.c_int32],
    "bsp_sparse_decode_step": [C.POINTER(DecodeStepArgs), C.c_void_p, C.c_void_p],
    "bsp_step_tables": [C.POINTER(StepTablesArgs), C.c_void_p],
    "bsp_norm_rope_write": [C.POINTER(NormRopeArgs), C.c_void_p],
    "bsp_kv_page_read": [C.POINTER(KvCacheDesc), C.POINTER(IndexCacheDesc), C.c_void_p, C.c_int32, C.c_void_p,
                         C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p],
    "bsp_dense_pa_workspace_bytes": [C.c_int32, C.c_int32, C.c_int32, C.c_int32],
    "bsp_dense_pa_decode": [C.POINTER(KvCacheDesc), C.c_void_p, C.c_int32, C.c_int32, C.c_void_p, C.c_int32,
                            C.c_void_p, C.c_void_p, C.c_int32, C.c_int32, C.c_float, C.c_void_p, C.c_void_p,
                            C.c_size_t, C.c_void_p, C.c_void_p],
    "bsp_kv_block_bytes": [C.c_int32, C.c_int32],
    "bsp_index_field_bytes": [C.c_int32],
    "bsp_status_str": [C.c_int32],
    "bsp_last_cuda_error": [],
    "bsp_launch_count": [],
    "bsp_version": [],
}
RESTYPES = {"bsp_sparse_pa_decode_workspace_bytes": C.c_size_t, "bsp_dense_pa_workspace_bytes": C.c_size_t,
            "bsp_kv_block_bytes": C.c_int64,
            "bsp_index_field_bytes": C.c_int64, "bsp_status_str": C.c_char_p, "bsp_launch_count": C.c_int64}


def library_path():
    return _build.LIB


def lib(build_if_missing=True):
    """Load libbsp.so (building it first when the CUDA toolkit is here)."""
    global _lib
    if _lib is None:
        path = _build.LIB
        if build_if_missing:
            path = _build.build()
        if not os.path.exists(path):
            raise RuntimeError(f"libbsp.so is not built ({path}); run __graft_entry__.build()")
        L = C.CDLL(path)
        for name, args in SYMBOLS.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = RESTYPES.get(name, C.c_int32)
        _lib = L
    return _lib


def _check(fn, status):
    if status != 0:
        raise BspError(fn, status)


def _ptr(t):
    """The device address of a CUDA tensor: caches, tables, lengths, score
    rows, selections and workspaces must live in device memory."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libbsp takes a CUDA tensor here (only per-token inputs and outputs may be pinned host "
                         "tensors)")
    return t.data_ptr()


def _io_ptr(t):
    """The address of a per-token input or output: a CUDA tensor, or a pinned
    host tensor (pinned memory is mapped into the device's address space;
    the kernels read or write it once, in place)."""
    if t is None:
        return None
    if not t.is_cuda and not t.is_pinned():
        raise ValueError("libbsp takes CUDA tensors or pinned host tensors")
    return t.data_ptr()


class _Current:
    """The current stream's handle and device (torch.cuda.current_stream() takes
    longer than everything else the binding does for a small call)."""
    __slots__ = ("cuda_stream", "device")
    raw = staticmethod(getattr(torch._C, "_cuda_getCurrentRawStream", None) or
                       (lambda index: torch.cuda.current_stream(index).cuda_stream))
    devices = {}

    def __init__(self):
        index = torch.cuda.current_device()
        self.cuda_stream = self.raw(index)
        self.device = self.devices.get(index) or self.devices.setdefault(index, torch.device("cuda", index))


def _on(stream):
    return stream if stream is not None else _Current()


def _stream(stream):
    return C.c_void_p(_on(stream).cuda_stream)


def _new(shape, dtype, device, stream, zeroed=False):
    """A buffer of a call's own.  From the pool of the stream the call runs on:
    memory of another stream's could still be in use there, and could be
    handed out there again while the call runs."""
    make = torch.zeros if zeroed else torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=device)


def launch_count():
    return int(lib().bsp_launch_count())


def kv_block_bytes(dtype, hkv):
    return int(lib().bsp_kv_block_bytes(dtype, hkv))


def index_field_bytes(dtype):
    return int(lib().bsp_index_field_bytes(dtype))


class KvCache:
    """An interleaved (bf16/fp8) or MXFP4 K/V cache in a caller-owned uint8 tensor."""

    def __init__(self, dtype, num_kv_heads, num_blocks, k_scale=1.0, v_scale=1.0, buffer=None, device="cuda"):
        nbytes = num_blocks * kv_block_bytes(dtype, num_kv_heads)
        self.buffer = buffer if buffer is not None else torch.zeros(nbytes, dtype=torch.uint8, device=device)
        assert self.buffer.numel() >= nbytes
        self.dtype, self.num_kv_heads, self.num_blocks = dtype, num_kv_heads, num_blocks
        self.desc = KvCacheDesc()
        _check("bsp_kv_cache_interleaved",
               lib().bsp_kv_cache_interleaved(dtype, num_kv_heads, _ptr(self.buffer), num_blocks, k_scale, v_scale,
                                              C.byref(self.desc)))


class IndexCache:
    """A packed index-key cache (one field per block and index head)."""

    def __init__(self, dtype, num_heads, num_blocks, buffer=None, device="cuda"):
        nbytes = num_blocks * num_heads * index_field_bytes(dtype)
        self.buffer = buffer if buffer is not None else torch.zeros(nbytes, dtype=torch.uint8, device=device)
        self.dtype, self.num_heads, self.num_blocks = dtype, num_heads, num_blocks
        self.desc = IndexCacheDesc()
        _check("bsp_index_cache_packed",
               lib().bsp_index_cache_packed(dtype, num_heads, _ptr(self.buffer), num_blocks, C.byref(self.desc)))


def kv_page_write(kv, idx, k, v, idx_k, slot, dev_err=None, stream=None):
    _check("bsp_kv_page_write",
           lib().bsp_kv_page_write(C.byref(kv.desc), C.byref(idx.desc) if idx is not None else None, _io_ptr(k),
                                   _io_ptr(v), _io_ptr(idx_k), _io_ptr(slot), slot.numel(), _ptr(dev_err),
                                   _stream(stream)))


def cast_e4m3(x, out=None, stream=None):
    out = out if out is not None else _new(x.shape, torch.uint8, x.device, stream)
    _check("bsp_cast_e4m3", lib().bsp_cast_e4m3(_io_ptr(x), _io_ptr(out), x.numel(), _stream(stream)))
    return out


def row_lengths_decode(seq_lens, q_len, num_heads, row_seq=None, row_len=None, stream=None):
    rows = seq_lens.numel() * q_len * num_heads
    row_seq = row_seq if row_seq is not None else _new(rows, torch.int32, seq_lens.device, stream)
    row_len = row_len if row_len is not None else _new(rows, torch.int32, seq_lens.device, stream)
    _check("bsp_row_lengths_decode", lib().bsp_row_lengths_decode(_io_ptr(seq_lens), seq_lens.numel(), q_len, num_heads,
                                                                  _ptr(row_seq), _ptr(row_len), _stream(stream)))
    return row_seq, row_len


def row_lengths_prefill(query_req_id, query_abs_pos, num_heads, row_seq=None, row_len=None, stream=None):
    rows = query_req_id.numel() * num_heads
    dev = query_req_id.device
    row_seq = row_seq if row_seq is not None else _new(rows, torch.int32, dev, stream)
    row_len = row_len if row_len is not None else _new(rows, torch.int32, dev, stream)
    _check("bsp_row_lengths_prefill",
           lib().bsp_row_lengths_prefill(_ptr(query_req_id), _ptr(query_abs_pos), query_req_id.numel(), num_heads,
                                         _ptr(row_seq), _ptr(row_len), _stream(stream)))
    return row_seq, row_len


def index_score(idx, idx_q, q_dtype, block_table, row_seq, row_len, q_group, max_pages, scores=None, dev_err=None,
                stream=None):
    rows = row_seq.numel()
    scores = scores if scores is not None else _new((rows, max_pages), torch.float32, idx_q.device, stream)
    _check("bsp_index_score",
           lib().bsp_index_score(C.byref(idx.desc), _ptr(idx_q), q_dtype, _ptr(block_table), block_table.shape[1],
                                 _ptr(row_seq), _ptr(row_len), rows, q_group, max_pages, _ptr(scores), _ptr(dev_err),
                                 _stream(stream)))
    return scores


def prefill_tiles(cu_tokens_host):
    """Host upper bound on the 128-row tiles of the prefill chunks."""
    sizes = [int(b) - int(a) for a, b in zip(cu_tokens_host[:-1], cu_tokens_host[1:])]
    return sum((s + 127) // 128 for s in sizes)


def index_score_prefill(idx, idx_q, q_dtype, block_table, row_seq, row_len, cu_tokens, num_chunks, max_tiles,
                        max_pages, scores=None, dev_err=None, stream=None):
    rows = row_seq.numel()
    scores = scores if scores is not None else _new((rows, max_pages), torch.float32, idx_q.device, stream)
    _check("bsp_index_score_prefill",
           lib().bsp_index_score_prefill(C.byref(idx.desc), _ptr(idx_q), q_dtype, _ptr(block_table),
                                         block_table.shape[1], _ptr(row_seq), _ptr(row_len), rows, _ptr(cu_tokens),
                                         num_chunks, max_tiles, max_pages, _ptr(scores), _ptr(dev_err),
                                         _stream(stream)))
    return scores


def topk_select(scores, row_seq, row_len, block_table, kv_dtype, k_pages, flags=FORCE_TAIL, topk_idx=None,
                sparse_bt=None, sparse_ctx=None, stream=None):
    rows, max_pages = scores.shape
    dev = scores.device
    topk_idx = topk_idx if topk_idx is not None else _new((rows, k_pages), torch.int32, dev, stream)
    sparse_bt = sparse_bt if sparse_bt is not None else _new((rows, k_pages), torch.int32, dev, stream)
    sparse_ctx = sparse_ctx if sparse_ctx is not None else _new(rows, torch.int32, dev, stream)
    _check("bsp_topk_select",
           lib().bsp_topk_select(_ptr(scores), rows, max_pages, _ptr(row_seq), _ptr(row_len), _ptr(block_table),
                                 block_table.shape[1], kv_dtype, k_pages, flags, _ptr(topk_idx), _ptr(sparse_bt),
                                 _ptr(sparse_ctx), _stream(stream)))
    return topk_idx, sparse_bt, sparse_ctx


def decode_workspace_bytes(num_rows, k_pages, group):
    return int(lib().bsp_sparse_pa_decode_workspace_bytes(num_rows, k_pages, group))


def decode_splits(kv_dtype, num_rows, k_pages):
    """CTAs per row of a decode attention call with these sizes (> 8: the
    splits merge through the workspace)."""
    return int(lib().bsp_sparse_pa_decode_splits(kv_dtype, num_rows, k_pages))


def decode_workspace(num_rows, k_pages, group, device="cuda", stream=None):
    """A zeroed split-K workspace (its arrival counters must start at zero)."""
    n = decode_workspace_bytes(num_rows, k_pages, group)
    return _new(max(n, 16), torch.uint8, device, stream, zeroed=True)


def sparse_pa_decode(kv, q, q_dtype, num_q_heads, sparse_bt, sparse_ctx, k_pages, sm_scale=None, out=None, ws=None,
                     dev_err=None, stream=None):
    rows = sparse_ctx.numel()
    sm_scale = sm_scale if sm_scale is not None else 1.0 / math.sqrt(128)
    out = out if out is not None else _new(q.shape, torch.bfloat16, q.device, stream)
    if ws is None:
        ws = decode_workspace(rows, k_pages, num_q_heads // kv.num_kv_heads, q.device, stream)
    _check("bsp_sparse_pa_decode",
           lib().bsp_sparse_pa_decode(C.byref(kv.desc), _io_ptr(q), q_dtype, num_q_heads, _ptr(sparse_bt),
                                      _ptr(sparse_ctx), rows, k_pages, sm_scale, _io_ptr(out), _ptr(ws), ws.numel(),
                                      _ptr(dev_err), _stream(stream)))
    return out


def sparse_pa_decode_noalloc(kv, q, q_dtype, num_q_heads, sparse_bt, sparse_ctx, k_pages, sm_scale=None, out=None,
                             dev_err=None, stream=None):
    """bsp_sparse_pa_decode without a caller workspace (the library's own
    fixed scratch; see include/bsp.h for the size limit and the sharing rule)."""
    rows = sparse_ctx.numel()
    sm_scale = sm_scale if sm_scale is not None else 1.0 / math.sqrt(128)
    out = out if out is not None else _new(q.shape, torch.bfloat16, q.device, stream)
    _check("bsp_sparse_pa_decode_noalloc",
           lib().bsp_sparse_pa_decode_noalloc(C.byref(kv.desc), _io_ptr(q), q_dtype, num_q_heads, _ptr(sparse_bt),
                                              _ptr(sparse_ctx), rows, k_pages, sm_scale, _io_ptr(out), _ptr(dev_err),
                                              _stream(stream)))
    return out


def sparse_pa_prefill(kv, q, q_dtype, num_q_heads, sparse_bt, sparse_ctx, k_pages, sm_scale=None, out=None,
                      dev_err=None, stream=None):
    rows = sparse_ctx.numel()
    sm_scale = sm_scale if sm_scale is not None else 1.0 / math.sqrt(128)
    out = out if out is not None else _new(q.shape, torch.bfloat16, q.device, stream)
    _check("bsp_sparse_pa_prefill",
           lib().bsp_sparse_pa_prefill(C.byref(kv.desc), _io_ptr(q), q_dtype, num_q_heads, _ptr(sparse_bt),
                                       _ptr(sparse_ctx), rows, k_pages, sm_scale, _io_ptr(out), _ptr(dev_err),
                                       _stream(stream)))
    return out


def sparse_decode_step(args, events=None, stream=None):
    """Run bsp_sparse_decode_step on a filled DecodeStepArgs (see DecodeStep)."""
    ev = None
    if events is not None:
        ev = (C.c_void_p * len(events))(*[e.cuda_event for e in events])
    _check("bsp_sparse_decode_step", lib().bsp_sparse_decode_step(C.byref(args), ev, _stream(stream)))


def _dense(name, t, dtype, device, numel=0):
    """The device address of a contiguous tensor of the given dtype on the
    stream's device, of at least `numel` elements (None: NULL)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.device != device or not t.is_contiguous() or t.numel() < numel:
        _complain(name, t, dtype, device, numel)
    return t.data_ptr()


def _complain(name, t, dtype, device, numel):
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the stream on {device}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} has dtype {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} is not contiguous")
    raise ValueError(f"{name} has {t.numel()} elements, {numel} are needed")


def _cache_desc(name, cache, device):
    """A reference to a cache's descriptor (None: NULL)."""
    if cache is None:
        return None
    if cache.buffer.device != device:
        raise ValueError(f"the {name} cache is on {cache.buffer.device}, the stream on {device}")
    return C.byref(cache.desc)


def _head_rows(name, t, tokens, heads, device):
    """(address, token stride) of bf16 rows [tokens, heads, 128] whose heads
    lie side by side; the tokens may be any distance apart."""
    if t is None:
        return None, 0
    if t.dtype is not torch.bfloat16 or t.shape != (tokens, heads, 128):
        raise ValueError(f"{name} is not bf16 [{tokens}, {heads}, 128]")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the stream on {device}")
    st = t.stride()
    if st[2] != 1 or (st[1] != 128 and heads > 1):
        raise ValueError(f"{name}: the heads of a token must lie side by side")
    return t.data_ptr(), st[0] if tokens > 1 else heads * 128


def step_tables(args, stream=None):
    """Run bsp_step_tables on a filled StepTablesArgs (see step.StepTables)."""
    _check("bsp_step_tables", lib().bsp_step_tables(C.byref(args), _stream(stream)))


def norm_rope_write(args, stream=None):
    """Run bsp_norm_rope_write on a filled NormRopeArgs (see step.NormRopeWrite)."""
    _check("bsp_norm_rope_write", lib().bsp_norm_rope_write(C.byref(args), _stream(stream)))


def kv_page_read(kv, idx, slot, k=None, v=None, idx_k=None, dev_err=None, stream=None):
    """Cached tokens by slot as bf16 rows: (k, v, idx_k), k and v of the K/V
    cache `kv`, idx_k of the index cache `idx`; either cache may be None."""
    s = _on(stream)
    dev = s.device
    T = slot.numel()
    kv_desc, idx_desc = _cache_desc("K/V", kv, dev), _cache_desc("index", idx, dev)
    if kv is not None:
        shape = (T, kv.num_kv_heads, 128)
        k = k if k is not None else _new(shape, torch.bfloat16, slot.device, stream)
        v = v if v is not None else _new(shape, torch.bfloat16, slot.device, stream)
    elif k is not None or v is not None:
        raise ValueError("k and v need a K/V cache")
    if idx is not None:
        shape = (T, idx.num_heads, 128)
        idx_k = idx_k if idx_k is not None else _new(shape, torch.bfloat16, slot.device, stream)
    elif idx_k is not None:
        raise ValueError("idx_k needs an index cache")
    if T == 0:  # (empty tensors have no address)
        return k, v, idx_k
    bf = torch.bfloat16
    n, ni = T * kv.num_kv_heads * 128 if kv is not None else 0, T * idx.num_heads * 128 if idx is not None else 0
    _check("bsp_kv_page_read",
           lib().bsp_kv_page_read(kv_desc, idx_desc,
                                  _dense("slot", slot, torch.int64, dev), T, _dense("k", k, bf, dev, n),
                                  _dense("v", v, bf, dev, n), _dense("idx_k", idx_k, bf, dev, ni),
                                  _dense("dev_err", dev_err, torch.int32, dev, 1), s.cuda_stream))
    return k, v, idx_k


def dense_pa_workspace_bytes(num_rows, num_kv_heads, group, q_group):
    return int(lib().bsp_dense_pa_workspace_bytes(num_rows, num_kv_heads, group, q_group))


def dense_pa_workspace(num_rows, num_kv_heads, group, q_group, device="cuda", stream=None):
    """A workspace for dense attention calls of these sizes that never overlap
    on the GPU (its contents need not be set)."""
    n = dense_pa_workspace_bytes(num_rows, num_kv_heads, group, q_group)
    return _new(max(n, 16), torch.uint8, device, stream)


def dense_pa_decode(kv, q, q_dtype, num_q_heads, block_table, row_seq, row_len, q_group, sm_scale=None, out=None,
                    ws=None, dev_err=None, stream=None):
    """Attention of each row over its whole context in an MXFP4 cache
    (bsp_dense_pa_decode); q [tokens, num_q_heads, 128], rows = tokens * Hkv."""
    s = _on(stream)
    dev, i32 = s.device, torch.int32
    desc = _cache_desc("K/V", kv, dev)
    rows, hkv = row_len.numel(), kv.num_kv_heads
    n = rows // hkv * num_q_heads * 128
    sm_scale = sm_scale if sm_scale is not None else 1.0 / math.sqrt(128)
    out = out if out is not None else _new(q.shape, torch.bfloat16, q.device, stream)
    if ws is None:
        ws = dense_pa_workspace(rows, hkv, num_q_heads // hkv, q_group, q.device, stream)
    if block_table.dim() != 2:
        raise ValueError("block_table is not [sequences, blocks]")
    # e4m3 queries may be given as the type or as bytes
    qt = torch.bfloat16 if q_dtype == BF16 else torch.float8_e4m3fn if q.dtype is torch.float8_e4m3fn else torch.uint8
    _check("bsp_dense_pa_decode",
           lib().bsp_dense_pa_decode(desc, _dense("q", q, qt, dev, n), q_dtype, num_q_heads,
                                     _dense("block_table", block_table, i32, dev), block_table.shape[1],
                                     _dense("row_seq", row_seq, i32, dev, rows), _dense("row_len", row_len, i32, dev),
                                     rows, q_group, sm_scale, _dense("out", out, torch.bfloat16, dev, n),
                                     _dense("ws", ws, torch.uint8, dev), ws.numel(),
                                     _dense("dev_err", dev_err, i32, dev, 1), s.cuda_stream))
    return out
