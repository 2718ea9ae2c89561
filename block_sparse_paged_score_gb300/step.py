"""One decode step of the sparse path as a single library call.

DecodeStep owns the step's caller-side buffers (row lengths, score rows,
selections, output, split-K workspace, error word) for a fixed batch shape and
runs ``bsp_sparse_decode_step`` -- write the new tokens, cast the queries to
e4m3 where the workload attends or scores in e4m3, row lengths, index
scores, top-k with the emitted sparse table, split-K attention and merge --
on one stream, without host synchronisation.

``HostDecodeStep`` is the end-to-end form a serving loop uses: the step's
inputs arrive in pinned host memory and its attention output must land
there.  Each direction either crosses by one copy-engine copy or is read or
written in place by the step's kernels (zero-copy).  ``MixedStep`` is the
chunked-prefill batch (decode rows first, then prefill chunks and pad rows)
as separate calls on one stream.

``StepTables``, ``NormRopeWrite`` and ``DenseStep`` are the step of a layer
without an indexer over a 4-bit cache, from the requests' lengths and the
projections' rows to the attention output: the block table and slot map, the
norms and rotation with the cache write, and the dense attention.
``StepTables`` and ``NormRopeWrite`` serve layers with an indexer as well.
``ScaledPromptStep`` and ``ScaledDecodeStep`` are the steps of such a layer over
an 8-bit cache with a scale for each block and head: prompts, or chunks of them
over what the cache holds, and decode tokens.
"""
import ctypes as C

import torch

from . import bsp


class DecodeStep:
    """select_in_scorer: hand the step a zeroed counter per (sequence, index
    head) so that the scorer's last CTA of each sequence selects its rows
    (where the library supports it; the outputs are the same, the step is
    slower on the benchmark workloads, so it is off by default)."""

    def __init__(self, w, kv, idx, block_table, device="cuda", flags=bsp.FORCE_TAIL, select_in_scorer=False):
        self.w = w
        self.kv, self.idx = kv, idx
        self.block_table = block_table
        tokens, rows = w.num_decode_tokens, w.num_decode_tokens * w.hkv
        self.tokens, self.rows = tokens, rows
        e = lambda *s, dt=torch.int32: torch.empty(s, dtype=dt, device=device)  # noqa: E731
        self.row_seq, self.row_len = e(rows), e(rows)
        self.scores = e(rows, w.max_pages, dt=torch.float32)
        self.topk_idx, self.sparse_bt, self.sparse_ctx = e(rows, w.k_pages), e(rows, w.k_pages), e(rows)
        self.out = e(tokens, w.hq, 128, dt=torch.bfloat16)
        self.q_cast = e(tokens, w.hq, 128, dt=torch.uint8)
        self.idx_q_cast = e(tokens, w.hidx, 128, dt=torch.uint8)
        self.ws = bsp.decode_workspace(rows, w.k_pages, w.group, device)
        self.dev_err = torch.zeros(1, dtype=torch.int32, device=device)
        self.args = bsp.DecodeStepArgs()
        a = self.args
        a.kv = C.pointer(kv.desc)
        a.idx = C.pointer(idx.desc)
        a.q_dtype, a.idx_q_dtype = w.q_dtype, w.idx_q_dtype
        a.q_cast, a.idx_q_cast = self.q_cast.data_ptr(), self.idx_q_cast.data_ptr()
        a.num_q_heads = w.hq
        a.num_seqs, a.q_len = w.num_decode, w.q_len
        a.block_table, a.bt_stride = block_table.data_ptr(), block_table.shape[1]
        a.max_pages, a.k_pages, a.flags, a.sm_scale = w.max_pages, w.k_pages, flags, w.sm_scale
        a.row_seq, a.row_len, a.scores = self.row_seq.data_ptr(), self.row_len.data_ptr(), self.scores.data_ptr()
        a.topk_idx, a.sparse_bt, a.sparse_ctx = (self.topk_idx.data_ptr(), self.sparse_bt.data_ptr(),
                                                 self.sparse_ctx.data_ptr())
        a.out, a.ws, a.ws_bytes, a.dev_err = self.out.data_ptr(), self.ws.data_ptr(), self.ws.numel(), \
            self.dev_err.data_ptr()
        self.sel_counters = torch.zeros(max(1, w.num_decode * w.hidx), dtype=torch.int32, device=device)
        a.sel_counters = self.sel_counters.data_ptr() if select_in_scorer else None

    def run(self, k_new, v_new, idx_k_new, slot, q, idx_q, seq_lens, events=None, stream=None):
        """Device tensors in; fills self.out (and the intermediate buffers)."""
        a = self.args
        a.k_new, a.v_new, a.idx_k_new, a.slot = (k_new.data_ptr(), v_new.data_ptr(), idx_k_new.data_ptr(),
                                                 slot.data_ptr())
        a.num_new_tokens = slot.numel()
        a.q, a.idx_q, a.seq_lens = q.data_ptr(), idx_q.data_ptr(), seq_lens.data_ptr()
        bsp.sparse_decode_step(a, events=events, stream=stream)
        return self.out


class HostDecodeStep:
    """End-to-end step: pinned host inputs -> device -> step -> host output.

    The step's inputs sit back to back (256-byte aligned) in one pinned host
    buffer.  `inputs` and `output` each choose how the bytes cross the link:
      "copy": one copy-engine copy (host-to-device of all the inputs, or
              device-to-host of the attention output) on the step's stream;
      "zero": no copy -- the step's kernels load the inputs straight from the
              pinned buffer, or the attention stores its output straight
              into pinned host memory (pinned memory is mapped into the
              device's address space; on a Grace-Blackwell node these loads
              and stores cross NVLink-C2C).
    zero_copy=True is inputs="zero", output="zero".  Works for a DecodeStep
    and for a MixedStep."""

    def __init__(self, step, host_inputs, device="cuda", zero_copy=False, inputs=None, output=None):
        self.step = step
        self.inputs = inputs or ("zero" if zero_copy else "copy")
        self.output = output or ("zero" if zero_copy else "copy")
        if "zero" in (self.inputs, self.output) and not isinstance(step, (DecodeStep, MixedStep)):
            raise ValueError("zero-copy transfer needs a DecodeStep or a MixedStep")
        offs, total = {}, 0
        for k, v in host_inputs.items():
            offs[k] = total
            total += (v.numel() * v.element_size() + 255) // 256 * 256
        self.nbytes = total
        self.host_buf = torch.empty(total, dtype=torch.uint8).pin_memory()
        self.dev_buf = torch.empty(total, dtype=torch.uint8, device=device)
        self.dev, self.host = {}, {}
        for k, v in host_inputs.items():
            n = v.numel() * v.element_size()
            self.host_buf[offs[k]:offs[k] + n].copy_(v.contiguous().view(-1).view(torch.uint8))
            self.dev[k] = self.dev_buf[offs[k]:offs[k] + n].view(v.dtype).view(v.shape)
            self.host[k] = self.host_buf[offs[k]:offs[k] + n].view(v.dtype).view(v.shape)
        self.out_host = torch.empty(step.out.shape, dtype=step.out.dtype).pin_memory()

    @property
    def h2d_bytes(self):
        return self.nbytes

    @property
    def d2h_bytes(self):
        return self.out_host.numel() * self.out_host.element_size()

    def run(self, stream=None):
        s = stream if stream is not None else torch.cuda.current_stream()
        with torch.cuda.stream(s):
            if self.inputs == "copy":
                self.dev_buf.copy_(self.host_buf, non_blocking=True)
            d = self.dev if self.inputs == "copy" else self.host
            if self.output == "zero" and isinstance(self.step, MixedStep):
                # the step's attention launches store into the pinned output
                dev_out = self.step.out
                self.step.out = self.out_host
                try:
                    self.step.run(d["k"], d["v"], d["idx_k"], d["slot"], d["q"], d["idx_q"], d["seq_lens"], stream=s)
                finally:
                    self.step.out = dev_out
            elif self.output == "zero":
                a = self.step.args
                dev_out = a.out
                a.out = self.out_host.data_ptr()
                try:
                    self.step.run(d["k"], d["v"], d["idx_k"], d["slot"], d["q"], d["idx_q"], d["seq_lens"], stream=s)
                finally:
                    a.out = dev_out
            else:
                self.step.run(d["k"], d["v"], d["idx_k"], d["slot"], d["q"], d["idx_q"], d["seq_lens"], stream=s)
                self.out_host.copy_(self.step.out, non_blocking=True)
        return self.out_host


class MixedStep:
    """A chunked-prefill batch: decode rows first, then prefill chunks and pad
    rows (the vLLM forward's decode-first order).  Decode rows score on the
    mma.sync scorer and attend with split-K; prefill rows score on the tcgen05
    scorer and attend plan-free.  Same run() signature as DecodeStep; `events`
    (5 torch events) mark the same phases."""

    def __init__(self, w, kv, idx, block_table, device="cuda", flags=bsp.FORCE_TAIL):
        self.w, self.kv, self.idx, self.block_table = w, kv, idx, block_table
        self.flags = flags
        T, rows = w.num_tokens, w.num_rows
        self.nd_tok, self.nd = w.num_decode_tokens, w.num_decode_rows
        e = lambda *s, dt=torch.int32: torch.empty(s, dtype=dt, device=device)  # noqa: E731
        self.scores = e(rows, w.max_pages, dt=torch.float32)
        self.topk_idx, self.sparse_bt, self.sparse_ctx = e(rows, w.k_pages), e(rows, w.k_pages), e(rows)
        self.out = e(T, w.hq, 128, dt=torch.bfloat16)
        self.q_cast = e(T, w.hq, 128, dt=torch.uint8)
        self.idx_q_cast = e(T, w.hidx, 128, dt=torch.uint8)
        self.row_seq, self.row_len = e(rows), e(rows)
        self.ws = bsp.decode_workspace(max(self.nd, 1), w.k_pages, w.group, device)
        self.dev_err = torch.zeros(1, dtype=torch.int32, device=device)
        self.query_req_id = torch.from_numpy(w.query_req_id).to(device)
        self.query_abs_pos = torch.from_numpy(w.query_abs_pos).to(device)
        self.cu = torch.from_numpy(w.cu_prefill).to(device)
        self.num_chunks = len(w.cu_prefill) - 1
        self.max_tiles = bsp.prefill_tiles(w.cu_prefill)

    def run(self, k_new, v_new, idx_k_new, slot, q, idx_q, seq_lens, events=None, stream=None):
        w, nd, ndt = self.w, self.nd, self.nd_tok
        s = stream if stream is not None else torch.cuda.current_stream()
        mark = (lambda i: events[i].record(s)) if events is not None else (lambda i: None)  # noqa: E731
        mark(0)
        bsp.kv_page_write(self.kv, self.idx, k_new, v_new, idx_k_new, slot, self.dev_err, s)
        if w.q_dtype == bsp.FP8_E4M3:
            q = bsp.cast_e4m3(q, self.q_cast, s)
        if w.idx_q_dtype == bsp.FP8_E4M3:
            idx_q = bsp.cast_e4m3(idx_q, self.idx_q_cast, s)
        bsp.row_lengths_decode(seq_lens, w.q_len, w.hkv, self.row_seq[:nd], self.row_len[:nd], s)
        bsp.row_lengths_prefill(self.query_req_id, self.query_abs_pos, w.hkv, self.row_seq[nd:], self.row_len[nd:], s)
        mark(1)
        if nd:
            bsp.index_score(self.idx, idx_q[:ndt], w.idx_q_dtype, self.block_table, self.row_seq[:nd],
                            self.row_len[:nd], w.q_len, w.max_pages, self.scores[:nd], self.dev_err, s)
        bsp.index_score_prefill(self.idx, idx_q[ndt:], w.idx_q_dtype, self.block_table, self.row_seq[nd:],
                                self.row_len[nd:], self.cu, self.num_chunks, self.max_tiles, w.max_pages,
                                self.scores[nd:], self.dev_err, s)
        mark(2)
        bsp.topk_select(self.scores, self.row_seq, self.row_len, self.block_table, w.kv_dtype, w.k_pages,
                        self.flags, self.topk_idx, self.sparse_bt, self.sparse_ctx, s)
        mark(3)
        if nd:
            bsp.sparse_pa_decode(self.kv, q[:ndt], w.q_dtype, w.hq, self.sparse_bt[:nd], self.sparse_ctx[:nd],
                                 w.k_pages, w.sm_scale, self.out[:ndt], self.ws, self.dev_err, s)
        bsp.sparse_pa_prefill(self.kv, q[ndt:], w.q_dtype, w.hq, self.sparse_bt[nd:], self.sparse_ctx[nd:],
                              w.k_pages, w.sm_scale, self.out[ndt:], self.dev_err, s)
        mark(4)
        return self.out


class StepTables:
    """Block table, slot map and positions of a step, built on the GPU from
    the requests' lengths (bsp_step_tables).  Owns the outputs: block_table
    [num_seqs, bt_stride] (kept from step to step; entries of blocks that hold
    no tokens are -1 at first, or block_table is the caller's), seq_lens,
    cu_tokens, blocks_taken, and slot, query_req_id, query_abs_pos of
    token_capacity rows, the last of them pad rows where the step has fewer
    tokens; dev_err is the caller's error word (None: one of its own)."""

    def __init__(self, num_seqs, bt_stride, token_capacity, num_blocks, block_table=None, device="cuda", dev_err=None):
        e = lambda n, dt=torch.int32: torch.empty(n, dtype=dt, device=device)  # noqa: E731
        self.num_seqs, self.token_capacity = num_seqs, token_capacity
        if block_table is None:
            block_table = torch.full((num_seqs, bt_stride), -1, dtype=torch.int32, device=device)
        if tuple(block_table.shape) != (num_seqs, bt_stride):
            raise ValueError(f"block_table is not [{num_seqs}, {bt_stride}]")
        self.block_table = block_table
        self.seq_lens, self.cu_tokens, self.blocks_taken = e(num_seqs), e(num_seqs + 1), e(1)
        self.slot = e(token_capacity, torch.int64)
        self.query_req_id, self.query_abs_pos = e(token_capacity), e(token_capacity)
        self.dev_err = dev_err if dev_err is not None else torch.zeros(1, dtype=torch.int32, device=device)
        a = self.args = bsp.StepTablesArgs()
        a.num_seqs, a.bt_stride, a.token_capacity, a.num_blocks = num_seqs, bt_stride, token_capacity, num_blocks
        a.block_table = bsp._dense("block_table", block_table, torch.int32, self.seq_lens.device)
        a.seq_lens, a.cu_tokens, a.blocks_taken = (self.seq_lens.data_ptr(), self.cu_tokens.data_ptr(),
                                                   self.blocks_taken.data_ptr())
        a.slot, a.query_req_id, a.query_abs_pos = (self.slot.data_ptr(), self.query_req_id.data_ptr(),
                                                   self.query_abs_pos.data_ptr())
        a.dev_err = bsp._dense("dev_err", self.dev_err, torch.int32, self.seq_lens.device, 1)

    def run(self, context_lens, new_lens, free_blocks, free_head=None, stream=None):
        """int32 lengths [num_seqs] before the step and of the step, the free
        block ids, and how many of them were taken before (a device scalar;
        None: 0); fills the outputs."""
        s = bsp._on(stream)
        a, i32, dev = self.args, torch.int32, s.device
        if self.seq_lens.device != dev:
            raise ValueError(f"the tables are on {self.seq_lens.device}, the stream on {dev}")
        a.context_lens = bsp._dense("context_lens", context_lens, i32, dev, self.num_seqs)
        a.new_lens = bsp._dense("new_lens", new_lens, i32, dev, self.num_seqs)
        a.free_blocks, a.num_free = bsp._dense("free_blocks", free_blocks, i32, dev), free_blocks.numel()
        a.free_head = bsp._dense("free_head", free_head, i32, dev, 1)
        bsp.step_tables(a, s)
        return self


class NormRopeWrite:
    """Norms, position rotation and cache write of a step's projections
    (bsp_norm_rope_write) for up to max_tokens tokens.  kv and idx are the
    caches (idx None: a layer without an indexer; kv None: queries and index
    keys alone, or with k_out_heads the keys of that many heads too, as bf16 rows
    in k_out).  Weights are bf16 [128] or None; rope_table is fp32
    [positions, rot_dim], cosines then sines (see rope_table), or None; dev_err is
    the caller's error word (None: one of its own)."""

    def __init__(self, kv, idx, num_q_heads, max_tokens, q_weight=None, k_weight=None, idx_q_weight=None,
                 idx_k_weight=None, weight_offset=0.0, eps=1e-6, rope_table=None, rope_pairs=False, q_dtype=bsp.BF16,
                 idx_q_dtype=bsp.BF16, device="cuda", dev_err=None, k_out_heads=0):
        if k_out_heads and kv is not None:
            raise ValueError("the keys go to the cache or to k_out")
        self.kv, self.idx, self.max_tokens = kv, idx, max_tokens
        a = self.args = bsp.NormRopeArgs()
        self.q_out = torch.empty(max_tokens, num_q_heads, 128, device=device,
                                 dtype=torch.uint8 if q_dtype == bsp.FP8_E4M3 else torch.bfloat16)
        self.idx_q_out = None
        self.dev_err = dev_err if dev_err is not None else torch.zeros(1, dtype=torch.int32, device=device)
        dev = self.device = self.q_out.device
        bsp._cache_desc("K/V", kv, dev), bsp._cache_desc("index", idx, dev)
        self.heads = (num_q_heads, kv.num_kv_heads if kv is not None else k_out_heads,
                      idx.num_heads if idx is not None else 0)
        a.num_q_heads, a.q_out_dtype, a.idx_q_out_dtype = num_q_heads, q_dtype, idx_q_dtype
        if kv is not None:
            a.kv, a.num_kv_heads = C.pointer(kv.desc), kv.num_kv_heads
        self.k_out = None
        if k_out_heads:
            self.k_out = torch.empty(max_tokens, k_out_heads, 128, dtype=torch.bfloat16, device=device)
            a.k_out, a.num_kv_heads = self.k_out.data_ptr(), k_out_heads
        if idx is not None:
            a.idx, a.num_idx_heads = C.pointer(idx.desc), idx.num_heads
            self.idx_q_out = torch.empty(max_tokens, idx.num_heads, 128, device=device,
                                         dtype=torch.uint8 if idx_q_dtype == bsp.FP8_E4M3 else torch.bfloat16)
        self.weights = (q_weight, k_weight, idx_q_weight, idx_k_weight)
        a.q_weight, a.k_weight, a.idx_q_weight, a.idx_k_weight = (
            bsp._dense("weight", w, torch.bfloat16, dev, 128) for w in self.weights)
        a.weight_offset, a.eps = weight_offset, eps
        self.rope_table = rope_table
        if rope_table is not None:
            a.rope_table = bsp._dense("rope_table", rope_table, torch.float32, dev)
            a.rope_rows, a.rot_dim = rope_table.shape
            a.rope_pairs = int(rope_pairs)
        a.dev_err = bsp._dense("dev_err", self.dev_err, torch.int32, dev, 1)
        a.q_out = self.q_out.data_ptr()

    def run(self, q, k, v, idx_q, idx_k, positions, slot, stream=None):
        """bf16 rows [T, heads, 128] (heads side by side, tokens any distance
        apart; idx_q and idx_k None without an index cache), int32 positions
        and int64 slots [T] (None without a cache); returns the queries and index
        queries (views of the object's buffers)."""
        s = bsp._on(stream)
        a, dev, rows = self.args, self.device, bsp._head_rows
        T = q.shape[0]
        if T > self.max_tokens:
            raise ValueError(f"{T} tokens, the buffers hold {self.max_tokens}")
        if s.device != dev:
            raise ValueError(f"the buffers are on {dev}, the stream on {s.device}")
        has_idx_q = idx_q is not None and self.idx_q_out is not None
        if T == 0:  # (empty tensors have no address)
            return self.q_out[:0], self.idx_q_out[:0] if has_idx_q else None
        hq, hkv, hidx = self.heads
        a.num_tokens = T
        a.q, a.q_stride = rows("q", q, T, hq, dev)
        a.k, a.k_stride = rows("k", k, T, hkv, dev)
        a.v, a.v_stride = rows("v", v, T, hkv, dev)
        a.idx_q, a.idx_q_stride = rows("idx_q", idx_q, T, hidx, dev)
        a.idx_k, a.idx_k_stride = rows("idx_k", idx_k, T, hidx, dev)
        a.positions = bsp._dense("positions", positions, torch.int32, dev, T)
        a.slot = bsp._dense("slot", slot, torch.int64, dev, T)
        a.idx_q_out = self.idx_q_out.data_ptr() if has_idx_q else None
        bsp.norm_rope_write(a, s)
        if T == self.max_tokens:
            return self.q_out, self.idx_q_out if has_idx_q else None
        return self.q_out[:T], self.idx_q_out[:T] if has_idx_q else None


def rope_table(positions, rot_dim, theta=10000.0, device="cuda"):
    """fp32 [positions, rot_dim]: cosines, then sines, of P * theta^(-2i/rot_dim)
    (angles in fp64: at far positions fp32 ones would be off by whole turns' parts)."""
    h = rot_dim // 2
    inv = float(theta) ** (-torch.arange(h, dtype=torch.float64, device=device) / h)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], 1).float()


class DenseStep:
    """One step of a layer without an indexer over an MXFP4 cache, from the
    requests' lengths to the attention output: the step's tables, norms and
    rotation with the cache write, row lengths, dense attention.  Every
    request brings q_len tokens (1..8) or none; batches padded to num_seqs
    have requests of context 0 and no tokens.  dev_err collects the error bits of
    all its calls."""

    def __init__(self, kv, num_q_heads, num_seqs, q_len, bt_stride, sm_scale=None, q_dtype=bsp.FP8_E4M3,
                 device="cuda", **norm):
        tokens = num_seqs * q_len
        self.kv, self.q_len, self.num_q_heads, self.sm_scale, self.q_dtype = kv, q_len, num_q_heads, sm_scale, q_dtype
        self.dev_err = torch.zeros(1, dtype=torch.int32, device=device)
        self.tables = StepTables(num_seqs, bt_stride, tokens, kv.num_blocks, device=device, dev_err=self.dev_err)
        self.norm = NormRopeWrite(kv, None, num_q_heads, tokens, q_dtype=q_dtype, device=device, dev_err=self.dev_err,
                                  **norm)
        rows = tokens * kv.num_kv_heads
        self.row_seq = torch.empty(rows, dtype=torch.int32, device=device)
        self.row_len = torch.empty(rows, dtype=torch.int32, device=device)
        self.ws = bsp.dense_pa_workspace(rows, kv.num_kv_heads, num_q_heads // kv.num_kv_heads, q_len, device)
        self.out = torch.empty(tokens, num_q_heads, 128, dtype=torch.bfloat16, device=device)

    def run(self, context_lens, new_lens, free_blocks, free_head, q, k, v, stream=None):
        """Lengths and free blocks as in StepTables.run; q, k, v bf16 rows of
        the step's tokens (num_seqs * q_len rows, pad rows last).  Returns the
        attention output; a request's rows are consecutive from
        tables.cu_tokens, pad rows are zero."""
        t = self.tables.run(context_lens, new_lens, free_blocks, free_head, stream=stream)
        qr, _ = self.norm.run(q, k, v, None, None, t.query_abs_pos, t.slot, stream=stream)
        bsp.row_lengths_prefill(t.query_req_id, t.query_abs_pos, self.kv.num_kv_heads, self.row_seq, self.row_len,
                                stream=stream)
        return bsp.dense_pa_decode(self.kv, qr, self.q_dtype, self.num_q_heads, t.block_table, self.row_seq,
                                   self.row_len, self.q_len, sm_scale=self.sm_scale, out=self.out, ws=self.ws,
                                   dev_err=self.dev_err, stream=stream)


class _ScaledStep:
    """What prompt and decode steps over a BlockScaledKvCache share: the step's
    tables, norms and rotation, and the write of the new tokens."""

    def __init__(self, cache, num_q_heads, num_seqs, token_capacity, bt_stride, sm_scale, q_dtype, block_table, device,
                 norm):
        self.cache, self.num_q_heads, self.sm_scale, self.q_dtype = cache, num_q_heads, sm_scale, q_dtype
        self.group = num_q_heads // cache.num_kv_heads
        self.dev_err = torch.zeros(1, dtype=torch.int32, device=device)
        self.tables = StepTables(num_seqs, bt_stride, token_capacity, cache.num_blocks, block_table, device=device,
                                 dev_err=self.dev_err)
        self.norm = NormRopeWrite(None, None, num_q_heads, token_capacity, q_dtype=q_dtype, device=device,
                                  dev_err=self.dev_err, k_out_heads=cache.num_kv_heads, **norm)
        self.out = torch.zeros(token_capacity, num_q_heads, 128, dtype=torch.bfloat16, device=device)

    def _write(self, context_lens, new_lens, free_blocks, free_head, q, k, v, stream):
        t = self.tables.run(context_lens, new_lens, free_blocks, free_head, stream=stream)
        T = q.shape[0]
        qr, _ = self.norm.run(q, k, None, None, None, t.query_abs_pos[:T], None, stream=stream)
        kr = self.norm.k_out[:T]
        bsp.kv_scaled_write(self.cache, kr, v, t.slot[:T], dev_err=self.dev_err, stream=stream)
        return qr, kr


class ScaledPromptStep(_ScaledStep):
    """Prompts of a layer without an indexer, from the requests' lengths to the
    attention output: the step's tables, norms and rotation, the write into a
    BlockScaledKvCache, causal attention.  A request brings any number of tokens.
    With key_capacity 0 every request is new (run's context_lens is None), and its
    queries see the step's own bf16 rows.  Else they see all of their request's tokens
    as the cache holds them, read back into key_capacity rows: a chunk over its
    context sees what its decode steps will.  block_table is the requests' (None: one
    of its own); dev_err collects the error bits of all calls."""

    def __init__(self, cache, num_q_heads, num_seqs, token_capacity, bt_stride, key_capacity=0, sm_scale=None,
                 block_table=None, device="cuda", **norm):
        super().__init__(cache, num_q_heads, num_seqs, token_capacity, bt_stride, sm_scale, bsp.BF16, block_table,
                         device, norm)
        hkv = cache.num_kv_heads
        self.key_capacity = key_capacity
        if not key_capacity:
            self.no_context = torch.zeros(num_seqs, dtype=torch.int32, device=device)
        else:
            e = lambda: torch.empty(key_capacity, hkv, 128, dtype=torch.bfloat16, device=device)  # noqa: E731
            self.k, self.v = e(), e()
            self.key = torch.arange(key_capacity, dtype=torch.int32, device=device)
            self.cu_k = torch.zeros(num_seqs + 1, dtype=torch.int32, device=device)
        self.ws = bsp.prompt_attention_workspace(token_capacity, num_seqs, hkv, self.group, device)

    def _key_slots(self, new_lens):
        """Slots of all tokens of the requests that have new ones, one request
        behind the other (-1 behind the last), and their offsets into cu_k."""
        t, n = self.tables, self.tables.num_seqs
        lens = torch.where(new_lens > 0, t.seq_lens, 0)
        torch.cumsum(lens, 0, dtype=torch.int32, out=self.cu_k[1:])
        seq = torch.searchsorted(self.cu_k[1:], self.key, right=True)
        live = seq < n
        seq = seq.clamp(max=n - 1)
        pos = torch.where(live, self.key - self.cu_k[seq], 0)
        block = t.block_table[seq, (pos // 128).clamp(max=t.block_table.shape[1] - 1)].long()
        return torch.where(live & (block >= 0), block * 128 + pos % 128, -1)

    def run(self, context_lens, new_lens, free_blocks, free_head, q, k, v, stream=None):
        """Lengths and free blocks as in StepTables.run; q, k, v bf16 rows of the
        step's tokens, any pad rows last.  Returns the attention output; a request's
        rows are consecutive from tables.cu_tokens, rows of no request are
        unspecified."""
        if (context_lens is None) != (self.key_capacity == 0):
            raise ValueError("contexts need key_capacity, and only they do")
        if context_lens is None:
            context_lens = self.no_context
        s = bsp._on(stream)
        qr, kr = self._write(context_lens, new_lens, free_blocks, free_head, q, k, v, s)
        T, cu_q, cu_k = q.shape[0], self.tables.cu_tokens, None
        if self.key_capacity:
            with torch.cuda.stream(stream):
                slot = self._key_slots(new_lens)
            kr, v = bsp.kv_scaled_read(self.cache, slot, self.k, self.v, dev_err=self.dev_err, stream=s)
            cu_k = self.cu_k
        return bsp.prompt_attention(qr, kr, v, cu_q, cu_k, sm_scale=self.sm_scale, out=self.out[:T], ws=self.ws,
                                    dev_err=self.dev_err, stream=s)


class ScaledDecodeStep(_ScaledStep):
    """Decode tokens of a layer without an indexer over a BlockScaledKvCache: as
    DenseStep, every request brings q_len tokens (1..8) or none.  block_table is
    the requests' (None: one of its own)."""

    def __init__(self, cache, num_q_heads, num_seqs, q_len, bt_stride, sm_scale=None, q_dtype=bsp.BF16,
                 block_table=None, device="cuda", **norm):
        tokens = num_seqs * q_len
        super().__init__(cache, num_q_heads, num_seqs, tokens, bt_stride, sm_scale, q_dtype, block_table, device, norm)
        self.q_len = q_len
        rows = tokens * cache.num_kv_heads
        self.row_seq = torch.empty(rows, dtype=torch.int32, device=device)
        self.row_len = torch.empty(rows, dtype=torch.int32, device=device)
        self.ws = bsp.dense_pa_fp8_workspace(rows, cache.num_kv_heads, self.group, q_len, device)

    def run(self, context_lens, new_lens, free_blocks, free_head, q, k, v, stream=None):
        """As DenseStep.run: num_seqs * q_len rows, pad rows last; pad rows of the
        output are zero."""
        t, s = self.tables, bsp._on(stream)
        qr, _ = self._write(context_lens, new_lens, free_blocks, free_head, q, k, v, s)
        bsp.row_lengths_prefill(t.query_req_id, t.query_abs_pos, self.cache.num_kv_heads, self.row_seq, self.row_len,
                                stream=s)
        return bsp.dense_pa_decode_fp8(self.cache, qr, self.q_dtype, self.num_q_heads, t.block_table, self.row_seq,
                                       self.row_len, self.q_len, sm_scale=self.sm_scale, out=self.out, ws=self.ws,
                                       dev_err=self.dev_err, stream=s)
