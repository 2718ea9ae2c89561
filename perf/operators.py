"""The operators of a decode or chunked-prefill step around the paged caches: their measured cases and plain forms.

  tables  block table, slot map and positions of a step from the requests' lengths
  norm    per-head RMS norm and position rotation of queries and keys, written straight into the K/V and index caches
  attend  dense grouped-query attention over a 4-bit (MXFP4) paged cache
  read    cached K and V gathered back by slot as bf16

``run`` computes an operator from elementary torch operations in 32 bits, or with ``own`` true by the framework's call.
"""
import math

import torch

own = False

BF16, FP8, MX = 0, 1, 2
BLK, PG, D = 128, 16, 128
MX_FIELD, MX_SCALES = 8704, 8192
K_SCALE, V_SCALE = 0.0095, 0.0105
EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ---- cases -----------------------------------------------------------------
def listed():
    return [
        # one request decoding one token: the latency of a single-user server
        dict(name="tables 1 request", op="tables", decode=1, q_len=1, prefill=0, chunk=0, pad=0, ctx=1024),
        # a chunked-prefill batch: 64 decoding requests, four 4096-token chunks, pad rows of a captured graph
        dict(name="tables 64 + 4 chunks", op="tables", decode=64, q_len=1, prefill=4, chunk=4096, pad=8, ctx=65536),
        # the widest batch: 4096 decoding requests beside sixteen chunks of 8192 tokens
        dict(name="tables 4096 + 16 chunks", op="tables", decode=4096, q_len=1, prefill=16, chunk=8192, pad=3, ctx=32768),
        # one token into a bf16 cache, all 128 dims rotated as adjacent pairs
        dict(name="norm 1 token bf16", op="norm", kv=BF16, idx=BF16, q8=False, T=1, hkv=1, group=4, rot=128, pairs=True, pad=0),
        # 64 decoding requests with a 4-bit cache and e4m3 queries
        dict(name="norm 64 tokens mxfp4", op="norm", kv=MX, idx=MX, q8=True, T=64, hkv=1, group=16, rot=64, pairs=False, pad=0),
        # a chunked-prefill batch with fp8 caches: 64 decode rows, 4 x 4096 prefill rows, 8 pad rows
        dict(name="norm 16456 tokens fp8", op="norm", kv=FP8, idx=FP8, q8=False, T=16456, hkv=1, group=16, rot=64, pairs=False, pad=8),
        # one short sequence, 4 heads, bf16 queries: latency
        dict(name="attend 1 x 1000", op="attend", n=1, ctx=1000, ragged=False, q_len=1, hkv=1, group=4, q8=False),
        # a small batch of ragged contexts of 4k to 8k tokens
        dict(name="attend 32 x 4k-8k", op="attend", n=32, ctx=8192, ragged=True, q_len=1, hkv=1, group=16, q8=True),
        # speculative decoding: four tokens a step, 32k contexts
        dict(name="attend 128 x 32k q4", op="attend", n=128, ctx=32768, ragged=False, q_len=4, hkv=1, group=16, q8=True),
        # long contexts: 64 sequences of 128k tokens
        dict(name="attend 64 x 128k", op="attend", n=64, ctx=131072, ragged=False, q_len=1, hkv=1, group=16, q8=True),
        # the last tokens of a few requests read back from an fp8 cache
        dict(name="read 333 fp8", op="read", kv=FP8, T=333, hkv=2, pad=1),
        # one long prompt read back from a 4-bit cache
        dict(name="read 131072 mxfp4", op="read", kv=MX, T=131072, hkv=1, pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "norm", "norm", "attend", "attend", "attend", "read"])
    hkv = rng.choice([1, 1, 2, 4])
    if op == "tables":
        prefill = rng.choice([0, 0, _log(rng, 1, 16)])
        return dict(op=op, decode=_log(rng, 1, 4096), q_len=rng.choice([1, 1, 2, 4, 7]), prefill=prefill,
                    chunk=_log(rng, 5, 6000) if prefill else 0, pad=rng.choice([0, 3, 8, 61]), ctx=_log(rng, 40, 65536))
    if op == "norm":
        return dict(op=op, kv=rng.choice([BF16, FP8, MX]), idx=rng.choice([BF16, FP8, MX]), q8=rng.random() < 0.5,
                    T=max(1, _log(rng, 1, 16000) // hkv), hkv=hkv, group=rng.choice([1, 2, 4, 8, 16]),
                    rot=rng.choice([0, 32, 64, 64, 96, 128]), pairs=rng.random() < 0.3, pad=rng.choice([0, 0, 1, 8]))
    if op == "attend":
        n, q_len = _log(rng, 1, 256), rng.choice([1, 1, 1, 2, 3, 4, 8])
        most = min(131072, 8_000_000 // (n * hkv), 16_000_000 // (n * hkv * q_len))
        return dict(op=op, n=n, ctx=_log(rng, 1, most), ragged=rng.random() < 0.7, q_len=q_len, hkv=hkv,
                    group=rng.choice([1, 2, 4, 8, 16, 16]), q8=rng.random() < 0.7)
    return dict(op=op, kv=rng.choice([BF16, FP8, MX]), T=max(1, _log(rng, 1, 131072) // hkv), hkv=hkv,
                pad=rng.choice([0, 0, 1, 8]))


# ---- inputs ----------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randint(g, lo, hi, *shape, dtype=torch.int64):
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=dtype)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _kv_block_bytes(dtype, hkv):
    return 2 * hkv * MX_FIELD if dtype == MX else 16 * hkv * (4096 if dtype == BF16 else 2048)


def _idx_field(dtype):
    return {BF16: 32768, FP8: 16896, MX: MX_FIELD}[dtype]


def _random_mx_fields(g, fields):
    """[fields, 8704] bytes: e2m1 codes as those of normal values, scales near 2^-1."""
    q = torch.erfinv((torch.arange(256, device="cuda", dtype=torch.float64) + 0.5) / 128 - 1) * math.sqrt(2)
    code = _e2m1_code((q * 2.4).float()).to(torch.uint8)
    out = torch.empty(fields, MX_FIELD, dtype=torch.uint8, device="cuda")
    step = 16384
    for a in range(0, fields, step):
        b = min(a + step, fields)
        r = _randint(g, 0, 256, 2, b - a, MX_SCALES, dtype=torch.uint8)
        out[a:b, :MX_SCALES] = code[r[0].int()] | (code[r[1].int()] << 4)
        out[a:b, MX_SCALES:] = (126 + _randn(g, b - a, MX_FIELD - MX_SCALES) * 0.7).round().clamp(120, 132).to(torch.uint8)
    return out


def _random_cache(g, dtype, hkv, blocks):
    """A K/V cache's bytes (and one spare block), holding values as written from normal ones."""
    n = (blocks + 1) * _kv_block_bytes(dtype, hkv)
    if dtype == MX:
        return _random_mx_fields(g, (blocks + 1) * 2 * hkv).view(-1)
    if dtype == FP8:
        return _e4m3(_randn(g, n) / 0.01).view(torch.uint8)
    return _randn(g, n // 2).bfloat16().view(torch.uint8)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    {"tables": _prepare_tables, "norm": _prepare_norm, "attend": _prepare_attend, "read": _prepare_read}[case["op"]](case, g, s)
    return s


def _prepare_tables(c, g, s):
    n = c["decode"] + c["prefill"]
    new = torch.full((n,), c["q_len"], device="cuda")
    ctx = _randint(g, max(1, c["ctx"] // 8), c["ctx"] + 1, n)
    if c["prefill"]:
        new[c["decode"]:] = c["chunk"] - _randint(g, 0, 1 + c["chunk"] // 16, c["prefill"])
        ctx[c["decode"]:] = _randint(g, 0, 1 + c["ctx"] // 4096, c["prefill"]) * c["chunk"]
    if n > 3:
        new[_randint(g, 0, n, 1 + n // 32)] = 0  # requests that sit this step out
        ctx[_randint(g, 0, n, 1 + n // 32)] //= BLK
    s["context_lens"], s["new_lens"] = ctx.int(), new.int()
    # both bounds are the scheduler's, known on the host without a copy from the device
    s["capacity"] = c["decode"] * c["q_len"] + c["prefill"] * c["chunk"] + c["pad"]
    longest = max(c["ctx"], (c["ctx"] // 4096) * c["chunk"]) + max(c["q_len"], c["chunk"])
    s["stride"] = longest // BLK + 2
    have, want = (ctx + BLK - 1) // BLK, (ctx + new + BLK - 1) // BLK
    total, fresh = int(have.sum()), int((want - have).sum())
    ids = torch.randperm(total + fresh + 40, generator=g, device="cuda")
    first = torch.cumsum(have, 0) - have
    col = torch.arange(s["stride"], device="cuda")
    at = (first[:, None] + col).clamp(max=ids.numel() - 1)
    s["table"] = torch.where(col < have[:, None], ids[at], torch.full_like(at, -1)).int()
    s["free"] = ids[total:].int().contiguous()
    s["free_head"] = torch.tensor([7], dtype=torch.int32, device="cuda")
    s["num_blocks"] = ids.numel()
    if own:
        from block_sparse_paged_score_gb300 import step
        s["op"] = step.StepTables(n, s["stride"], s["capacity"], s["num_blocks"], block_table=s["table"])


def _prepare_norm(c, g, s):
    T, hkv, hq = c["T"], c["hkv"], c["hkv"] * c["group"]
    heads = hq + 4 * hkv
    # the projection's row: q heads, k, v, index q, index k, side by side
    row = (_randn(g, T, heads * D) * (0.3 + 3 * torch.rand(T, 1, generator=g, device="cuda"))).bfloat16()
    parts = torch.split(row, [hq * D, hkv * D, hkv * D, hkv * D, hkv * D], dim=1)
    s["q"], s["k"], s["v"], s["idx_q"], s["idx_k"] = (p.view(T, -1, D) for p in parts)
    s["offset"] = 1.0 if c["rot"] == 64 else 0.0
    for k in ("q", "k", "idx_q", "idx_k"):
        s["w_" + k] = (1 - s["offset"] + 0.2 * _randn(g, D)).bfloat16()
    s["max_pos"] = 131072
    if c["rot"]:
        h = c["rot"] // 2
        inv = 5_000_000.0 ** (-torch.arange(h, device="cuda", dtype=torch.float64) / h)
        angle = torch.arange(s["max_pos"], device="cuda", dtype=torch.float64)[:, None] * inv
        s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    else:
        s["rope"] = None
    s["pos"] = _randint(g, 0, s["max_pos"], T).int()
    blocks = 2 * (-(-T // BLK))
    s["blocks"] = blocks
    s["slot"] = torch.randperm(blocks * BLK, generator=g, device="cuda")[:T].contiguous()
    if T > 64:  # prefill: runs of consecutive slots, whole blocks at a time
        order = torch.randperm(blocks, generator=g, device="cuda")
        t = torch.arange(T, device="cuda")
        s["slot"] = (order[t // BLK] * BLK + t % BLK).contiguous()
    if c["pad"] and T > c["pad"]:
        s["pos"][T - c["pad"]:] = -1
        s["slot"][T - c["pad"]:] = -1
    s["kv"] = torch.zeros((blocks + 1) * _kv_block_bytes(c["kv"], hkv), dtype=torch.uint8, device="cuda")
    s["idx"] = torch.zeros((blocks + 1) * hkv * _idx_field(c["idx"]), dtype=torch.uint8, device="cuda")
    if own:
        from block_sparse_paged_score_gb300 import bsp, step
        kv = bsp.KvCache(c["kv"], hkv, blocks, K_SCALE, V_SCALE, buffer=s["kv"])
        idx = bsp.IndexCache(c["idx"], hkv, blocks, buffer=s["idx"])
        s["cache"], s["index_cache"] = kv, idx
        s["op"] = step.NormRopeWrite(kv, idx, hq, T, q_weight=s["w_q"], k_weight=s["w_k"], idx_q_weight=s["w_idx_q"],
                                     idx_k_weight=s["w_idx_k"], weight_offset=s["offset"], eps=EPS, rope_table=s["rope"],
                                     rope_pairs=c["pairs"], q_dtype=bsp.FP8_E4M3 if c["q8"] else bsp.BF16,
                                     idx_q_dtype=bsp.FP8_E4M3 if c["q8"] else bsp.BF16)


def _prepare_attend(c, g, s):
    n, hkv, ql = c["n"], c["hkv"], c["q_len"]
    lens = _randint(g, max(1, c["ctx"] // 2), c["ctx"] + 1, n) if c["ragged"] else torch.full((n,), c["ctx"], device="cuda")
    if c["ragged"] and n > 4:
        lens[_randint(g, 0, n, 1)] = 0  # a padded batch: a sequence with nothing to attend to
    s["nb"] = -(-c["ctx"] // BLK)
    blocks = n * s["nb"]
    s["blocks"] = blocks
    s["kv"] = _random_cache(g, MX, hkv, blocks)
    s["table"] = torch.randperm(blocks, generator=g, device="cuda").int().view(n, s["nb"])
    q = _randn(g, n * ql, hkv * c["group"], D)
    s["q"] = _e4m3(q).view(torch.uint8) if c["q8"] else q.bfloat16()
    j = torch.arange(ql, device="cuda")
    seen = (lens[:, None] - (ql - 1 - j)).clamp(min=0)
    s["row_len"] = seen[:, :, None].expand(n, ql, hkv).reshape(-1).int().contiguous()
    s["row_seq"] = torch.arange(n, device="cuda")[:, None].expand(n, ql * hkv).reshape(-1).int().contiguous()
    if own:
        from block_sparse_paged_score_gb300 import bsp
        s["cache"] = bsp.KvCache(bsp.MXFP4, hkv, blocks, buffer=s["kv"])
        s["ws"] = bsp.dense_pa_workspace(n * ql * hkv, hkv, c["group"], ql)
        s["out"] = torch.empty(n * ql, hkv * c["group"], D, dtype=torch.bfloat16, device="cuda")


def _prepare_read(c, g, s):
    T, hkv = c["T"], c["hkv"]
    blocks = -(-T // BLK) + 3
    s["blocks"] = blocks
    s["kv"] = _random_cache(g, c["kv"], hkv, blocks)
    order = torch.randperm(blocks, generator=g, device="cuda")
    t = torch.arange(T, device="cuda") + 5
    s["slot"] = (order[t // BLK] * BLK + t % BLK).contiguous()
    if c["pad"] and T > c["pad"]:
        s["slot"][T - c["pad"]:] = -1
    if own:
        from block_sparse_paged_score_gb300 import bsp
        s["cache"] = bsp.KvCache(c["kv"], hkv, blocks, K_SCALE, V_SCALE, buffer=s["kv"])
        s["k"] = torch.empty(T, hkv, D, dtype=torch.bfloat16, device="cuda")
        s["v"] = torch.empty(T, hkv, D, dtype=torch.bfloat16, device="cuda")


# ---- one pass --------------------------------------------------------------
def run(s):
    return {"tables": _run_tables, "norm": _run_norm, "attend": _run_attend, "read": _run_read}[s["case"]["op"]](s)


def _run_tables(s):
    if own:
        t = s["op"]
        t.run(s["context_lens"], s["new_lens"], s["free"], s["free_head"])
        return dict(table=t.block_table, seq_lens=t.seq_lens, cu=t.cu_tokens, taken=t.blocks_taken, slot=t.slot,
                    req=t.query_req_id, pos=t.query_abs_pos)
    ctx, new, table, free = s["context_lens"].long(), s["new_lens"].long(), s["table"], s["free"]
    n, width = table.shape
    have, want = (ctx + BLK - 1) // BLK, (ctx + new + BLK - 1) // BLK
    fresh = want - have
    cu = torch.cat([new.new_zeros(1), torch.cumsum(new, 0)])
    taken = torch.cumsum(fresh, 0)
    first = taken - fresh + s["free_head"].long()
    col = torch.arange(width, device="cuda")
    at = (first[:, None] + col - have[:, None]).clamp(0, free.numel() - 1)
    table = torch.where((col >= have[:, None]) & (col < want[:, None]), free[at], table)
    t = torch.arange(s["capacity"], device="cuda")
    req = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=n - 1)
    live = t < cu[-1]
    pos = ctx[req] + t - cu[req]
    slot = table[req, (pos // BLK).clamp(0, width - 1)].long() * BLK + pos % BLK
    return dict(table=table, seq_lens=(ctx + new).int(), cu=cu.int(), taken=taken[-1:].int(),
                slot=torch.where(live, slot, -torch.ones_like(slot)),
                req=torch.where(live, req, torch.zeros_like(req)).int(),
                pos=torch.where(live, pos, -torch.ones_like(pos)).int())


def _e4m3(x):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _e2m1_code(x):
    """Nearest e2m1 code, ties to the even one, saturating."""
    a = x.abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
            + (a >= 3.5).int() + (a > 5).int())
    return code + 8 * torch.signbit(x).int()


def _mx_encode(x):
    """[..., 128] fp32 -> packed e2m1 [..., 64] and e8m0 [..., 4] bytes: the exponent is floor(log2(amax)) - 2."""
    grp = x.reshape(*x.shape[:-1], 4, 32)
    amax = grp.abs().amax(-1)
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 3, torch.full_like(amax, -127).int()).clamp(-127, 127)
    code = _e2m1_code(torch.ldexp(grp, -e[..., None])).reshape(*x.shape[:-1], 64, 2)
    return (code[..., 0] | (code[..., 1] << 4)).to(torch.uint8), (e + 127).to(torch.uint8)


def _mx_values(data, scales):
    """Packed e2m1 [..., 64] and e8m0 [..., 4] bytes -> fp32 [..., 128]."""
    lut = torch.tensor(E2M1, device="cuda")
    d = data.int()
    v = torch.stack([lut[d & 15], lut[d >> 4]], -1).reshape(*data.shape[:-1], 4, 32)
    return (v * torch.exp2(scales.float() - 127)[..., None]).reshape(*data.shape[:-1], D)


def _page_elements(slot, hkv, x):
    """Element numbers of K and V [T, Hkv, 128] in an interleaved cache whose 16-byte rows hold x elements."""
    h, d = torch.arange(hkv, device="cuda")[:, None], torch.arange(D, device="cuda")
    o = slot % BLK
    page = (slot // BLK) * 16 + o // PG
    t = (o % PG)[:, None, None]
    base = (page[:, None, None] * hkv + h) * (PG * D)
    return base + (d // x) * (PG * x) + t * x + d % x, base + 8 * hkv * PG * D + (t // x) * (D * x) + d * x + t % x


def _mx_bytes(slot, heads, first, per_block):
    """Byte numbers of the data [T, heads, 64] and scales [T, heads, 4] of fields `first`.. of a slot's block."""
    h = torch.arange(heads, device="cuda")[:, None]
    field = ((slot // BLK)[:, None, None] * per_block + first + h) * MX_FIELD
    o = (slot % BLK)[:, None, None]
    return field + o * 64 + torch.arange(64, device="cuda"), field + MX_SCALES + o * 4 + torch.arange(4, device="cuda")


def _put_kv(buf, dtype, hkv, slot, k, v):
    if dtype == MX:
        for first, x in ((0, k), (hkv, v)):
            data, scales = _mx_encode(x)
            a, b = _mx_bytes(slot, hkv, first, 2 * hkv)
            buf[a], buf[b] = data, scales
        return
    a, b = _page_elements(slot, hkv, 8 if dtype == BF16 else 16)
    if dtype == BF16:
        flat = buf.view(torch.int16)
        flat[a], flat[b] = k.bfloat16().view(torch.int16), v.bfloat16().view(torch.int16)
    else:
        buf[a], buf[b] = _e4m3(k / K_SCALE).view(torch.uint8), _e4m3(v / V_SCALE).view(torch.uint8)


def _get_kv(buf, dtype, hkv, slot):
    """fp32 K and V [T, Hkv, 128] of the slots (-1: the spare block's)."""
    if dtype == MX:
        got = []
        for first in (0, hkv):
            a, b = _mx_bytes(slot, hkv, first, 2 * hkv)
            got.append(_mx_values(buf[a], buf[b]))
        return got
    a, b = _page_elements(slot, hkv, 8 if dtype == BF16 else 16)
    if dtype == BF16:
        flat = buf.view(torch.bfloat16)
        return flat[a].float(), flat[b].float()
    return buf[a].view(torch.float8_e4m3fn).float() * K_SCALE, buf[b].view(torch.float8_e4m3fn).float() * V_SCALE


def _put_idx(buf, dtype, heads, slot, x):
    h, o, d = torch.arange(heads, device="cuda")[:, None], (slot % BLK)[:, None, None], torch.arange(D, device="cuda")
    field = ((slot // BLK)[:, None, None] * heads + h) * _idx_field(dtype)
    if dtype == BF16:
        buf.view(torch.int16)[field // 2 + o * D + d] = x.bfloat16().view(torch.int16)
    elif dtype == FP8:
        amax = x.abs().amax(-1, keepdim=True)
        sc = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
        buf[field + o * D + d] = _e4m3(x / sc).view(torch.uint8)
        buf.view(torch.float32)[field // 4 + 4096 + o] = sc
    else:
        data, scales = _mx_encode(x)
        a, b = _mx_bytes(slot, heads, 0, heads)
        buf[a], buf[b] = data, scales


def _norm_rope(x, w, s):
    c, x = s["case"], x.float()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * (w.float() + s["offset"])
    live = (s["pos"] >= 0)[:, None, None]
    if c["rot"]:
        h = c["rot"] // 2
        cs = s["rope"][s["pos"].clamp(min=0).long()][:, None]
        cos, sin = cs[..., :h], cs[..., h:]
        r = y[..., :c["rot"]]
        if c["pairs"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = r[..., :h], r[..., h:]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        y = torch.cat([r, y[..., c["rot"]:]], -1)
    return torch.where(live, y, torch.zeros_like(y))


def _caches_out(s):
    """The caches as the values they hold: fp8 and bf16 ones whole, through views; 4-bit ones read back by slot."""
    c, out = s["case"], {}
    kv = s["kv"][: s["blocks"] * _kv_block_bytes(c["kv"], c["hkv"])]
    idx = s["idx"][: s["blocks"] * c["hkv"] * _idx_field(c["idx"])]
    if c["kv"] != MX:
        out["kv"] = kv.view(torch.bfloat16 if c["kv"] == BF16 else torch.float8_e4m3fn)
    if c["idx"] == BF16:
        out["idx"] = idx.view(torch.bfloat16)
    elif c["idx"] == FP8:
        f = idx.view(-1, _idx_field(FP8))
        out["idx"], out["idx_scale"] = f[:, :16384].view(torch.float8_e4m3fn), f[:, 16384:].view(torch.float32)
    return out


def _run_norm(s):
    c = s["case"]
    if own:
        from block_sparse_paged_score_gb300 import bsp
        op = s["op"]
        q, idx_q = op.run(s["q"], s["k"], s["v"], s["idx_q"], s["idx_k"], s["pos"], s["slot"])
        if c["q8"]:
            q, idx_q = q.view(torch.float8_e4m3fn), idx_q.view(torch.float8_e4m3fn)
        out = dict(q=q, idx_q=idx_q, **_caches_out(s))
        if c["kv"] == MX or c["idx"] == MX:
            k, v, ik = bsp.kv_page_read(s["cache"], s["index_cache"], s["slot"])
            if c["kv"] == MX:
                out["k"], out["v"] = k.to(torch.float8_e5m2), v.to(torch.float8_e5m2)
            if c["idx"] == MX:
                out["idx_k"] = ik.to(torch.float8_e5m2)
        return out
    q, k = _norm_rope(s["q"], s["w_q"], s), _norm_rope(s["k"], s["w_k"], s)
    idx_q, idx_k = _norm_rope(s["idx_q"], s["w_idx_q"], s), _norm_rope(s["idx_k"], s["w_idx_k"], s)
    slot = torch.where(s["slot"] < 0, s["blocks"] * BLK, s["slot"])  # the spare block takes the pad rows
    _put_kv(s["kv"], c["kv"], c["hkv"], slot, k, s["v"].float())
    _put_idx(s["idx"], c["idx"], c["hkv"], slot, idx_k)
    r = _e4m3 if c["q8"] else (lambda x: x.bfloat16())
    out = dict(q=r(q), idx_q=r(idx_q), **_caches_out(s))
    live = (s["slot"] >= 0)[:, None, None]
    if c["kv"] == MX:
        k, v = _get_kv(s["kv"], MX, c["hkv"], slot)
        out["k"], out["v"] = (torch.where(live, x, torch.zeros_like(x)).to(torch.float8_e5m2) for x in (k, v))
    if c["idx"] == MX:
        a, b = _mx_bytes(slot, c["hkv"], 0, c["hkv"])
        x = _mx_values(s["idx"][a], s["idx"][b])
        out["idx_k"] = torch.where(live, x, torch.zeros_like(x)).to(torch.float8_e5m2)
    return out


def _run_attend(s):
    c = s["case"]
    n, ql, hkv, G, nb = c["n"], c["q_len"], c["hkv"], c["group"], s["nb"]
    if own:
        from block_sparse_paged_score_gb300 import bsp
        return bsp.dense_pa_decode(s["cache"], s["q"], bsp.FP8_E4M3 if c["q8"] else bsp.BF16, hkv * G, s["table"],
                                   s["row_seq"], s["row_len"], ql, out=s["out"], ws=s["ws"])
    q = (s["q"].view(torch.float8_e4m3fn) if c["q8"] else s["q"]).float()
    q = q.view(n, ql, hkv, G, D).transpose(1, 2).reshape(n, hkv, ql * G, D)
    blocks = s["kv"].view(-1, 2 * hkv, MX_FIELD)[s["table"].long()]  # [n, nb, 2 Hkv, 8704]

    def side(f):
        v = _mx_values(f[..., :MX_SCALES].reshape(*f.shape[:-1], BLK, 64), f[..., MX_SCALES:].reshape(*f.shape[:-1], BLK, 4))
        return v.permute(0, 2, 1, 3, 4).reshape(n, hkv, nb * BLK, D)

    z = torch.matmul(q, side(blocks[:, :, :hkv]).transpose(-1, -2)) * (1 / math.sqrt(D))
    seen = s["row_len"].view(n, ql, hkv).transpose(1, 2).repeat_interleave(G, 2)  # [n, Hkv, ql * G]
    z = torch.where(torch.arange(nb * BLK, device="cuda") < seen[..., None], z, torch.full_like(z, -math.inf))
    p = torch.exp(z - z.amax(-1, keepdim=True).clamp(min=-1e30))
    o = torch.matmul(p, side(blocks[:, :, hkv:])) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return o.view(n, hkv, ql, G, D).transpose(1, 2).reshape(n * ql, hkv * G, D).bfloat16()


def _run_read(s):
    c = s["case"]
    if own:
        from block_sparse_paged_score_gb300 import bsp
        k, v, _ = bsp.kv_page_read(s["cache"], None, s["slot"], k=s["k"], v=s["v"])
        return dict(k=k, v=v)
    live = (s["slot"] >= 0)[:, None, None]
    k, v = _get_kv(s["kv"], c["kv"], c["hkv"], torch.where(s["slot"] < 0, s["blocks"] * BLK, s["slot"]))
    return dict(k=torch.where(live, k, torch.zeros_like(k)).bfloat16(), v=torch.where(live, v, torch.zeros_like(v)).bfloat16())


# ---- what a pass cannot do without -------------------------------------------
def work(c):
    if c["op"] == "tables":
        n = c["decode"] + c["prefill"]
        tokens = c["decode"] * c["q_len"] + c["prefill"] * c["chunk"] + c["pad"]
        fresh = tokens // BLK  # the new blocks' ids read and written; each request's current block read
        return dict(bytes=n * (4 + 4 + 4 + 4 + 4) + tokens * (8 + 4 + 4) + fresh * 8, flops=0)
    per = {BF16: 2, FP8: 1, MX: 68 / 128}
    if c["op"] == "norm":
        T, hkv, hq = c["T"], c["hkv"], c["hkv"] * c["group"]
        read = T * ((hq + 4 * hkv) * D * 2 + 4 * c["rot"] + 12) + 4 * D * 2
        wrote = T * ((hq + hkv) * D * (1 if c["q8"] else 2) + 2 * hkv * D * per[c["kv"]] + hkv * D * per[c["idx"]])
        return dict(bytes=read + wrote, flops=T * (hq + 3 * hkv) * D * 8)
    if c["op"] == "read":
        return dict(bytes=c["T"] * (8 + 2 * c["hkv"] * D * (per[c["kv"]] + 2)), flops=c["T"] * 2 * c["hkv"] * D)
    tokens = c["n"] * c["ctx"] * (0.75 if c["ragged"] else 1)
    rows = c["n"] * c["q_len"] * c["hkv"]
    q = rows * c["group"] * D
    return dict(bytes=tokens * c["hkv"] * 136 + tokens / BLK * 4 + q * ((1 if c["q8"] else 2) + 2) + rows * 8,
                flops=tokens * c["hkv"] * c["q_len"] * c["group"] * D * 4)


# ---- the definitions in 64 bits ------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"tables": lambda s: None, "norm": _exact_norm, "attend": _exact_attend, "read": _exact_read}[case["op"]](s)


def _grid_code_values(mag):
    """Magnitudes rounded to the e2m1 grid by the two-sided definition: steps of 1/2 below 2, 1 below 4, 2 above; at most 6."""
    step = torch.where(mag < 2, 0.5, torch.where(mag < 4, 1.0, 2.0)).to(mag.dtype)
    return (torch.round(mag / step) * step).clamp(max=6.0)


def _exact_mx(x):
    """float64 [..., 128] as an MXFP4 cache holds it."""
    g = x.unflatten(-1, (4, 32))
    top = g.abs().amax(-1, keepdim=True)
    unit = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -120))) - 2)
    return (torch.sign(g) * _grid_code_values(g.abs() / unit) * unit).flatten(-2)


def _exact_e4m3(x):
    """float64 rounded to the e4m3 grid: steps of 2^(e-3), no finer than 2^-9, at most 448."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_heads(x, w, s):
    c, x = s["case"], x.double()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * (w.double() + s["offset"])
    if c["rot"]:
        h = c["rot"] // 2
        t = s["rope"].double()[s["pos"].long().clamp(min=0)]
        turn = torch.complex(t[:, :h], t[:, h:])[:, None]
        r = y[..., :c["rot"]]
        if c["pairs"]:
            r = torch.view_as_real(torch.view_as_complex(r.unflatten(-1, (h, 2)).contiguous()) * turn).flatten(-2)
        else:
            z = torch.complex(r[..., :h].contiguous(), r[..., h:].contiguous()) * turn
            r = torch.cat([z.real, z.imag], -1)
        y = torch.cat([r, y[..., c["rot"]:]], -1)
    y[s["pos"] < 0] = 0
    return y


def _exact_norm(s):
    c = s["case"]
    hkv, nb = c["hkv"], s["blocks"]
    q, k = _exact_heads(s["q"], s["w_q"], s), _exact_heads(s["k"], s["w_k"], s)
    iq, ik = _exact_heads(s["idx_q"], s["w_idx_q"], s), _exact_heads(s["idx_k"], s["w_idx_k"], s)
    v = s["v"].double()
    out = dict(q=_exact_e4m3(q) if c["q8"] else q, idx_q=_exact_e4m3(iq) if c["q8"] else iq)
    ok = s["slot"] >= 0
    slot = s["slot"][ok]
    b, o = slot // BLK, slot % BLK
    if c["kv"] == MX:
        live = ok[:, None, None].double()
        out["k"], out["v"] = _exact_mx(k) * live, _exact_mx(v) * live
    else:
        x = 8 if c["kv"] == BF16 else 16
        if c["kv"] == FP8:
            k, v = _exact_e4m3(k / K_SCALE), _exact_e4m3(v / V_SCALE)
        page = torch.zeros(nb, 16, hkv, PG * D, dtype=torch.float64, device="cuda")
        keys = page[:, :8].unflatten(-1, (D // x, PG, x)).permute(0, 1, 4, 2, 3, 5)  # [nb, page, t, h, d/x, x]
        keys[b, o // PG, o % PG] = k[ok].unflatten(-1, (D // x, x))
        vals = page[:, 8:].unflatten(-1, (PG // x, D, x)).permute(0, 1, 3, 5, 2, 4)  # [nb, page, t/x, t%x, h, d]
        vals[b, o // PG, o % PG // x, o % x] = v[ok]
        out["kv"] = page.flatten()
    if c["idx"] == MX:
        out["idx_k"] = _exact_mx(ik) * ok[:, None, None].double()
    elif c["idx"] == BF16:
        field = torch.zeros(nb, hkv, BLK, D, dtype=torch.float64, device="cuda")
        field.transpose(1, 2)[b, o] = ik[ok]
        out["idx"] = field.flatten()
    else:
        field = torch.zeros(nb, hkv, BLK, D, dtype=torch.float64, device="cuda")
        scale = torch.zeros(nb, hkv, BLK, dtype=torch.float64, device="cuda")
        top = ik[ok].abs().amax(-1)
        unit = torch.where(top > 0, top / 448, torch.ones_like(top))
        field.transpose(1, 2)[b, o] = _exact_e4m3(ik[ok] / unit[..., None])
        scale.transpose(1, 2)[b, o] = unit
        out["idx"], out["idx_scale"] = field.reshape(nb * hkv, -1), scale.reshape(nb * hkv, -1)
    return out


def _exact_fields(f):
    """[..., 8704] bytes -> float64 [..., 128 tokens, 128 dims], from the sign, exponent and mantissa bits."""
    nib = torch.stack([f[..., :MX_SCALES] % 16, f[..., :MX_SCALES] // 16], -1).flatten(-2).to(torch.int8)
    e, m = (nib // 2) % 4, (nib % 2).double()
    mag = torch.where(e > 0, (1 + m / 2) * torch.exp2(e.double() - 1), m / 2)
    val = torch.where(nib >= 8, -mag, mag).unflatten(-1, (BLK, 4, 32))
    return (val * torch.exp2(f[..., MX_SCALES:].double() - 127).unflatten(-1, (BLK, 4))[..., None]).flatten(-2)


def _exact_attend(s):
    c = s["case"]
    n, ql, hkv, G = c["n"], c["q_len"], c["hkv"], c["group"]
    q = (s["q"].view(torch.float8_e4m3fn) if c["q8"] else s["q"]).double().view(n, ql, hkv, G, D)
    seen = s["row_len"].view(n, ql, hkv)
    fields = s["kv"].view(-1, 2, hkv, MX_FIELD)
    out = torch.zeros(n, ql, hkv, G, D, dtype=torch.float64, device="cuda")
    longest = seen.amax((1, 2)).tolist()
    for i in range(n):
        L = longest[i]
        if L == 0:
            continue
        x = _exact_fields(fields[s["table"][i, : -(-L // BLK)].long()]).permute(1, 2, 0, 3, 4).flatten(2, 3)[:, :, :L]
        z = torch.einsum("jhgd,htd->jhgt", q[i], x[0]) / math.sqrt(D)
        z.masked_fill_(torch.arange(L, device="cuda") >= seen[i][:, :, None, None], -math.inf)
        out[i] = torch.einsum("jhgt,htd->jhgd", torch.nan_to_num(torch.softmax(z, -1), nan=0.0), x[1])
    return out.view(n * ql, hkv * G, D)


def _exact_read(s):
    c = s["case"]
    hkv, x = c["hkv"], 8 if c["kv"] == BF16 else 16
    ok = s["slot"] >= 0
    slot = s["slot"].clamp(min=0)
    b, o = slot // BLK, slot % BLK
    got = []
    for side in (0, 1):
        if c["kv"] == MX:
            f = s["kv"].view(-1, 2, hkv, MX_FIELD)[:, side]
            blocks, inverse = torch.unique(b, return_inverse=True)
            r = _exact_fields(f[blocks])[inverse, :, o]
        else:
            raw = s["kv"].view(torch.bfloat16 if c["kv"] == BF16 else torch.float8_e4m3fn).view(-1, 2, 8, hkv, PG * D)[:, side]
            raw = raw.double() * (1 if c["kv"] == BF16 else (K_SCALE, V_SCALE)[side])
            if side == 0:
                r = raw.unflatten(-1, (D // x, PG, x)).permute(0, 1, 4, 2, 3, 5)[b, o // PG, o % PG].flatten(-2)
            else:
                r = raw.unflatten(-1, (PG // x, D, x)).permute(0, 1, 3, 5, 2, 4)[b, o // PG, o % PG // x, o % x]
        got.append(r * ok[:, None, None])
    return dict(k=got[0], v=got[1])
