"""Operators of the layers without an indexer over 8-bit caches whose scales are per block and head: their measured
cases and plain forms.

  prompt  causal grouped-query attention of whole prompts or chunks, packed sequences of different lengths
  attend  dense grouped-query attention over an fp8 paged cache with a scale for each 128-token block and head
  write   new K and V quantised into such a cache, its blocks' scales growing with their tokens
  read    cached K and V gathered back by slot as bf16

``run`` computes an operator from elementary torch operations in 32 bits, or with ``own`` true by the framework's call.
"""
import math

import torch

own = False

BLK, PG, D = 128, 16, 128
LOW, HIGH = -60, 119  # exponents a written scale may have


# ---- cases -----------------------------------------------------------------
def listed():
    return [
        # one short prompt of a single user: latency
        dict(name="prompt 1 x 100", op="prompt", n=1, new=100, ctx=0, ragged=False, hkv=1, group=4, pad=0),
        # a batch of ordinary prompts packed one behind the other, rows of a captured size behind them
        dict(name="prompt 32 x 250-2000", op="prompt", n=32, new=2000, ctx=0, ragged=True, hkv=1, group=16, pad=61),
        # a follow-up question of some tokens on each of three long documents
        dict(name="prompt 3 x 77 over 100000", op="prompt", n=3, new=77, ctx=100000, ragged=False, hkv=2, group=8, pad=0),
        # one long prompt
        dict(name="prompt 1 x 32768", op="prompt", n=1, new=32768, ctx=0, ragged=False, hkv=1, group=16, pad=0),
        # one short sequence, 4 heads, bf16 queries: latency
        dict(name="attend 1 x 1000", op="attend", n=1, ctx=1000, ragged=False, q_len=1, hkv=1, group=4, q8=False),
        # a small batch of ragged contexts of 4k to 8k tokens
        dict(name="attend 32 x 4k-8k", op="attend", n=32, ctx=8192, ragged=True, q_len=1, hkv=1, group=16, q8=False),
        # speculative decoding: four tokens a step, 32k contexts
        dict(name="attend 128 x 32k q4", op="attend", n=128, ctx=32768, ragged=False, q_len=4, hkv=1, group=16, q8=True),
        # long contexts: 64 sequences of 128k tokens
        dict(name="attend 64 x 128k", op="attend", n=64, ctx=131072, ragged=False, q_len=1, hkv=1, group=16, q8=False),
        # a decode step of 64 requests: one token each into blocks that hold some already
        dict(name="write 64 x 1", op="write", n=64, new=1, ragged=False, hkv=1, fresh=False, pad=0),
        # prompts of a chunked-prefill batch
        dict(name="write 8 x 300-2400", op="write", n=8, new=2400, ragged=True, hkv=2, fresh=True, pad=8),
        # the last tokens of a few requests
        dict(name="read 333", op="read", T=333, hkv=2, pad=1),
        # the context of a long document, for the next chunk's attention
        dict(name="read 131072", op="read", T=131072, hkv=1, pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt", "attend", "attend", "attend", "write", "write", "read"])
    hkv = rng.choice([1, 1, 2, 4])
    if op == "prompt":
        n, group = _log(rng, 1, 64), rng.choice([1, 2, 4, 8, 16, 16])
        ctx = rng.choice([0, 0, _log(rng, 10, 100000)])
        ctx = min(ctx, 300_000 // n)
        new = min(_log(rng, 1, 20000), 100_000 // n)
        while n * hkv * group * new * (ctx + new / 2) > 8e9:
            new = max(1, new // 2)
            if new == 1:
                ctx //= 2
        return dict(op=op, n=n, new=new, ctx=ctx, ragged=rng.random() < 0.6, hkv=hkv, group=group,
                    pad=rng.choice([0, 0, 1, 61]))
    if op == "attend":
        n, q_len = _log(rng, 1, 256), rng.choice([1, 1, 1, 2, 3, 4, 8])
        most = min(131072, 8_000_000 // (n * hkv), 16_000_000 // (n * hkv * q_len))
        return dict(op=op, n=n, ctx=_log(rng, 1, most), ragged=rng.random() < 0.7, q_len=q_len, hkv=hkv,
                    group=rng.choice([1, 2, 4, 8, 16, 16]), q8=rng.random() < 0.5)
    if op == "write":
        fresh = rng.random() < 0.5
        n = _log(rng, 1, 64 if fresh else 1024)
        new = min(_log(rng, 1, 16000), 64000 // (n * hkv)) if fresh else rng.choice([1, 1, 2, 4, 7])
        return dict(op=op, n=n, new=max(1, new), ragged=rng.random() < 0.5, hkv=hkv, fresh=fresh, pad=rng.choice([0, 0, 3, 8]))
    return dict(op=op, T=max(1, _log(rng, 1, 131072) // hkv), hkv=hkv, pad=rng.choice([0, 0, 1, 8]))


# ---- inputs ----------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randint(g, lo, hi, *shape, dtype=torch.int64):
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=dtype)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _lengths(g, n, lo, hi, ragged):
    """n lengths, evenly spaced from lo to hi in an order of the seed's (their sum is the case's), or all hi."""
    if not ragged:
        return torch.full((n,), hi, device="cuda")
    return (lo + (hi - lo) * (torch.arange(n, device="cuda") + 1) // n)[torch.randperm(n, generator=g, device="cuda")]


def _rows(g, T, heads, most):
    """bf16 rows [T, heads, 128] of normal values, a size of its own for each token."""
    return (_randn(g, T, heads, D) * (0.5 + most * torch.rand(T, 1, 1, generator=g, device="cuda"))).bfloat16()


def _random_cache(g, hkv, blocks):
    """An fp8 cache's bytes (and one spare block) and scales, holding values of about 1."""
    def scales():
        return torch.exp2(_randint(g, -8, -4, blocks + 1, hkv).float())
    return _e4m3(_randn(g, (blocks + 1) * hkv * 32768) * 80).view(torch.uint8), scales(), scales()


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    {"prompt": _prepare_prompt, "attend": _prepare_attend, "write": _prepare_write, "read": _prepare_read}[case["op"]](case, g, s)
    return s


def _prepare_prompt(c, g, s):
    n, hkv, hq = c["n"], c["hkv"], c["hkv"] * c["group"]
    new = _lengths(g, n, c["new"] // 8, c["new"], c["ragged"])
    ctx = _lengths(g, n, c["ctx"] // 8, c["ctx"], c["ragged"])
    if c["ragged"] and n > 3:
        new[new.argmin()] = 0  # a request that sits this step out
    s["new"], s["keys"] = new.tolist(), (ctx + new).tolist()  # the scheduler's, known on the host
    zero = new.new_zeros(1)
    s["cu_q"] = torch.cat([zero, torch.cumsum(new, 0)]).int()
    s["cu_k"] = torch.cat([zero, torch.cumsum(ctx + new, 0)]).int()
    Tq, Tk = sum(s["new"]) + c["pad"], sum(s["keys"])
    s["q"] = _rows(g, Tq, hq, 1.5)
    # keys and values side by side, as a projection leaves them
    kv = _rows(g, Tk, 2 * hkv, 1.0)
    s["k"], s["v"] = kv[:, :hkv], kv[:, hkv:]
    s["out"] = torch.zeros(Tq, hq, D, dtype=torch.bfloat16, device="cuda")
    if own:
        from block_sparse_paged_score_gb300 import bsp
        s["ws"] = bsp.prompt_attention_workspace(Tq, n, hkv, c["group"])


def _prepare_attend(c, g, s):
    n, hkv, ql = c["n"], c["hkv"], c["q_len"]
    lens = _lengths(g, n, c["ctx"] // 2, c["ctx"], c["ragged"])
    if c["ragged"] and n > 4:
        lens[lens.argmin()] = 0  # a padded batch: a sequence with nothing to attend to
    s["nb"] = -(-c["ctx"] // BLK)
    blocks = n * s["nb"]
    s["blocks"] = blocks
    s["kv"], s["ks"], s["vs"] = _random_cache(g, hkv, blocks)
    s["table"] = torch.randperm(blocks, generator=g, device="cuda").int().view(n, s["nb"])
    q = _randn(g, n * ql, hkv * c["group"], D)
    s["q"] = _e4m3(q).view(torch.uint8) if c["q8"] else q.bfloat16()
    j = torch.arange(ql, device="cuda")
    seen = (lens[:, None] - (ql - 1 - j)).clamp(min=0)
    s["row_len"] = seen[:, :, None].expand(n, ql, hkv).reshape(-1).int().contiguous()
    s["row_seq"] = torch.arange(n, device="cuda")[:, None].expand(n, ql * hkv).reshape(-1).int().contiguous()
    if own:
        from block_sparse_paged_score_gb300 import bsp
        s["cache"] = bsp.BlockScaledKvCache(hkv, blocks, buffer=s["kv"], k_scales=s["ks"], v_scales=s["vs"])
        s["ws"] = bsp.dense_pa_fp8_workspace(n * ql * hkv, hkv, c["group"], ql)
        s["out"] = torch.empty(n * ql, hkv * c["group"], D, dtype=torch.bfloat16, device="cuda")


def _prepare_write(c, g, s):
    n, hkv = c["n"], c["hkv"]
    new = _lengths(g, n, c["new"] // 8, c["new"], c["ragged"])
    at = torch.zeros_like(new) if c["fresh"] else _randint(g, 1, BLK, n)
    want = (at + new + BLK - 1) // BLK
    T = int(new.sum())
    s["blocks"] = blocks = T // BLK + 2 * n + 5
    ids = torch.randperm(blocks, generator=g, device="cuda")
    seq = torch.repeat_interleave(torch.arange(n, device="cuda"), new)
    t = at[seq] + torch.arange(T, device="cuda") - (torch.cumsum(new, 0) - new)[seq]
    slot = ids[(torch.cumsum(want, 0) - want)[seq] + t // BLK] * BLK + t % BLK
    s["slot"] = torch.cat([slot, slot.new_full((c["pad"],), -1)])
    s["kv"], s["ks"], s["vs"] = _random_cache(g, hkv, blocks)
    row = _rows(g, T + c["pad"], 2 * hkv, 3.0)
    s["k"], s["v"] = row[:, :hkv], row[:, hkv:]
    if own:
        from block_sparse_paged_score_gb300 import bsp
        s["cache"] = bsp.BlockScaledKvCache(hkv, blocks, buffer=s["kv"], k_scales=s["ks"], v_scales=s["vs"])


def _prepare_read(c, g, s):
    T, hkv = c["T"], c["hkv"]
    s["blocks"] = blocks = -(-T // BLK) + 3
    s["kv"], s["ks"], s["vs"] = _random_cache(g, hkv, blocks)
    order = torch.randperm(blocks, generator=g, device="cuda")
    t = torch.arange(T, device="cuda") + 5
    s["slot"] = (order[t // BLK] * BLK + t % BLK).contiguous()
    if c["pad"] and T > c["pad"]:
        s["slot"][T - c["pad"]:] = -1
    if own:
        from block_sparse_paged_score_gb300 import bsp
        s["cache"] = bsp.BlockScaledKvCache(hkv, blocks, buffer=s["kv"], k_scales=s["ks"], v_scales=s["vs"])
        s["k"] = torch.empty(T, hkv, D, dtype=torch.bfloat16, device="cuda")
        s["v"] = torch.empty(T, hkv, D, dtype=torch.bfloat16, device="cuda")


# ---- one pass --------------------------------------------------------------
def run(s):
    return {"prompt": _run_prompt, "attend": _run_attend, "write": _run_write, "read": _run_read}[s["case"]["op"]](s)


def _e4m3(x):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _sides(s):
    """The cache's K pages [blocks, 8, Hkv, 128 / 16, 16 tokens, 16] and V pages [blocks, 8, Hkv, 128, 16 tokens]."""
    hkv = s["case"]["hkv"]
    pages = s["kv"].view(torch.float8_e4m3fn).view(-1, 16, hkv, PG * D)
    return pages[:, :8].unflatten(-1, (D // 16, PG, 16)), pages[:, 8:].unflatten(-1, (D, PG))


def _blocks_of(s, ids):
    """fp32 K and V [*ids, Hkv, 128 tokens, 128] of whole blocks."""
    kp, vp = _sides(s)
    k = kp.view(torch.uint8)[ids].view(torch.float8_e4m3fn).float().movedim(-5, -4)  # [*, Hkv, 8, D/16, PG, 16]
    v = vp.view(torch.uint8)[ids].view(torch.float8_e4m3fn).float().movedim(-4, -3)  # [*, Hkv, 8, D, PG]
    k = k.transpose(-3, -2).flatten(-2).flatten(-3, -2) * s["ks"][ids][..., None, None]
    v = v.transpose(-2, -1).flatten(-3, -2) * s["vs"][ids][..., None, None]
    return k, v


def _run_prompt(s):
    c = s["case"]
    if own:
        from block_sparse_paged_score_gb300 import bsp
        return bsp.prompt_attention(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], out=s["out"], ws=s["ws"])
    hkv, G = c["hkv"], c["group"]
    out = s["out"].clone()
    a = b = 0
    for nq, nk in zip(s["new"], s["keys"]):
        step = max(1, (1 << 28) // (G * max(nk, 1)))
        for h in range(hkv):
            k, v = s["k"][b:b + nk, h].float(), s["v"][b:b + nk, h].float()
            for i in range(0, nq, step):
                m = min(step, nq - i)
                q = s["q"][a + i:a + i + m, h * G:(h + 1) * G].float().reshape(m * G, D)
                seen = (nk - nq + i + 1 + torch.arange(m, device="cuda")).repeat_interleave(G)[:, None]
                z = torch.matmul(q, k.t()) * (1 / math.sqrt(D))
                z = torch.where(torch.arange(nk, device="cuda") < seen, z, torch.full_like(z, -math.inf))
                p = torch.exp(z - z.amax(-1, keepdim=True).clamp(min=-1e30))
                o = torch.matmul(p, v) / p.sum(-1, keepdim=True).clamp(min=1e-30)
                out[a + i:a + i + m, h * G:(h + 1) * G] = o.view(m, G, D).bfloat16()
        a, b = a + nq, b + nk
    return out


def _run_attend(s):
    c = s["case"]
    n, ql, hkv, G, nb = c["n"], c["q_len"], c["hkv"], c["group"], s["nb"]
    if own:
        from block_sparse_paged_score_gb300 import bsp
        return bsp.dense_pa_decode_fp8(s["cache"], s["q"], bsp.FP8_E4M3 if c["q8"] else bsp.BF16, hkv * G, s["table"],
                                       s["row_seq"], s["row_len"], ql, out=s["out"], ws=s["ws"])
    q = (s["q"].view(torch.float8_e4m3fn) if c["q8"] else s["q"]).float()
    q = q.view(n, ql, hkv, G, D).transpose(1, 2).reshape(n, hkv, ql * G, D)
    k, v = _blocks_of(s, s["table"].long())  # [n, nb, Hkv, 128, 128]
    k, v = (x.transpose(1, 2).reshape(n, hkv, nb * BLK, D) for x in (k, v))
    z = torch.matmul(q, k.transpose(-1, -2)) * (1 / math.sqrt(D))
    seen = s["row_len"].view(n, ql, hkv).transpose(1, 2).repeat_interleave(G, 2)  # [n, Hkv, ql * G]
    z = torch.where(torch.arange(nb * BLK, device="cuda") < seen[..., None], z, torch.full_like(z, -math.inf))
    p = torch.exp(z - z.amax(-1, keepdim=True).clamp(min=-1e30))
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return o.view(n, hkv, ql, G, D).transpose(1, 2).reshape(n * ql, hkv * G, D).bfloat16()


def _run_write(s):
    if own:
        from block_sparse_paged_score_gb300 import bsp
        bsp.kv_scaled_write(s["cache"], s["k"], s["v"], s["slot"])
    else:
        hkv, nb = s["case"]["hkv"], s["blocks"]
        live = s["slot"] >= 0
        slot = s["slot"][live]
        blk, o = slot // BLK, slot % BLK
        touched = torch.zeros(nb + 1, dtype=torch.bool, device="cuda")
        fresh = torch.zeros_like(touched)
        touched[blk] = True
        fresh[blk[o == 0]] = True
        for side, x, scales in zip(_sides(s), (s["k"], s["v"]), (s["ks"], s["vs"])):
            x = x[live].float()
            top = torch.zeros(nb + 1, hkv, device="cuda").index_reduce_(0, blk, x.abs().amax(-1), "amax")
            m, e = torch.frexp(top)  # top = m 2^e, and 448 = 0.875 * 2^9
            e = torch.where(top > 0, e - 9 + (m > 0.875).int(), torch.full_like(e, LOW)).clamp(LOW, HIGH)
            want = torch.ldexp(torch.ones_like(top), e)
            want = torch.where(fresh[:, None], want, torch.maximum(want, scales))
            scale = torch.where(touched[:, None], want, scales)
            # the tokens that the grown blocks held
            grown = (touched & ~fresh & (scale > scales).any(-1)).nonzero()[:, 0]
            raw = side.view(torch.uint8)
            f = (scales[grown] / scale[grown]).view(-1, 1, hkv, *[1] * (side.dim() - 3))
            raw[grown] = _e4m3(raw[grown].view(torch.float8_e4m3fn).float() * f).view(torch.uint8)
            scales.copy_(scale)
            val = _e4m3(x / scale[blk][..., None]).view(torch.uint8)
            page, t = o // PG, o % PG
            raw[blk, page, :, :, t] = val.unflatten(-1, (D // 16, 16)) if side.dim() == 6 else val
    n = s["blocks"]
    return dict(kv=s["kv"].view(n + 1, -1)[:n].view(torch.float8_e4m3fn), ks=s["ks"][:n], vs=s["vs"][:n])


def _run_read(s):
    if own:
        from block_sparse_paged_score_gb300 import bsp
        k, v = bsp.kv_scaled_read(s["cache"], s["slot"], k=s["k"], v=s["v"])
        return dict(k=k, v=v)
    slot = torch.where(s["slot"] < 0, s["blocks"] * BLK, s["slot"])  # the spare block's for pad rows
    blk, o = slot // BLK, slot % BLK
    live = (s["slot"] >= 0)[:, None, None]
    out = {}
    for name, side, scales in zip("kv", _sides(s), (s["ks"], s["vs"])):
        x = side.view(torch.uint8)[blk, o // PG, :, :, o % PG].view(torch.float8_e4m3fn).float()
        x = (x.flatten(-2) if side.dim() == 6 else x) * scales[blk][..., None]
        out[name] = torch.where(live, x, torch.zeros_like(x)).bfloat16()
    return out


# ---- what a pass cannot do without -------------------------------------------
def _moments(lo, hi, ragged):
    """Means of a length and of its square, uniform from lo to hi, or always hi."""
    return ((lo + hi) / 2, (lo * lo + lo * hi + hi * hi) / 3) if ragged else (hi, hi * hi)


def work(c):
    hkv = c["hkv"]
    if c["op"] == "prompt":
        n, hq = c["n"], hkv * c["group"]
        new, new2 = _moments(c["new"] // 8, c["new"], c["ragged"])
        ctx, _ = _moments(c["ctx"] // 8, c["ctx"], c["ragged"])
        pairs = n * (new * ctx + (new2 + new) / 2)
        return dict(bytes=n * (new * hq * D * 4 + (new + ctx) * hkv * D * 4), flops=pairs * hq * D * 4)
    if c["op"] == "attend":
        tokens = c["n"] * c["ctx"] * (0.75 if c["ragged"] else 1)
        rows = c["n"] * c["q_len"] * hkv
        q = rows * c["group"] * D
        return dict(bytes=tokens * hkv * 256 + tokens / BLK * (4 + 8 * hkv) + q * ((1 if c["q8"] else 2) + 2) + rows * 8,
                    flops=tokens * hkv * c["q_len"] * c["group"] * D * 4)
    if c["op"] == "write":
        new, _ = _moments(c["new"] // 8, c["new"], c["ragged"])
        T = c["n"] * new
        return dict(bytes=T * (8 + 2 * hkv * D * 3) + (T / BLK + c["n"]) * hkv * 8, flops=T * 2 * hkv * D * 3)
    return dict(bytes=c["T"] * (8 + 2 * hkv * D * 3), flops=c["T"] * 2 * hkv * D)


# ---- the definitions in 64 bits ------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"prompt": _exact_prompt, "attend": _exact_attend, "write": _exact_write, "read": _exact_read}[case["op"]](s)


def _exact_rows(q, k, v, seen):
    """float64 attention of rows q [R, 128] over the first seen[r] of k, v [n, 128]."""
    z = (q @ k.t()) / D ** 0.5
    z = z.masked_fill(torch.arange(k.shape[0], device="cuda")[None] >= seen[:, None], -math.inf)
    w = torch.exp(z - torch.logsumexp(z, -1, keepdim=True))
    return torch.where(seen[:, None] > 0, w, torch.zeros_like(w)) @ v


def _exact_prompt(s):
    c = s["case"]
    hq, G = c["hkv"] * c["group"], c["group"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    cu_q, cu_k = s["cu_q"].tolist(), s["cu_k"].tolist()
    for a, a2, b, b2 in zip(cu_q, cu_q[1:], cu_k, cu_k[1:]):
        for head in range(hq):
            k, v = s["k"][b:b2, head // G].double(), s["v"][b:b2, head // G].double()
            lo = a
            while lo < a2:  # queries lo.. with the keys that the last of them sees
                hi = min(a2, lo + max(1, min(4096, (1 << 26) // max(1, b2 - b))))
                last = b2 - b - (a2 - hi)
                seen = last - (hi - 1 - torch.arange(lo, hi, device="cuda"))
                out[lo:hi, head] = _exact_rows(s["q"][lo:hi, head].double(), k[:last], v[:last], seen)
                lo = hi
    return out


def _e4m3_values():
    b = torch.arange(256, device="cuda")
    e, m = (b // 8 % 16).double(), (b % 8).double()
    x = torch.where(e > 0, (8 + m) * torch.exp2(e - 10), m * 2.0 ** -9)
    x[[127, 255]] = math.nan
    return torch.where(b >= 128, -x, x)


def _exact_tokens(s, slot, h):
    """float64 K and V [T, 128] of head h at the slots."""
    hkv, lut = s["case"]["hkv"], _e4m3_values()
    blk, o, d = slot // BLK, slot % BLK, torch.arange(D, device="cuda")
    k_page = ((blk * 16 + o // PG) * hkv + h) * (PG * D)
    k_at = k_page[:, None] + d // 16 * 256 + (o % PG)[:, None] * 16 + d % 16
    v_at = k_page[:, None] + 8 * hkv * PG * D + d * PG + (o % PG)[:, None]
    return (lut[s["kv"][k_at].int()] * s["ks"].double()[blk, h][:, None],
            lut[s["kv"][v_at].int()] * s["vs"].double()[blk, h][:, None])


def _exact_attend(s):
    c = s["case"]
    n, ql, hkv, G = c["n"], c["q_len"], c["hkv"], c["group"]
    q = (s["q"].view(torch.float8_e4m3fn) if c["q8"] else s["q"]).double().view(n, ql, hkv, G, D)
    seen = s["row_len"].view(n, ql, hkv)
    out = torch.zeros(n, ql, hkv, G, D, dtype=torch.float64, device="cuda")
    longest = seen.amax((1, 2)).tolist()
    for i in range(n):
        t = torch.arange(longest[i], device="cuda")
        slot = s["table"][i].long()[t // BLK] * BLK + t % BLK
        if longest[i] == 0:
            continue
        for h in range(hkv):
            k, v = _exact_tokens(s, slot, h)
            o = _exact_rows(q[i, :, h].reshape(ql * G, D), k, v, seen[i, :, h].repeat_interleave(G))
            out[i, :, h] = o.view(ql, G, D)
    return out.view(n * ql, hkv * G, D)


def _exact_e4m3(x):
    """float64 rounded to the e4m3 grid: steps of 2^(e-3), no finer than 2^-9, at most 448."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_write(s):
    hkv, nb, lut = s["case"]["hkv"], s["blocks"], _e4m3_values()
    page = lut[s["kv"].int()].view(nb + 1, 16, hkv, PG * D)[:nb].clone()
    slot = s["slot"][s["slot"] >= 0]
    blk, o = slot // BLK, slot % BLK
    order = torch.argsort(blk, stable=True)
    ids, count = torch.unique_consecutive(blk[order], return_counts=True)
    first = torch.cumsum(count, 0) - count
    anew = torch.zeros(nb, dtype=torch.float64, device="cuda").index_add_(0, blk, (o == 0).double()) > 0
    out = {}
    for half, x, name in ((page[:, :8], s["k"], "ks"), (page[:, 8:], s["v"], "vs")):
        x = x[s["slot"] >= 0].double()
        top = torch.segment_reduce(x.abs().amax(-1)[order], "max", lengths=count)  # [touched, Hkv]
        low = torch.floor(torch.log2((top / 448).clamp(min=2.0 ** -200))) - 1
        e = (low + sum((448 * torch.exp2(low + i) < top).double() for i in range(4))).clamp(LOW, HIGH)
        old = s[name].double()[:nb]
        new = old.clone()
        new[ids] = torch.where(anew[ids][:, None], torch.exp2(e), torch.maximum(torch.exp2(e), old[ids]))
        grew = (new > old) & ~anew[:, None]
        which = grew.any(-1).nonzero()[:, 0]
        ratio = (old / new)[which][:, None, :, None]
        half[which] = torch.where(ratio < 1, _exact_e4m3(half[which] * ratio), half[which])
        val = _exact_e4m3(x / new[blk][..., None])
        h = torch.arange(hkv, device="cuda")[None, :, None]
        d, t = torch.arange(D, device="cuda")[None, None], (o % PG)[:, None, None]
        at = d // 16 * 256 + t * 16 + d % 16 if name == "ks" else d * PG + t
        half[blk[:, None, None], (o // PG)[:, None, None], h, at] = val
        out[name] = new
    return dict(kv=page.view(nb, -1), ks=out["ks"], vs=out["vs"])


def _exact_read(s):
    ok = (s["slot"] >= 0).double()[:, None]
    heads = [_exact_tokens(s, s["slot"].clamp(min=0), h) for h in range(s["case"]["hkv"])]
    return dict(k=torch.stack([k * ok for k, _ in heads], 1), v=torch.stack([v * ok for _, v in heads], 1))
