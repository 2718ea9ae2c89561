"""Plain 64-bit forms of the step-table, norm-and-rotation, cache-read and
dense-attention operators on the CPU (numpy), and the decoding of cache bytes
they share.  Independent of the library and of the C oracle."""
import math

import numpy as np

BF16, FP8, MX = 0, 1, 2
FIELD = 8704


def bf16_to_f64(bits):
    return (np.ascontiguousarray(bits).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def f64_to_bf16(x):
    """float -> bf16 bits, round to nearest even."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def _e4m3_table():
    out = np.zeros(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[b] = math.nan if (b & 127) == 127 else (-v if b & 128 else v)
    return out


E4M3 = _e4m3_table()
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def mx_field(field):
    """[8704] bytes -> float64 [128 tokens, 128 dims]"""
    d, s = field[:8192].reshape(128, 64), field[8192:].reshape(128, 4)
    v = np.empty((128, 128))
    v[:, 0::2], v[:, 1::2] = E2M1[d & 15], E2M1[d >> 4]
    return v * np.repeat(2.0 ** (s.astype(np.float64) - 127), 32, axis=1)


def kv_token(cache, dtype, hkv, slot, k_scale=1.0, v_scale=1.0):
    """(K, V) float64 [Hkv, 128] of one slot of a packed cache's bytes."""
    blk, o = divmod(int(slot), 128)
    k, v = np.zeros((hkv, 128)), np.zeros((hkv, 128))
    d = np.arange(128)
    for h in range(hkv):
        if dtype == MX:
            base = blk * 2 * hkv * FIELD
            k[h] = mx_row(cache[base + h * FIELD:], o)
            v[h] = mx_row(cache[base + (hkv + h) * FIELD:], o)
            continue
        x = 8 if dtype == BF16 else 16
        t = o % 16
        page = ((blk * 16 + o // 16) * hkv + h) * 2048
        vpage = page + 8 * hkv * 2048
        ke, ve = page + (d // x) * 16 * x + t * x + d % x, vpage + (t // x) * 128 * x + d * x + t % x
        if dtype == BF16:
            w = cache.view(np.uint16)
            k[h], v[h] = bf16_to_f64(w[ke]), bf16_to_f64(w[ve])
        else:
            k[h], v[h] = E4M3[cache[ke]] * k_scale, E4M3[cache[ve]] * v_scale
    return k, v


def mx_row(field, o):
    """token o of a field's bytes -> float64 [128]"""
    d, s = field[o * 64:o * 64 + 64], field[8192 + 4 * o:8192 + 4 * o + 4]
    v = np.empty(128)
    v[0::2], v[1::2] = E2M1[d & 15], E2M1[d >> 4]
    return v * np.repeat(2.0 ** (s.astype(np.float64) - 127), 32)


def idx_token(cache, dtype, heads, slot):
    """(values float64 [heads, 128], scales float64 [heads]) of one slot of a
    packed index cache; values of an fp8 cache are before the scale."""
    size = {BF16: 32768, FP8: 16896, MX: FIELD}[dtype]
    blk, o = divmod(int(slot), 128)
    out, sc = np.zeros((heads, 128)), np.ones(heads)
    for h in range(heads):
        f = cache[(blk * heads + h) * size:(blk * heads + h + 1) * size]
        if dtype == BF16:
            out[h] = bf16_to_f64(f.view(np.uint16)[o * 128:o * 128 + 128])
        elif dtype == FP8:
            out[h] = E4M3[f[o * 128:o * 128 + 128]]
            sc[h] = float(f[16384:].view(np.float32)[o])
        else:
            out[h] = mx_row(f, o)
    return out, sc


def step_tables(context, new, table, free, head, capacity, num_blocks):
    """The definition of bsp_step_tables, request by request; also the error bits."""
    table = table.copy()
    n, width = table.shape
    err = 0
    slot, req, pos = [-1] * capacity, [0] * capacity, [-1] * capacity
    cu, lens, taken, t = [], [], 0, 0

    def fresh(j):
        nonlocal err
        if not 0 <= head + j < len(free):
            err |= 32
            return -1
        b = int(free[head + j])
        if not 0 <= b < num_blocks:
            err |= 2
            return -1
        return b

    for s in range(n):
        c, m = max(int(context[s]), 0), max(int(new[s]), 0)
        cu.append(min(t, capacity))
        lens.append(c + m)
        have, want = min(-(-c // 128), width), min(-(-(c + m) // 128), width)
        for i in range(want - have):
            table[s, have + i] = fresh(taken + i)
        for i in range(m):
            if t + i >= capacity:
                err |= 32
                break
            p = c + i
            req[t + i], pos[t + i] = s, p
            if p // 128 >= width:
                err |= 32
                continue
            b = int(table[s, p // 128])
            if p // 128 < have and not 0 <= b < num_blocks:
                err |= 2
                b = -1
            if b >= 0:
                slot[t + i] = b * 128 + p % 128
        t += m
        taken += want - have
    cu.append(min(t, capacity))
    return dict(block_table=table, seq_lens=np.array(lens, np.int32), cu_tokens=np.array(cu, np.int32),
                blocks_taken=np.array([taken], np.int32), slot=np.array(slot, np.int64),
                query_req_id=np.array(req, np.int32), query_abs_pos=np.array(pos, np.int32)), err


def norm_rope(x, weight, offset, eps, rope, rot, pairs, positions):
    """float64 x [T, H, 128] -> (rows, pair magnitudes hypot(y_a, y_b) of the
    rotated dims, |y| of the others); pad rows are zero."""
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if weight is not None:
        y = y * (weight + offset)
    mag = np.abs(y)
    if rot:
        h = rot // 2
        cs = rope[np.maximum(positions, 0)][:, None].astype(np.float64)
        c, s = cs[..., :h], cs[..., h:]
        ia = np.arange(0, rot, 2) if pairs else np.arange(h)
        ib = ia + 1 if pairs else ia + h
        a, b = y[..., ia], y[..., ib]
        y = y.copy()
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        mag[..., ia] = mag[..., ib] = np.hypot(a, b)
    y[positions < 0] = 0
    return y, mag


def dense_attention(fields_of, table, q, row_seq, row_len, hkv, group, scale):
    """fields_of(block, side, head) -> float64 [128, 128].  q float64 [tokens,
    Hkv*G, 128].  Returns (o, a): the attention and sum p |v| / sum p."""
    tokens = q.shape[0]
    o, a = np.zeros((tokens, hkv * group, 128)), np.zeros((tokens, hkv * group, 128))
    width = table.shape[1]
    kept = {}

    def rows(seq, h, n):
        if (seq, h) not in kept:
            nb = max(-(-int(min(max(row_len[r], 0), width * 128)) // 128)
                     for r in range(len(row_len)) if row_seq[r] == seq)
            kept[seq, h] = [np.concatenate([fields_of(table[seq, b], side, h) for b in range(nb)]) if nb else
                            np.zeros((0, 128)) for side in (0, 1)]
        return [x[:n] for x in kept[seq, h]]

    for r in range(tokens * hkv):
        t, h = divmod(r, hkv)
        n = int(min(max(row_len[r], 0), width * 128))
        if n == 0:
            continue
        k, v = rows(int(row_seq[r]), h, n)
        z = q[t, h * group:(h + 1) * group] @ k.T * scale
        p = np.exp(z - z.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        o[t, h * group:(h + 1) * group] = p @ v
        a[t, h * group:(h + 1) * group] = p @ np.abs(v)
    return o, a
