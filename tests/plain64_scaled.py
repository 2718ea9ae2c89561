"""Plain 64-bit forms of the block-scaled cache's write and read and of the
prompt attention on the CPU (numpy), token by token from their definitions."""
import math

import numpy as np

from plain64 import E4M3, bf16_to_f64

# the finite e4m3 values in order, for rounding by table
_CODES = np.array([b for b in range(127)])
_VALUES = E4M3[_CODES]


def e4m3(x):
    """float64 -> e4m3 bytes, to nearest, ties to the even code, saturating; NaN stays NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.searchsorted(_VALUES, np.where(np.isnan(a), 0, a))  # the first value >= a
    lo = np.maximum(hi - 1, 0)
    d_hi, d_lo = _VALUES[hi] - a, a - _VALUES[lo]
    code = np.where((d_lo < d_hi) | ((d_lo == d_hi) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.isnan(x), 127, code)
    return (code + 128 * np.signbit(x)).astype(np.uint8)


def addresses(hkv, blk, off, h, side):
    """byte numbers of the 128 dims of a token in a packed interleaved fp8 cache"""
    d = np.arange(128)
    page = ((blk * 16 + 8 * side + off // 16) * hkv + h) * 2048
    return page + (d // 16 * 256 + off % 16 * 16 + d % 16 if side == 0 else d * 16 + off % 16)


def block_addresses(hkv, blk, h, side):
    return np.stack([addresses(hkv, blk, o, h, side) for o in range(128)])


def block_values(cache, scales, hkv, blk, h, side):
    """float64 [128 tokens, 128] of one block"""
    return E4M3[cache[block_addresses(hkv, blk, h, side)]] * float(scales[side][blk, h])


def least_scale(a):
    e = -60
    while e < 119 and 448.0 * 2.0 ** e < a:
        e += 1
    return 2.0 ** e


def scaled_write(cache, scales, hkv, k, v, slot, num_blocks):
    """The definition, run by run: k, v float64 [T, Hkv, 128]; cache bytes and
    scales [K, V] are changed in place.  Returns the error bits."""
    err, i, T = 0, 0, len(slot)
    blk = [s // 128 if 0 <= s < num_blocks * 128 else -1 for s in slot]
    err |= 16 if any(s >= num_blocks * 128 for s in slot) else 0
    while i < T:
        j = i + 1
        while j < T and blk[j] == blk[i]:
            j += 1
        b = blk[i]
        if b >= 0:
            last = {int(slot[t]) % 128: t for t in range(i, j)}  # the last token of a slot
            for side, x in ((0, k), (1, v)):
                for h in range(hkv):
                    rows = np.abs(x[list(last.values()), h])
                    fin = rows[np.isfinite(rows)]
                    run = least_scale(fin.max() if fin.size else 0.0)
                    old = float(scales[side][b, h])
                    s = run if 0 in last else max(run, old)
                    if 0 not in last and s > old:
                        for o in range(128):
                            if o not in last:
                                at = addresses(hkv, b, o, h, side)
                                nan = (cache[at] & 127) == 127
                                new = e4m3(E4M3[cache[at]] * (old / s))
                                cache[at] = np.where(nan, cache[at] | 127, new)
                    for o, t in last.items():
                        cache[addresses(hkv, b, o, h, side)] = e4m3(x[t, h] / s)
                    scales[side][b, h] = s
        i = j
    return err


def prompt(q, k, v, cu_q, cu_k, scale):
    """float64 q [T, Hq, 128], k, v [K, Hkv, 128] -> (o, a): the attention and
    sum p |v| / sum p; rows of no sequence are NaN."""
    T, hq, _ = q.shape
    hkv = k.shape[1]
    g = hq // hkv
    o, a = np.full(q.shape, math.nan), np.full(q.shape, math.nan)
    for s in range(len(cu_q) - 1):
        q0, q1, k0, k1 = cu_q[s], cu_q[s + 1], cu_k[s], cu_k[s + 1]
        for h in range(hkv):
            kk, vv = k[k0:k1, h], v[k0:k1, h]
            for i in range(q1 - q0):
                n = max(0, (k1 - k0) - (q1 - q0) + i + 1)
                rows = slice(h * g, (h + 1) * g)
                if n == 0:
                    o[q0 + i, rows] = a[q0 + i, rows] = 0
                    continue
                z = q[q0 + i, rows] @ kk[:n].T * scale
                p = np.exp(z - z.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                o[q0 + i, rows] = p @ vv[:n]
                a[q0 + i, rows] = p @ np.abs(vv[:n])
    return o, a


def bits_f64(t):
    """a bf16 torch tensor as float64 numpy"""
    return bf16_to_f64(t.detach().cpu().contiguous().view(__import__("torch").int16).numpy().view(np.uint16))
