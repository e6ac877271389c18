"""The 8-bit cache with a scale per block and KV head, and the rotary append,
in 64 bits from their definitions: numpy loops that share no code with the
library.  Caches are E4M3 codes (uint8) [num_blocks, num_kv_heads, block_size,
head_dim], scales float32 [num_blocks, num_kv_heads, 2] (K, V)."""
import numpy as np

from . import E4M3, decode as dec, encode_e4m3


def power_of_two_scale(bound):
    """Smallest power of two s >= 2^-126 with bound <= 448 s."""
    e = -126
    while float(bound) > 448.0 * 2.0 ** e:
        e += 1
    return np.float32(2.0 ** e)


def rotate(x, positions, inv_freq, interleaved=False, mscale=1.0):
    """x float64 [rows, heads, D] turned by positions [rows]."""
    y = np.array(x, np.float64)
    r = 2 * len(inv_freq)
    ang = np.asarray(positions, np.longdouble)[:, None] * np.asarray(inv_freq, np.longdouble)
    c = (np.cos(ang)[:, None] * mscale).astype(np.float64)
    s = (np.sin(ang)[:, None] * mscale).astype(np.float64)
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y[..., :r // 2], y[..., r // 2:r] = a * c - b * s, b * c + a * s
    return y


def append_scaled(codes, scales, which, new, raw, factor, cu, tables, ctx):
    """Append rows `new` (float64 [rows, Hkv, D], to be rounded; `raw` the rows
    before the rotation) to `codes` (K: which 0, V: which 1), in place."""
    bs = codes.shape[2]
    for s in range(len(ctx)):
        n = int(cu[s + 1] - cu[s])
        first = int(ctx[s]) - n
        for b in range(first // bs, -(-int(ctx[s]) // bs) if n else 0):
            lo, hi = max(first, b * bs), min(int(ctx[s]), (b + 1) * bs)
            phys = int(tables[s, b])
            rows = slice(int(cu[s]) + lo - first, int(cu[s]) + hi - first)
            for h in range(codes.shape[1]):
                a = np.abs(raw[rows, h])
                a = a[np.isfinite(a)]
                amax = np.float32(a.max()) if a.size else np.float32(0)
                need = power_of_two_scale(np.float32(amax * np.float32(factor)))
                sc = need
                if lo > b * bs:
                    old = scales[phys, h, which]
                    sc = max(old, need)
                    if sc != old:
                        # every slot; those of the new tokens are written below
                        o = codes[phys, h]
                        o[...] = encode_e4m3((dec(E4M3, o) * (float(old) / float(sc))).astype(np.float32))
                scales[phys, h, which] = sc
                # sc is a power of two: the fp32 quotient is the value's own rounding
                codes[phys, h, lo - b * bs:hi - b * bs] = encode_e4m3(
                    (new[rows, h].astype(np.float32) / sc).astype(np.float32))


def gather(codes, scales, which, table, c, head):
    """Values [c, D] of one KV head in logical order."""
    bs = codes.shape[2]
    ids = np.asarray(table[:-(-c // bs)], np.int64)
    x = dec(E4M3, np.ascontiguousarray(codes[ids, head])) * \
        scales[ids, head, which].astype(np.float64)[:, None, None]
    return x.reshape(-1, codes.shape[3])[:c]


def attention(k_codes, v_codes, scales, q, cu, tables, ctx, scale):
    """Causal attention of the rows of q (float64 [rows, H, D]), the last tokens
    of each context; a decode has one row per sequence (or none in its
    context: zeros)."""
    out = np.zeros(q.shape, np.float64)
    hkv = k_codes.shape[1]
    G = q.shape[1] // hkv
    for s in range(len(ctx)):
        n, c = int(cu[s + 1] - cu[s]), int(ctx[s])
        if c == 0:
            continue
        rows = slice(int(cu[s]), int(cu[s + 1]))
        for h in range(hkv):
            k = gather(k_codes, scales, 0, tables[s], c, h)
            v = gather(v_codes, scales, 1, tables[s], c, h)
            x = np.einsum("ngd,td->ngt", q[rows, h * G:(h + 1) * G], k) * scale
            hidden = np.arange(c)[None] > (c - n + np.arange(n))[:, None]
            x = np.where(hidden[:, None], -np.inf, x)
            p = np.exp(x - x.max(-1, keepdims=True))
            p = p / p.sum(-1, keepdims=True)
            o = np.einsum("ngt,td->ngd", p, np.nan_to_num(v, nan=0.0))
            # a NaN of V reaches exactly the rows that see its token
            seen = (~hidden).astype(np.int64) @ np.isnan(v).astype(np.int64) > 0
            out[rows, h * G:(h + 1) * G] = np.where(seen[:, None], np.nan, o)
    return out
