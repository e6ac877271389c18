"""Attention weights and eviction in 64 bits from their definitions: numpy loops
that share no code with the library."""
import numpy as np


def weights(keys, q, cu, window, ctx, scale):
    """Totals float64 [num_seqs, kv_heads, max(ctx)] that the last `window` rows of
    q (float64 [rows, H, D]) of each sequence add, and the largest sum of
    |scale q k| over the rows and keys that take part, which a rounding error of a
    score is relative to.  keys(s, h): float64 [ctx[s], D]."""
    hkv = keys.heads
    G = q.shape[1] // hkv
    out = np.zeros((len(ctx), hkv, max(1, int(max(ctx)))), np.float64)
    size = 0.0
    for s, c in enumerate(int(x) for x in ctx):
        n = min(int(cu[s + 1] - cu[s]), window)
        if n == 0 or c == 0:
            continue
        rows = q[int(cu[s + 1]) - n:int(cu[s + 1])]
        for h in range(hkv):
            k = keys(s, h)
            r = rows[:, h * G:(h + 1) * G]
            x = np.einsum("ngd,td->ngt", r, k) * scale
            size = max(size, abs(scale) * float(np.einsum("ngd,td->ngt", abs(r), abs(k)).max()))
            hidden = np.arange(c)[None] > (c - n + np.arange(n))[:, None]
            x = np.where(hidden[:, None], -np.inf, x)
            p = np.exp(x - x.max(-1, keepdims=True))
            # (a row whose sum is NaN does not reach the keys it does not see)
            out[s, h, :c] = np.where(hidden[:, None], 0.0, p / p.sum(-1, keepdims=True)).sum((0, 1))
    return out, size


def kept(w, n, first, last):
    """Indexes, in order, of the n of len(w) tokens that stay."""
    c = len(w)
    last = min(last, n)
    first = min(first, n - last)
    stay = list(range(first)) + list(range(c - last, c))
    order = sorted(range(first, c - last),
                   key=lambda i: (-np.inf if np.isnan(w[i]) else float(w[i])), reverse=True)
    # (sorted keeps equal ones in their order, also in reverse)
    return np.array(sorted(stay + order[:n - first - last]), np.int64)
