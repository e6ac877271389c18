"""The scaled-cache calls where precision is lost first, against the 64-bit
oracle, with bounds from the arithmetic:

* a weight times its block's V scale is rounded to fp16: off by 2^-11 of itself,
  or by half of the subnormal step, but never by more than itself.  That half
  step is 2^-31 of the largest weight in the prefill (weights are held times
  2^6), 2^-30 of the largest weight times the largest scale in the decode (held
  times at least 2^5);
* the prefill holds codes times a power of two relative to the largest scale in
  fp16: exact down to 2^-22 of it, else off by 2^-31 of the largest scale (half
  of fp16's smallest step at 2^7 units, times less than 2 for the rest);
* scores: the matrix unit adds 16 products at a time to an fp32 sum, up to
  D / 16 + 8 truncations of 2^-23 of sum |q k| scale (16 of them at most, with
  the two factors behind it), in numerator and denominator alike;
* exponentials, sums and the division in fp32: 2^-18 of sum p |v|;
* the output's own rounding: half a step of its type.
"""
import numpy as np
import pytest
import torch

import harness as H
from oracle import scaled as OS
from test_gpu_scaled import TD, Batch

from paged_kv_cache_130_gb300 import workloads as W

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -11


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    H.build_library()


def bounds(b, scale, decode):
    """The bound above on every output, before the output's own rounding."""
    err = np.zeros(b.q.shape)
    G = b.heads // b.kv
    for s, c in enumerate(int(x) for x in b.ctx):
        n = int(b.cu[s + 1] - b.cu[s])
        if c == 0 or n == 0:
            continue
        rows = slice(int(b.cu[s]), int(b.cu[s + 1]))
        ids = b.tables[s, :-(-c // b.bs)]
        for h in range(b.kv):
            ks, vs = (b.scales[ids, h, i].astype(np.float64).repeat(b.bs)[:c] for i in range(2))
            k = OS.gather(b.k, b.scales, 0, b.tables[s], c, h)
            v = np.abs(OS.gather(b.v, b.scales, 1, b.tables[s], c, h))
            q = b.q[rows, h * G:(h + 1) * G]
            x = np.einsum("ngd,td->ngt", q, k) * scale
            hidden = np.arange(c)[None] > (c - n + np.arange(n))[:, None]
            x = np.where(hidden[:, None], -np.inf, x)
            w = np.exp(x - x.max(-1, keepdims=True))
            size = (np.einsum("ngd,td->ngt", np.abs(q), np.abs(k)) * abs(scale)).max(-1)
            ds = 16 * 2.0 ** -23 * size
            if decode:
                floor, dv = 2.0 ** -30 * vs.max() / vs, 0.0
            else:
                floor = 2.0 ** -31
                dv = np.where(vs < 2.0 ** -22 * vs.max(), 2.0 ** -31 * vs.max(), 0.0)
                if (ks < 2.0 ** -22 * ks.max()).any():
                    ds = ds + abs(scale) * np.abs(q).sum(-1) * 2.0 ** -31 * ks.max()
            rel = EPS + 2.0 ** -18 + 2 * ds
            e = np.einsum("ngt,td->ngd", w * rel[..., None] + np.minimum(w, floor), v)
            e = e + (w * dv).sum(-1)[..., None]
            err[rows, h * G:(h + 1) * G] = e / w.sum(-1)[..., None]
    return err


def assert_within(got, b, scale, what, decode):
    ref, err = b.attention(scale), bounds(b, scale, decode)
    bound = err + torch.finfo(TD[b.dt]).eps / 2 * (np.abs(ref) + err)
    bound = bound + (2.0 ** -25 if b.dt == W.F16 else 0.0)
    off = np.abs(H.out_to_double(got) - ref)
    assert (off <= bound).all(), (what, float((off / np.maximum(bound, 1e-300)).max()), off.max())
    assert int(b.err.item()) == 0


def long_batch(seed, dt, heads, kv, d, bs, n, new=1):
    """`new` tokens at the end of one context of n: codes of 0, scales of 1."""
    b = Batch(seed, dt, heads, kv, d, bs, [new], [0])
    b.nb = -(-n // bs) + 3
    b.tables = b.r.permutation(b.nb).astype(np.int32)[None, :-(-n // bs)].copy()
    b.k, b.v = (np.zeros((b.nb, kv, bs, d), np.uint8) for _ in range(2))
    b.scales = np.ones((b.nb, kv, 2), np.float32)
    b.ctx = np.array([n], np.int32)
    return b


def random_codes(b):
    """Normal values at the blocks' scales, codes up to 64 or so."""
    from oracle import encode_e4m3
    for t in (b.k, b.v):
        t[...] = encode_e4m3((b.r.standard_normal(t.shape) * 16).astype(np.float32))


@pytest.mark.parametrize("dt,bs,n", [(W.F16, 16, 32768), (W.BF16, 32, 131072)])
def test_faint_weights_behind_one_large_one(dt, bs, n):
    """One key 17.5 nats above all others, whose V is 0: what the others bring
    is the output, and grows with the context."""
    b = long_batch(200, dt, 2, 1, 64, bs, n)
    b.v[...] = 0x7e                                # 448
    first = b.tables[0, 0]
    b.k[first, 0, 5, 0] = 0x38                     # 1
    b.v[first, 0, 5] = 0
    b.q[...] = 0
    b.q[..., 0] = 1
    b.upload()
    assert 0.3 < b.attention(17.5).max() < 2
    assert_within(b.prefill(17.5), b, 17.5, "prefill", False)
    assert_within(b.decode(17.5), b, 17.5, "decode", True)


SCALES = [
    # dtype, heads, kv, D, bs, new, cached
    (W.F16, 4, 2, 64, 8, [3, 130, 1], [700, 40, 0]),
    (W.BF16, 8, 1, 128, 16, [40, 300], [500, 0]),
    (W.F16, 16, 2, 128, 32, [20, 1, 17], [100, 1100, 15]),
]


@pytest.mark.parametrize("i", range(len(SCALES)))
def test_scales_that_are_no_powers_of_two(i):
    """A cache quantised by its largest value: any fp32 scale, sharp scores."""
    dt, h, kv, d, bs, new, cached = SCALES[i]
    b = Batch(210 + i, dt, h, kv, d, bs, new, cached, size=1.0, spread=1.0)
    b.oracle_append()
    b.scales = (b.scales * b.r.uniform(1, 2, b.scales.shape)).astype(np.float32)
    b.upload()
    scale = 5 / np.sqrt(d)
    assert_within(b.prefill(scale), b, scale, "prefill", False)
    # each sequence's last token alone
    b.q = np.ascontiguousarray(b.q[b.cu[1:] - 1])
    b.cu = np.arange(len(new) + 1, dtype=np.int32)
    assert_within(b.decode(scale), b, scale, "decode", True)


@pytest.mark.parametrize("which,log2", [("v", 18), ("v", 22), ("v", 30), ("k", 18), ("k", 22), ("k", 26)])
def test_one_block_far_above_the_others(which, log2):
    """The largest scale of a long context sits in its 600th block; those keys
    have next to no weight (V) or nothing to do with q (K), and the other
    blocks keep what the bound says."""
    d, bs = 64, 8
    b = long_batch(220 + log2, W.F16, 4, 1, d, bs, 700 * bs - 3, new=3)
    random_codes(b)
    b.scales[...] = 2.0 ** -4 * b.r.uniform(1, 2, b.scales.shape) if log2 == 18 else 2.0 ** -4
    big = b.tables[0, 600]
    b.q[..., :16] = 0
    if which == "v":
        b.scales[big, 0, 1] = 2.0 ** (log2 - 4)
        b.q[..., 16] = 4
        b.k[big] = 0
        b.k[big, :, :, 16] = 0xfe                  # -448: scores of -14 and less
    else:
        b.scales[big, 0, 0] = 2.0 ** (log2 - 4)
        b.k[big, :, :, 16:] = 0
        assert (b.k[big, :, :, :16] != 0).any()
    b.upload()
    scale = 0.125
    assert_within(b.prefill(scale), b, scale, "prefill", False)
    b.q, b.cu = np.ascontiguousarray(b.q[-1:]), np.array([0, 1], np.int32)
    assert_within(b.decode(scale), b, scale, "decode", True)
