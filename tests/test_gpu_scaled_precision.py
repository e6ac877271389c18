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


def with_output(b, ref, err):
    """err and the output's own rounding."""
    return err + torch.finfo(TD[b.dt]).eps / 2 * (np.abs(ref) + err) + \
        (2.0 ** -25 if b.dt == W.F16 else 0.0)


def assert_within(got, b, scale, what, decode):
    ref = b.attention(scale)
    bound = with_output(b, ref, bounds(b, scale, decode))
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
    (W.BF16, 6, 2, 128, 8, [129, 2], [900, 0]),
    (W.F16, 7, 1, 64, 32, [50], [1400]),
    (W.BF16, 2, 2, 64, 16, [300, 9], [0, 2000]),
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


@pytest.mark.parametrize("partition", [0, 64, 1024])
@pytest.mark.parametrize("heads,kv,d,bs,n,hi", [
    (6, 2, 64, 8, 60, 1500), (16, 1, 128, 16, 3, 4000), (4, 4, 128, 32, 9, 2000),
    (8, 1, 64, 16, 1, 5000), (2, 2, 64, 16, 300, 1100), (24, 2, 128, 8, 33, 3000)])
def test_every_token_counts_once_wherever_shares_are_cut(heads, kv, d, bs, n, hi, partition):
    """Equal weights, and V of token t in channel t mod D alone: a token lost or
    counted twice changes its channel by one part in (tokens / D), several times
    the bound.  Lengths around every multiple that matters."""
    r = np.random.default_rng(400 + n)
    edges = np.array([0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 191, 192, 193, 1023, 1024, 1025])
    ctx = np.where(r.random(n) < 0.4, edges[r.integers(0, len(edges), n)], r.integers(0, hi, n))
    ctx[-1] = hi
    b = Batch(401, W.F16, heads, kv, d, bs, [1] * n, ctx, fill=False)
    b.ctx = ctx.astype(np.int32)
    b.k[...] = 0
    b.v[...] = 0
    b.scales[...] = 1
    for s, c in enumerate(b.ctx):
        t = np.arange(c)
        phys = b.tables[s, t // bs]
        for h in range(kv):
            b.scales[phys, h, 1] = 2.0 ** r.integers(-3, 4)
            b.v[phys, h, t % bs, t % d] = 0x38 + r.integers(0, 8, c)      # 1 to 15 / 8
    b.upload()
    if partition == 0:
        from paged_kv_cache_130_gb300 import binding as B
        assert B.pkv_decode_scaled_partition_size(b.desc, n, heads, hi) == 0
    bound = with_output(b, b.attention(0.125), bounds(b, 0.125, True))
    for s, c in enumerate(b.ctx):
        for h in range(kv):
            if c:
                token = b.scales[b.tables[s, 0], h, 1] / c
                assert token > 5 * bound[s, h * heads // kv:(h + 1) * heads // kv].max()
    assert_within(b.decode(0.125, partition_size=partition), b, 0.125, "tokens", True)


@pytest.mark.parametrize("bs", [8, 16, 32])
def test_append_beside_a_scale_of_the_callers(bs):
    """A part-filled block whose scale is no power of two: kept while it is large
    enough, its codes re-rounded to the new one otherwise."""
    import oracle
    r = np.random.default_rng(500 + bs)
    new = 3
    for k_scale, v_scale in ((0.7, 0.3), (0.7, 1e-3), (1e-4, 0.0123)):
        b = Batch(501, W.BF16, 2, 2, 64, bs, [new], [bs + 2], fill=False)
        phys = b.tables[0, 1]
        b.k[phys], b.v[phys] = (r.integers(0, 0x7f, b.k[phys].shape) for _ in range(2))
        b.scales[phys, :, 0], b.scales[phys, :, 1] = k_scale, v_scale
        b.upload()
        b.append(None)
        torch.cuda.synchronize()
        for i, (codes, x) in enumerate(((b.k, b.nk), (b.v, b.nv))):
            got = (b.gk, b.gv)[i].cpu().numpy()
            for h in range(2):
                old = b.scales[phys, h, i]
                need = OS.power_of_two_scale(np.float32(np.abs(x[:, h]).max()))
                sc = max(old, need)
                want = codes[phys, h].copy()
                if sc != old:
                    want = oracle.encode_e4m3((oracle.decode(oracle.E4M3, want) *
                                               (float(old) / float(sc))).astype(np.float32))
                want[2:2 + new] = oracle.encode_e4m3(x[:, h].astype(np.float32) *
                                                     (np.float32(1) / sc))
                assert b.gs[phys, h, i].item() == sc
                assert np.array_equal(got[phys, h], want), (k_scale, v_scale, i, h)
        assert int(b.err.item()) == 0
