"""The scaled 8-bit cache (a power-of-two scale per block and KV head) and the
rotary append against the 64-bit oracle (oracle/scaled.py).

Bounds, from the arithmetic:
* rotated values: the fp32 cosine and sine are off by at most 2^-21 (a half
  turn's fraction rounded to 24 bits gives pi 2^-25, sincospi itself 2^-22), the
  two products and the sum by 2^-23 of |a| + |b|; e = 2^-20 m (|a| + |b|) covers
  both.  Then one rounding: half a step of the 16-bit type, or of E4M3 (2^-4 of
  the code, half a subnormal step 2^-10) times the scale.
* scales, V's codes, and K's codes without a rotation: exact.
* attention: 2e-3 + 2e-3 |ref|, plus half a bf16 step (harness): the weights are
  rounded to fp16 (2^-12 each), scores carry fp32 sums of exact products.
Unwritten slots hold 0xFF (NaN codes) and unused scales NaN, so that a read of
either shows.
"""
import numpy as np
import pytest
import torch

import harness as H
import oracle
from oracle import scaled as OS
from paged_kv_cache_130_gb300 import binding as B
from paged_kv_cache_130_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    H.build_library()


TD = {W.F16: torch.float16, W.BF16: torch.bfloat16}


class Batch:
    """Sequences with `new` tokens after `cached` ones over a scattered pool.
    Host copies (codes, scales) evolve through the oracle, device ones through
    the library; both start from the same cached tokens."""

    def __init__(self, seed, dt, heads, kv, d, bs, new, cached, size=1.0, spread=0.0, fill=True):
        r = self.r = np.random.default_rng(seed)
        self.dt, self.heads, self.kv, self.d, self.bs = dt, heads, kv, d, bs
        self.new, self.cached = np.asarray(new), np.asarray(cached)
        self.ctx = (self.new + self.cached).astype(np.int32)
        self.cu = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        counts = -(-self.ctx // bs)
        self.nb = int(counts.sum()) + 5
        order = r.permutation(self.nb).astype(np.int32)
        self.tables = np.full((len(self.ctx), max(1, int(counts.max()))), -1, np.int32)
        at = 0
        for i, n in enumerate(counts):
            self.tables[i, :n] = order[at:at + n]
            at += n
        shape = (self.nb, kv, bs, d)
        self.k, self.v = np.full(shape, 0xff, np.uint8), np.full(shape, 0xff, np.uint8)
        self.scales = np.full((self.nb, kv, 2), np.nan, np.float32)
        self.size, self.spread = size, spread
        if fill and self.cached.sum():
            n = int(self.cached.sum())
            cu = np.concatenate([[0], np.cumsum(self.cached)])
            for w, c in ((0, self.k), (1, self.v)):
                x = self.values(n, kv)
                OS.append_scaled(c, self.scales, w, x, x, 1.0, cu, self.tables, self.cached)
        rows = int(self.cu[-1])
        self.q = self.values(rows, heads, 1.0, 0.0)
        self.nk, self.nv = self.values(rows, kv), self.values(rows, kv)
        self.upload()

    def values(self, rows, heads, size=None, spread=None):
        size, spread = (self.size if size is None else size), (self.spread if spread is None else spread)
        x = self.r.standard_normal((rows, heads, self.d)) * size
        x = x * np.exp2(np.round(spread * self.r.standard_normal((rows, heads, 1))))
        return torch.from_numpy(x).to(TD[self.dt]).double().numpy()

    def dev16(self, x):
        return torch.from_numpy(np.ascontiguousarray(x)).to(TD[self.dt]).cuda()

    def upload(self):
        self.gk, self.gv = torch.from_numpy(self.k.copy()).cuda(), torch.from_numpy(self.v.copy()).cuda()
        self.gs = torch.from_numpy(self.scales.copy()).cuda()
        self.desc = B.cache_desc(self.gk, self.gv)
        self.gt, self.gctx = torch.from_numpy(self.tables).cuda(), torch.from_numpy(self.ctx).cuda()
        self.gcu = torch.from_numpy(self.cu).cuda()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.max_ctx, self.max_new = int(self.ctx.max()), int(self.new.max())

    def append(self, inv_freq=None, interleaved=False, mscale=1.0, q=None, k=None, v=None, **kw):
        f = torch.from_numpy(np.asarray(inv_freq)).double().cuda() if inv_freq is not None else None
        args = [self.dev16(a) if b is None else b
                for a, b in ((self.q, q), (self.nk, k), (self.nv, v))]
        return B.pkv_rope_append(self.desc, *args, f, self.gcu, self.max_new, self.gt, self.gctx,
                                 self.max_ctx, interleaved=interleaved, mscale=mscale,
                                 scales=self.gs, dev_err=self.err, **kw)

    def positions(self):
        return np.concatenate([np.arange(c - n, c) for n, c in zip(self.new, self.ctx)])

    def oracle_append(self, inv_freq=(), interleaved=False, mscale=1.0):
        """Appends on the host copies; returns (rotated q, rotated K)."""
        pos = self.positions()
        q = OS.rotate(self.q, pos, inv_freq, interleaved, mscale)
        k = OS.rotate(self.nk, pos, inv_freq, interleaved, mscale)
        f = max(np.float32(1), np.float32(1.41421356) * np.float32(abs(mscale))) if len(inv_freq) else 1.0
        OS.append_scaled(self.k, self.scales, 0, k, self.nk, f, self.cu, self.tables, self.ctx)
        OS.append_scaled(self.v, self.scales, 1, self.nv, self.nv, 1.0, self.cu, self.tables, self.ctx)
        return q, k

    def attention(self, scale):
        return OS.attention(self.k, self.v, self.scales, self.q, self.cu, self.tables, self.ctx, scale)

    def decode(self, scale, **kw):
        return B.pkv_paged_attention_decode_scaled(self.desc, self.gs, self.dev16(self.q), self.gt,
                                                   self.gctx, self.max_ctx, scale,
                                                   dev_err=self.err, **kw)


    def prefill(self, scale, **kw):
        return B.pkv_paged_attention_prefill_scaled(self.desc, self.gs, self.dev16(self.q),
                                                    self.gcu, self.max_new, self.gt, self.gctx,
                                                    self.max_ctx, scale, dev_err=self.err, **kw)


def freqs(rot, base=10000.0):
    return base ** (-np.arange(0, rot, 2) / rot)


def check_rotated(got, x, ref, m, dt, what):
    """got (device) against ref, the rotation of x, within the bound above."""
    got = got.double().cpu().numpy()
    e = 2.0 ** -20 * abs(m) * 2 * np.abs(x).max(-1, keepdims=True)
    half = torch.finfo(TD[dt]).eps / 2
    tiny = 2.0 ** -25 if dt == W.F16 else 0.0
    bad = np.abs(got - ref) > half * (np.abs(ref) + e) + e + tiny
    assert not bad.any(), (what, int(bad.sum()), np.abs(got - ref).max())


def canon(codes):
    """Codes with one NaN: a re-rounded NaN stays one, of either sign."""
    codes = codes.cpu().numpy() if isinstance(codes, torch.Tensor) else codes
    return np.where(codes & 0x7f == 0x7f, 0x7f, codes)


CASES = [
    # dtype, heads, kv, D, bs, new, cached, rot, interleaved, mscale
    (W.BF16, 4, 2, 128, 16, [1, 1, 1], [0, 16, 30], 128, False, 1.0),
    (W.F16, 5, 5, 64, 16, [1, 1, 1, 1], [4, 15, 31, 63], 64, True, 1.0),
    (W.BF16, 8, 1, 128, 32, [70, 1, 33, 0, 17], [0, 31, 7, 20, 96], 64, False, 1.3466),
    (W.F16, 3, 3, 128, 8, [7, 8, 9, 1], [1, 0, 23, 7], 96, False, 0.5),
    (W.F16, 6, 2, 64, 8, [40, 3], [5, 8], 16, True, 1.0),
    (W.BF16, 2, 2, 64, 32, [5, 64, 100], [3, 0, 31], 48, False, 1.0),
    (W.BF16, 17, 1, 128, 16, [19, 2], [1000, 2047], 0, False, 1.0),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_rope_append_scaled(i):
    dt, h, kv, d, bs, new, cached, rot, inter, m = CASES[i]
    b = Batch(40 + i, dt, h, kv, d, bs, new, cached, spread=1.5)
    f = freqs(rot) if rot else ()
    q = b.append(f if rot else None, inter, m)
    torch.cuda.synchronize()
    rq, rk = b.oracle_append(f, inter, m)
    if not rot:
        assert np.array_equal(H.to_bits(q), H.to_bits(b.dev16(b.q)))
    check_rotated(q, b.q, rq, m if rot else 1.0, dt, "q")
    gs = b.gs.cpu().numpy()
    assert np.array_equal(gs, b.scales, equal_nan=True)
    assert np.array_equal(canon(b.gv), canon(b.v)), "V codes"
    gk = b.gk.cpu().numpy()
    if not rot:
        assert np.array_equal(canon(gk), canon(b.k)), "K codes"
    else:
        # the new tokens' values; every other byte exactly
        same = np.ones(gk.shape, bool)
        row = 0
        for s, c in enumerate(b.ctx):
            for p in range(c - new[s], c):
                phys, off = b.tables[s, p // bs], p % bs
                same[phys, :, off] = False
                sc = gs[phys, :, 0].astype(np.float64)[:, None]
                got = oracle.decode(oracle.E4M3, gk[phys, :, off]) * sc
                e = 2.0 ** -20 * abs(m) * 2 * np.abs(b.nk[row]).max(-1, keepdims=True)
                bound = np.maximum(2.0 ** -4 * (np.abs(rk[row]) + e), 2.0 ** -10 * sc) + e
                assert (np.abs(got - rk[row]) <= bound).all(), (s, p)
                row += 1
        assert np.array_equal(canon(gk[same]), canon(b.k[same])), "bytes the call does not own"
    assert int(b.err.item()) == 0


@pytest.mark.parametrize("bs", [8, 16, 32])
def test_rope_append_raises_the_scale_of_a_part_filled_block(bs):
    """Each new token is twice the one before: every append after a block's
    first raises the scale and re-rounds the codes before it, exactly as the
    oracle does, and the neighbouring heads and blocks keep theirs."""
    n = 2 * bs + 3
    b = Batch(59, W.F16, 2, 2, 64, bs, [1], [n - 1], fill=False)
    r = np.random.default_rng(59)
    for p in range(n):
        b.ctx = np.array([p + 1], np.int32)
        b.gctx.fill_(p + 1)
        x = r.standard_normal((1, 2, 64)) * 2.0 ** (p % 11 - 5)
        x = torch.from_numpy(x).half().double().numpy()
        before = b.scales.copy()
        b.nk = b.nv = x
        b.append(None)
        b.oracle_append()
        if p % bs and p % 11:
            phys = b.tables[0, p // bs]
            assert (b.scales[phys] >= before[phys]).all()
    assert np.array_equal(b.gs.cpu().numpy(), b.scales, equal_nan=True)
    assert np.array_equal(canon(b.gk), canon(b.k)) and np.array_equal(canon(b.gv), canon(b.v))
    assert int(b.err.item()) == 0


@pytest.mark.parametrize("cache", [W.F16, W.BF16, W.E4M3])
def test_rope_append_other_caches(cache):
    """Caches without block scales: rotated K rounded once to the cache type,
    V as pkv_kv_append writes it; strided inputs of one projection."""
    dt = W.F16 if cache == W.E4M3 else cache
    b = Batch(60, dt, 6, 2, 128, 16, [20, 1, 7], [3, 16, 0])
    f = freqs(64)
    shape = b.k.shape
    if cache == W.E4M3:
        kc, vc = b.gk, b.gv
        desc = B.cache_desc(kc, vc, 0.03125, 0.0625)
    else:
        kc = torch.full(shape, float("nan"), dtype=TD[dt], device="cuda")
        vc = kc.clone()
        desc = B.cache_desc(kc, vc)
    qkv = torch.cat([b.dev16(x) for x in (b.q, b.nk, b.nv)], 1)
    q, k, v = qkv[:, :6], qkv[:, 6:8], qkv[:, 8:]
    out = B.pkv_rope_append(desc, q, k, v, torch.from_numpy(f).cuda(), b.gcu, b.max_new, b.gt,
                            b.gctx, b.max_ctx, dev_err=b.err)
    pos = b.positions()
    check_rotated(out, b.q, OS.rotate(b.q, pos, f), 1.0, dt, "q")
    rk = OS.rotate(b.nk, pos, f)
    seq = np.repeat(np.arange(3), b.new)
    slots = b.tables[seq, pos // 16].astype(np.int64) * 16 + pos % 16
    # V (and where it goes) exactly as the append without a rotation
    k2, v2 = (torch.full_like(t, 0xff if cache == W.E4M3 else float("nan")) for t in (kc, vc))
    d2 = B.cache_desc(k2, v2, desc.k_scale, desc.v_scale)
    B.pkv_kv_append(d2, k.contiguous(), v.contiguous(), torch.from_numpy(slots).cuda())
    if cache == W.E4M3:
        same = (vc.cpu().numpy()[slots // 16, :, slots % 16] ==
                v2.cpu().numpy()[slots // 16, :, slots % 16]).all()
        got = oracle.decode(oracle.E4M3, kc.cpu().numpy()[slots // 16, :, slots % 16]) * 0.03125
        e = 2.0 ** -20 * 2 * np.abs(b.nk).max(-1, keepdims=True)
        sat = np.minimum(np.abs(rk), 448 * 0.03125) * np.sign(rk)
        assert (np.abs(got - sat) <= np.maximum(2.0 ** -4 * (np.abs(rk) + e), 2.0 ** -10 * 0.03125) + e).all()
        assert same
    else:
        assert np.array_equal(H.to_bits(vc), H.to_bits(v2))
        i = torch.from_numpy(slots).cuda()
        check_rotated(kc[i // 16, :, i % 16], b.nk, rk, 1.0, dt, "K")
        # nothing else is written
        assert np.array_equal(H.to_bits(kc.isnan()), H.to_bits(k2.isnan()))
    assert int(b.err.item()) == 0


def test_rope_append_far_positions_and_in_place():
    """Positions past 2^24 (where an fp32 angle is off by radians), q rotated
    in place, rows behind the last sequence untouched."""
    d, bs = 64, 8
    far = [(1 << 24) + 12345, (1 << 27) + 7]
    r = np.random.default_rng(3)
    q = r.standard_normal((4, 2, d)).astype(np.float16).astype(np.float64)
    gq = torch.from_numpy(q).half().cuda()
    # a table row long enough is all the call reads of the far blocks
    nblk = far[1] // bs + 1
    tables = torch.zeros(2, nblk, dtype=torch.int32, device="cuda")
    tables[1, far[1] // bs] = 1
    kc = torch.zeros(2, 2, bs, d, dtype=torch.float16, device="cuda")
    vc = kc.clone()
    ctx = torch.tensor([far[0] + 1, far[1] + 1], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    f = freqs(d)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = B.pkv_rope_append(B.cache_desc(kc, vc), gq, gq.clone(), gq.clone(),
                            torch.from_numpy(f).cuda(), cu, 1, tables, ctx, far[1] + 1,
                            dev_err=err, q_out=gq)
    torch.cuda.synchronize()
    ref = OS.rotate(q[:2], np.array(far), f)
    check_rotated(out[:2], q[:2], ref, 1.0, W.F16, "far")
    assert np.array_equal(out[2:].double().cpu().numpy(), q[2:])
    assert int(err.item()) == 0


def test_rope_append_without_q_and_non_finite_inputs():
    b = Batch(61, W.BF16, 2, 2, 64, 16, [6, 1], [0, 3])
    b.nv[1, 0, 5] = np.inf
    b.nv[2, 1, 7] = -np.inf
    b.nv[3, 0, 9] = np.nan
    b.nv[4] = 0.0
    b.nk[4] = 0.0
    assert b.append(q=None, inv_freq=None) is not None
    b2 = Batch(61, W.BF16, 2, 2, 64, 16, [6, 1], [0, 3])
    out = B.pkv_rope_append(b2.desc, None, b.dev16(b.nk), b.dev16(b.nv), None, b2.gcu, b2.max_new,
                            b2.gt, b2.gctx, b2.max_ctx, scales=b2.gs)
    assert out is None
    b.oracle_append()
    for x in (b, b2):
        assert np.array_equal(x.gs.cpu().numpy(), b.scales, equal_nan=True)
        got = oracle.decode(oracle.E4M3, x.gv.cpu().numpy())
        ref = oracle.decode(oracle.E4M3, b.v)
        assert np.array_equal(got, ref, equal_nan=True)
        assert np.array_equal(canon(x.gk), canon(b.k))
    phys = b.tables[0, 0]
    assert oracle.decode(oracle.E4M3, b.v)[phys, 0, 1, 5] == 448


def test_rope_append_bad_inputs_are_flagged_and_skipped():
    b = Batch(62, W.F16, 2, 2, 64, 16, [5, 6, 7], [0, 30, 9])
    before = (b.gk.clone(), b.gv.clone(), b.gs.clone())
    ctx = b.ctx.copy()
    ctx[0] = 3                                    # fewer tokens than new ones
    b.gctx.copy_(torch.from_numpy(ctx))
    t = b.tables.copy()
    t[1, 2] = b.nb                                # outside the pool
    b.gt.copy_(torch.from_numpy(t))
    q_out = torch.full((18, 2, 64), 7.0, dtype=torch.float16, device="cuda")
    b.append(freqs(64), q_out=q_out)
    torch.cuda.synchronize()
    assert int(b.err.item()) == B.PKV_DEVERR_CONTEXT | B.PKV_DEVERR_BLOCK_ID
    assert (q_out[:5] == 7).all() and not (q_out[5:] == 7).all()
    for a, c in zip(before, (b.gk, b.gv, b.gs)):
        for s, blk in ((0, 0), (1, 2)):
            i = int(b.tables[s, blk])
            assert torch.equal(a[i].view(torch.uint8), c[i].view(torch.uint8))
    rq = OS.rotate(b.q, b.positions(), freqs(64))
    check_rotated(q_out[5:], b.q[5:], rq[5:], 1.0, W.F16, "other sequences")


DECODE = [
    # dtype, heads, kv, D, bs, ctx, partition, size of values, spread of rows (log2)
    (W.F16, 8, 8, 64, 16, [5, 17, 33, 64], 0, 1.0, 0.0),
    (W.BF16, 16, 2, 128, 16, [1, 300, 129, 0, 777], 0, 1.0, 1.0),
    (W.BF16, 16, 2, 128, 16, [1, 300, 129, 0, 777], 64, 1.0, 1.0),
    (W.F16, 3, 1, 128, 32, [1000, 31, 32, 33], 96, 0.01, 2.0),
    (W.F16, 16, 1, 64, 8, [7, 8, 9, 200, 0], 16, 10.0, 1.0),
    (W.BF16, 10, 1, 128, 8, [65, 511], 0, 1.0, 1.0),
    (W.BF16, 5, 5, 64, 32, [2500, 1], 0, 1e-6, 1.0),
    (W.F16, 4, 4, 128, 8, [15, 1023], 48, 1.0, 3.0),
    (W.BF16, 14, 2, 64, 16, [0, 0, 1], 0, 1.0, 0.0),
]


@pytest.mark.parametrize("i", range(len(DECODE)))
def test_decode_scaled(i):
    dt, h, kv, d, bs, ctx, part, size, spread = DECODE[i]
    b = Batch(80 + i, dt, h, kv, d, bs, [1] * len(ctx), ctx, size=size, spread=spread)
    # the contexts as cached (the row's own token is not appended here)
    b.ctx = np.asarray(ctx, np.int32)
    b.gctx.copy_(torch.from_numpy(b.ctx))
    b.max_ctx = max(ctx)
    out = b.decode(1 / np.sqrt(d), partition_size=part)
    again = b.decode(1 / np.sqrt(d), partition_size=part)
    torch.cuda.synchronize()
    ref = b.attention(1 / np.sqrt(d))
    # the bound is absolute and relative to values of size one
    H.assert_attention_close(H.out_to_double(out) / size, ref / size, "decode scaled %d" % i, dt)
    assert torch.equal(out, again)
    assert int(b.err.item()) == 0


@pytest.mark.parametrize("heads,kv,d,bs,n,hi", [(6, 2, 64, 8, 40, 1500), (16, 1, 128, 16, 3, 4000),
                                                (4, 4, 128, 32, 9, 2000), (8, 1, 64, 16, 1, 5000)])
def test_decode_scaled_equal_shares(heads, kv, d, bs, n, hi):
    """Ragged batches whose items are cut at every kind of place: empty
    contexts, unusable ones (zeros, flagged), whole items, long ones; a
    workspace full of NaN."""
    r = np.random.default_rng(100 + n)
    ctx = r.integers(0, hi, n).astype(np.int32)
    ctx[-1] = hi
    if n > 5:
        ctx[2] = 0
    b = Batch(97, W.BF16, heads, kv, d, bs, [1] * n, ctx, spread=1.0)
    b.ctx = ctx
    b.max_ctx = hi
    seen = ctx.copy()
    if n > 5:
        seen[4], seen[5] = -1, hi + 1              # flagged
        ctx[4] = ctx[5] = 0
    b.gctx.copy_(torch.from_numpy(seen))
    assert B.pkv_decode_scaled_partition_size(b.desc, n, heads, hi) == 0
    ws = torch.full((B.pkv_decode_scaled_workspace_bytes(b.desc, n, heads, hi),), 0xff,
                    dtype=torch.uint8, device="cuda")
    out = b.decode(0.11, workspace=ws)
    again = b.decode(0.11)
    torch.cuda.synchronize()
    assert int(b.err.item()) == (B.PKV_DEVERR_CONTEXT if n > 5 else 0)
    H.assert_attention_close(H.out_to_double(out), b.attention(0.11), "equal shares %d" % n, W.BF16)
    assert torch.equal(out, again)


def test_scaled_calls_in_graphs_and_on_another_stream():
    """An append, decode and prefill captured once and replayed after the inputs
    changed in place, while other calls use the same workspace on the capture's
    stream in between."""
    b = Batch(98, W.BF16, 8, 2, 64, 16, [1, 1, 1], [700, 30, 1200])
    f = torch.from_numpy(freqs(64)).cuda()
    ws = torch.empty(B.pkv_decode_scaled_workspace_bytes(b.desc, 3, 8, b.max_ctx), dtype=torch.uint8,
                     device="cuda")
    q, k, v = (b.dev16(x) for x in (b.q, b.nk, b.nv))
    qr, out, pre = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)

    def step():
        B.pkv_rope_append(b.desc, q, k, v, f, b.gcu, 1, b.gt, b.gctx, b.max_ctx, scales=b.gs,
                          q_out=qr, dev_err=b.err)
        B.pkv_paged_attention_decode_scaled(b.desc, b.gs, qr, b.gt, b.gctx, b.max_ctx, 0.125,
                                            workspace=ws, out=out, dev_err=b.err)
        B.pkv_paged_attention_prefill_scaled(b.desc, b.gs, qr, b.gcu, 1, b.gt, b.gctx, b.max_ctx,
                                             0.125, out=pre, dev_err=b.err)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            step()
    torch.cuda.synchronize()
    for i in range(3):
        x = b.values(3, 8, 1.0, 0.0)
        b.q = x
        q.copy_(b.dev16(x))
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            g.replay()
            first = out.clone()
            step()
            second = out.clone()
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, second) and torch.equal(first, out)
        if i == 0:
            b.oracle_append(freqs(64))
        # the attention of the kernel's own rotated q and K, which have tests of
        # their own
        b.q = qr.double().cpu().numpy()
        b.k, b.scales = b.gk.cpu().numpy(), b.gs.cpu().numpy()
        ref = b.attention(0.125)
        H.assert_attention_close(H.out_to_double(out), ref, "graph decode", W.BF16)
        H.assert_attention_close(H.out_to_double(pre), ref, "graph prefill", W.BF16)
    assert int(b.err.item()) == 0


def test_decode_scaled_large_ratio_of_scales():
    """V of one block 2^12 larger than the others but with no weight (its keys
    point away): the small blocks keep their precision."""
    b = Batch(95, W.F16, 4, 1, 128, 16, [1], [160])
    b.ctx = np.array([160], np.int32)
    b.q[...] = np.abs(b.q)
    big = b.tables[0, 4]
    x = np.full((16, 1, 128), -8.0)
    OS.append_scaled(b.k, b.scales, 0, x, x, 1.0, [0, 16], np.array([[big]]), [16])
    x = b.values(16, 1, 4096.0, 0.0)
    OS.append_scaled(b.v, b.scales, 1, x, x, 1.0, [0, 16], np.array([[big]]), [16])
    b.upload()
    out = b.decode(1.0)
    ref = b.attention(1.0)
    H.assert_attention_close(H.out_to_double(out), ref, "decode scaled ratio", W.F16)
    assert np.abs(ref).max() < 8


def test_decode_scaled_range_checks():
    b = Batch(96, W.F16, 4, 2, 64, 16, [1, 1, 1], [40, 50, 60])
    b.ctx = np.array([40, 50, 60], np.int32)
    ref = b.attention(0.125)
    t = b.tables.copy()
    t[0, 1] = -7
    b.gt.copy_(torch.from_numpy(t))
    b.gctx.copy_(torch.tensor([40, 9999, 60], dtype=torch.int32))
    out = b.decode(0.125, partition_size=32)
    torch.cuda.synchronize()
    assert int(b.err.item()) == B.PKV_DEVERR_BLOCK_ID | B.PKV_DEVERR_CONTEXT
    assert (out[1] == 0).all() and not out.isnan().any()
    H.assert_attention_close(H.out_to_double(out)[2:], ref[2:], "decode scaled good", W.F16)


PREFILL = [
    # dtype, heads, kv, D, bs, new, cached, size, spread of rows (log2)
    (W.BF16, 4, 4, 128, 16, [70, 1, 129, 64], [0, 0, 0, 0], 1.0, 1.0),
    (W.F16, 4, 4, 128, 16, [300, 1, 257], [0, 0, 0], 1.0, 0.0),
    (W.BF16, 8, 2, 64, 32, [33, 100, 7], [40, 0, 200], 10.0, 2.0),
    (W.F16, 16, 2, 128, 8, [17, 65, 3, 0], [5, 130, 64, 9], 0.01, 1.0),
    (W.BF16, 16, 1, 64, 16, [9, 20], [100, 0], 1e-6, 1.0),
    (W.F16, 128, 1, 64, 16, [3, 2], [31, 0], 1.0, 1.0),
    (W.BF16, 6, 2, 128, 16, [50, 23], [10, 77], 1.0, 3.0),
    (W.F16, 2, 2, 64, 8, [600], [519], 1.0, 1.0),
    (W.BF16, 7, 1, 128, 32, [1, 1, 130], [1000, 0, 31], 1.0, 1.0),
]


@pytest.mark.parametrize("i", range(len(PREFILL)))
def test_prefill_scaled(i):
    dt, h, kv, d, bs, new, cached, size, spread = PREFILL[i]
    b = Batch(120 + i, dt, h, kv, d, bs, new, cached, size=size, spread=spread)
    b.oracle_append()
    b.upload()
    out = b.prefill(1 / np.sqrt(d))
    again = b.prefill(1 / np.sqrt(d))
    torch.cuda.synchronize()
    assert int(b.err.item()) == 0
    ref = b.attention(1 / np.sqrt(d))
    H.assert_attention_close(H.out_to_double(out) / size, ref / size, "prefill scaled %d" % i, dt)
    assert torch.equal(out, again)


@pytest.mark.parametrize("scale", [-0.3, 0.0])
def test_attention_scaled_other_signs_of_the_scale(scale):
    b = Batch(140, W.F16, 4, 2, 64, 16, [40, 1], [7, 30])
    b.oracle_append()
    b.upload()
    H.assert_attention_close(H.out_to_double(b.prefill(scale)), b.attention(scale),
                             "prefill scaled sign", W.F16)
    b = Batch(141, W.F16, 4, 2, 64, 16, [1, 1], [70, 30])
    b.oracle_append()
    b.upload()
    H.assert_attention_close(H.out_to_double(b.decode(scale)), b.attention(scale),
                             "decode scaled sign", W.F16)


@pytest.mark.parametrize("zero", ["k", "v", "both"])
def test_attention_scaled_over_zeros(zero):
    """Contexts whose K, V or both are all zeros (the smallest scale there is):
    the mean of V, or zeros."""
    for new in ([70, 1], [1, 1]):
        b = Batch(145, W.BF16, 4, 2, 64, 16, new, [40, 600])
        for name in (("k",) if zero == "k" else ("v",) if zero == "v" else ("k", "v")):
            getattr(b, name)[...] = 0
            b.scales[..., "kv".index(name)] = 2.0 ** -126
            getattr(b, "n" + name)[...] = 0
        b.oracle_append()
        b.upload()
        out = b.prefill(0.125) if max(new) > 1 else b.decode(0.125)
        H.assert_attention_close(H.out_to_double(out), b.attention(0.125), "zeros", W.BF16)


@pytest.mark.parametrize("n", [1, 127, 128, 129, 1000, 1024, 1025])
def test_decode_scaled_many_sequences(n):
    """Batches around the number of sequences that equal shares scan (1,024)."""
    r = np.random.default_rng(n)
    ctx = r.integers(0, 40, n).astype(np.int32)
    ctx[0] = 2000                                  # long enough for equal shares
    b = Batch(146, W.F16, 2, 1, 64, 16, [1] * n, ctx)
    b.ctx, b.max_ctx = ctx, 2000
    b.gctx.copy_(torch.from_numpy(ctx))
    assert (B.pkv_decode_scaled_partition_size(b.desc, n, 2, 2000) == 0) == (n <= 1024)
    out = b.decode(0.125)
    H.assert_attention_close(H.out_to_double(out), b.attention(0.125), "many sequences", W.F16)
    assert int(b.err.item()) == 0


def test_prefill_scaled_nan_of_a_later_token_stays_there():
    """A NaN in K or V of a token reaches the rows that see the token (V: in its
    own column) and no other."""
    b = Batch(142, W.BF16, 4, 2, 64, 16, [150, 20], [3, 0])
    b.nv[100, 1, 17] = np.nan
    b.nk[120, 0, 5] = np.nan
    b.oracle_append()
    b.upload()
    got = H.out_to_double(b.prefill(0.125))
    ref = b.attention(0.125)
    nan = np.isnan(ref)
    assert nan.any() and not nan[:100].any() and not nan[150:].any()
    assert np.array_equal(np.isnan(got), nan)
    H.assert_attention_close(np.where(nan, 0, got), np.where(nan, 0, ref), "prefill nan", W.BF16)


def test_prefill_scaled_range_checks():
    b = Batch(143, W.F16, 4, 2, 64, 16, [40, 50, 300], [0, 10, 5])
    b.oracle_append()
    b.upload()
    ref = b.attention(0.125)
    t = b.tables.copy()
    t[2, 10] = b.nb + 3                            # keys 160..175 of sequence 2
    b.gt.copy_(torch.from_numpy(t))
    c = b.ctx.copy()
    c[0] = 39                                      # fewer tokens than new ones
    b.gctx.copy_(torch.from_numpy(c))
    out = b.prefill(0.125)
    torch.cuda.synchronize()
    assert int(b.err.item()) == B.PKV_DEVERR_BLOCK_ID | B.PKV_DEVERR_CONTEXT
    assert (out[:40] == 0).all() and not out.isnan().any()
    keep = np.r_[np.arange(40, 90), np.arange(90, 90 + 155)]
    H.assert_attention_close(H.out_to_double(out)[keep], ref[keep], "prefill scaled good", W.F16)


def test_prefill_scaled_padded_batch():
    """Rows behind the last sequence, an empty sequence and a bound above every
    length: rows that belong to nobody stay as they were."""
    b = Batch(144, W.F16, 4, 2, 64, 16, [40, 0, 50], [0, 0, 10])
    b.oracle_append()
    b.upload()
    q = torch.cat([b.dev16(b.q), torch.ones(7, 4, 64, dtype=torch.float16, device="cuda")])
    out = torch.full_like(q, 3.0)
    B.pkv_paged_attention_prefill_scaled(b.desc, b.gs, q, b.gcu, 1000, b.gt, b.gctx, b.max_ctx,
                                         0.125, dev_err=b.err, out=out)
    assert (out[90:] == 3).all() and int(b.err.item()) == 0
    H.assert_attention_close(H.out_to_double(out[:90]), b.attention(0.125), "prefill padded", W.F16)


def test_copy_blocks_scaled():
    """Copy-on-write in two layers and a swap through pinned host memory, byte
    for byte, scales included; a bad pair is flagged and skipped."""
    r = np.random.default_rng(4)
    shape = (20, 3, 8, 64)
    ks = [torch.from_numpy(r.integers(0, 256, shape).astype(np.uint8)).cuda() for _ in range(2)]
    vs = [torch.from_numpy(r.integers(0, 256, shape).astype(np.uint8)).cuda() for _ in range(2)]
    ss = [torch.from_numpy(r.standard_normal((20, 3, 2)).astype(np.float32)).cuda() for _ in range(2)]
    ref = [[t.clone() for t in x] for x in (ks, vs, ss)]
    pairs = [(1, 17), (1, 18), (5, 19), (20, 3), (4, -1)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    descs = [B.cache_desc(k, v) for k, v in zip(ks, vs)]
    B.pkv_copy_blocks_scaled(descs, ss, torch.tensor(pairs, device="cuda"), dev_err=err)
    for x in ref:
        for t in x:
            for a, c in pairs[:3]:
                t[c] = t[a].clone()
    for x, y in zip((ks, vs, ss), ref):
        assert all(torch.equal(a, c) for a, c in zip(x, y))
    assert int(err.item()) == B.PKV_DEVERR_COPY_PAIR
    # out to the host and back to other blocks
    hk = torch.zeros((6,) + shape[1:], dtype=torch.uint8).pin_memory()
    hv, hs = hk.clone().pin_memory(), torch.zeros(6, 3, 2).pin_memory()
    out = torch.tensor([(7, 2), (8, 0)], device="cuda")
    B.pkv_copy_blocks_scaled(descs[0], ss[0], out, B.cache_desc(hk, hv), hs)
    torch.cuda.synchronize()
    assert torch.equal(hk[2], ks[0][7].cpu()) and torch.equal(hs[0], ss[0][8].cpu())
    back = torch.tensor([(2, 9), (0, 10)], device="cuda")
    B.pkv_copy_blocks_scaled(B.cache_desc(hk, hv), hs, back, descs[0], ss[0])
    for x in (ks[0], vs[0], ss[0]):
        assert torch.equal(x[9], x[7]) and torch.equal(x[10], x[8])


def test_scaled_path_end_to_end():
    """As an engine runs it: prompts appended and prefilled, every prompt forked
    into three samples, copy-on-write with scales, twenty decode steps of append
    and decode; each call against the oracle on the cache as it then is, and the
    cache against the values that went in."""
    from paged_kv_cache_130_gb300.block_manager import BlockManager, BlockPool
    h, kv, d, bs, f = 8, 2, 64, 16, freqs(64)
    r = np.random.default_rng(7)
    mgr = BlockManager(BlockPool(200, bs, r.permutation(200)))
    k8 = torch.full((200, kv, bs, d), 0xff, dtype=torch.uint8, device="cuda")
    v8, sc = k8.clone(), torch.full((200, kv, 2), float("nan"), device="cuda")
    desc = B.cache_desc(k8, v8)
    gf = torch.from_numpy(f).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept = {}                                      # sequence -> its (K rotated, V) rows so far

    def call(seqs, new):
        """Append `new` tokens to each sequence and attend; returns nothing."""
        n = sum(new)
        x = [torch.from_numpy(r.standard_normal((n, m, d))).bfloat16().cuda() for m in (h, kv, kv)]
        ctx = np.array([s.num_tokens for s in seqs], np.int32)
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        bt = BlockManager.block_table_array(seqs)
        g = [torch.from_numpy(a).cuda() for a in (cu, bt, ctx)]
        q = B.pkv_rope_append(desc, *x, gf, g[0], max(new), g[1], g[2], int(ctx.max()), scales=sc,
                              dev_err=err)
        if max(new) > 1:
            out = B.pkv_paged_attention_prefill_scaled(desc, sc, q, g[0], max(new), g[1], g[2],
                                                       int(ctx.max()), 0.125, dev_err=err)
        else:
            out = B.pkv_paged_attention_decode_scaled(desc, sc, q, g[1], g[2], int(ctx.max()), 0.125,
                                                      dev_err=err)
        kc, vc, s_ = k8.cpu().numpy(), v8.cpu().numpy(), sc.cpu().numpy()
        ref = OS.attention(kc, vc, s_, q.double().cpu().numpy(), cu, bt, ctx, 0.125)
        H.assert_attention_close(H.out_to_double(out), ref, "path", W.BF16)
        pos = np.concatenate([np.arange(c - m, c) for c, m in zip(ctx, new)])
        rk = OS.rotate(x[1].double().cpu().numpy(), pos, f)
        for i, s in enumerate(seqs):
            rows = slice(cu[i], cu[i + 1])
            old = kept.get(id(s), (np.zeros((0, kv, d)),) * 2)
            kept[id(s)] = tuple(np.concatenate([a, b[rows]]) for a, b in
                                zip(old, (rk, x[2].double().cpu().numpy())))
            for which, codes in ((0, kc), (1, vc)):
                for hd in range(kv):
                    got = OS.gather(codes, s_, which, bt[i], int(ctx[i]), hd)
                    want = kept[id(s)][which][:, hd]
                    # E4M3 of the value, and a second rounding where a later token
                    # raised the block's scale: half a step of the value, and half
                    # a subnormal step of each scale that its block has had
                    top = s_[bt[i, :-(-int(ctx[i]) // bs)], hd, which].repeat(bs)[:int(ctx[i]), None]
                    bound = 2.0 ** -4 * 1.0625 * np.abs(want) + 2.0 ** -9 * top + 1e-5
                    assert (np.abs(got - want) <= bound).all()

    prompts = [mgr.new_sequence() for _ in range(3)]
    lens = [37, 130, 16]
    for s, n in zip(prompts, lens):
        mgr.append_tokens(s, n)
    call(prompts, lens)
    seqs = []
    for s in prompts:
        for t in [s] + [mgr.fork(s) for _ in range(2)]:
            kept[id(t)] = kept[id(s)]
            seqs.append(t)
    for step in range(20):
        pairs = [p for _, p in (mgr.append_slot(s) for s in seqs) if p is not None]
        if pairs:
            assert step == 0
            B.pkv_copy_blocks_scaled(desc, sc, torch.tensor(pairs, device="cuda"), dev_err=err)
        call(seqs, [1] * len(seqs))
    assert int(err.item()) == 0


def test_scaled_calls_beyond_four_gigabytes():
    """Blocks whose byte offsets pass 32 bits: the same bits as the same blocks
    at the front of a pool."""
    b = Batch(150, W.BF16, 8, 2, 128, 32, [70, 1, 40], [100, 1200, 0])
    f = torch.from_numpy(freqs(128)).cuda()
    n = (1 << 32) // (2 * 32 * 128) + 1000          # K codes alone past 2^32 bytes
    far = [torch.empty(n, 2, 32, 128, dtype=torch.uint8, device="cuda") for _ in range(2)]
    fs = torch.empty(n, 2, 2, device="cuda")
    at = n - b.nb
    for t, src in zip(far + [fs], (b.gk, b.gv, b.gs)):
        t[at:] = src
    desc, tables = B.cache_desc(*far), torch.where(b.gt >= 0, b.gt + at, b.gt)
    args = [b.dev16(x) for x in (b.q, b.nk, b.nv)]
    outs = []
    for d, s, t in ((b.desc, b.gs, b.gt), (desc, fs, tables)):
        q = B.pkv_rope_append(d, *args, f, b.gcu, b.max_new, t, b.gctx, b.max_ctx, scales=s,
                              dev_err=b.err)
        pre = B.pkv_paged_attention_prefill_scaled(d, s, q, b.gcu, b.max_new, t, b.gctx, b.max_ctx,
                                                   0.1, dev_err=b.err)
        dec = B.pkv_paged_attention_decode_scaled(d, s, q[b.gcu[1:].long() - 1].contiguous(), t,
                                                  b.gctx, b.max_ctx, 0.1, dev_err=b.err)
        outs.append((q, pre, dec))
    B.pkv_copy_blocks_scaled(desc, fs, torch.tensor([[at + 1, 0], [at + 2, at + 3]], device="cuda"),
                             dev_err=b.err)
    torch.cuda.synchronize()
    assert int(b.err.item()) == 0
    for x, y in zip(*outs):
        assert torch.equal(x, y) and not x.isnan().any()
    for t in far + [fs]:
        for src, dst in ((at + 1, 0), (at + 2, at + 3)):
            assert torch.equal(t[dst].view(torch.uint8), t[src].view(torch.uint8))
    keep = [i for i in range(b.nb) if i != 3]
    assert torch.equal(far[0][at:][keep], b.gk[keep]) and torch.equal(far[1][at:][keep], b.gv[keep])


def test_scaled_calls_with_nothing_to_do():
    b = Batch(151, W.F16, 4, 2, 64, 16, [1], [20])
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    rows = [torch.empty(0, h, 64, dtype=torch.float16, device="cuda") for h in (4, 2, 2)]
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    empty_table = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    q = B.pkv_rope_append(b.desc, *rows, None, zero, 0, empty_table, none, 0, scales=b.gs)
    assert q.shape == (0, 4, 64)
    out = B.pkv_paged_attention_decode_scaled(b.desc, b.gs, rows[0], empty_table, none, 0, 0.1)
    assert out.shape == (0, 4, 64)
    out = B.pkv_paged_attention_prefill_scaled(b.desc, b.gs, rows[0], zero, 0, empty_table, none, 0, 0.1)
    assert out.shape == (0, 4, 64)
    B.pkv_copy_blocks_scaled(b.desc, b.gs, torch.empty(0, 2, dtype=torch.int64, device="cuda"))
    # sequences without new tokens, and contexts of length 0
    b = Batch(152, W.F16, 4, 2, 64, 16, [0, 3, 0], [5, 0, 0])
    before = b.gk.clone()
    b.append()
    out = b.prefill(0.1)
    b.oracle_append()
    H.assert_attention_close(H.out_to_double(out), b.attention(0.1), "one of three", W.F16)
    same = torch.ones(b.nb, dtype=torch.bool)
    same[int(b.tables[1, 0])] = False
    assert torch.equal(before[same], b.gk[same])
    assert int(b.err.item()) == 0


def test_scaled_calls_with_a_bound_below_a_length():
    """max_q_len smaller than a sequence's tokens: that sequence is flagged, its
    rows are zero (prefill) or untouched (append), the others are right."""
    b = Batch(153, W.F16, 4, 2, 64, 16, [300, 20], [0, 40])
    before = (b.gk.clone(), b.gs.clone())
    q_out = torch.full((320, 4, 64), 5.0, dtype=torch.float16, device="cuda")
    b.max_new = 25
    b.append(freqs(64), q_out=q_out)
    assert int(b.err.item()) == B.PKV_DEVERR_CONTEXT and (q_out[:300] == 5).all()
    own = torch.from_numpy(b.tables[0][b.tables[0] >= 0]).long().cuda()
    assert torch.equal(before[0][own], b.gk[own])
    check_rotated(q_out[300:], b.q[300:], OS.rotate(b.q, b.positions(), freqs(64))[300:], 1.0, W.F16, "q")
    b.err.zero_()
    out = b.prefill(0.1)
    assert int(b.err.item()) == B.PKV_DEVERR_CONTEXT and (out[:300] == 0).all()
    b.k, b.v, b.scales = (t.cpu().numpy() for t in (b.gk, b.gv, b.gs))
    b.scales = np.where(np.isnan(b.scales), 1, b.scales)
    ref = b.attention(0.1)
    H.assert_attention_close(H.out_to_double(out)[300:], ref[300:], "bound", W.F16)


def test_scaled_calls_on_an_explicit_stream():
    """Calls that allocate their outputs and workspace, issued on a stream that is
    not the current one, as an object and as a number, two at once."""
    b = Batch(154, W.BF16, 8, 2, 64, 16, [1, 1, 1], [1500, 30, 1200])
    b.oracle_append(freqs(64))
    ref_q = OS.rotate(b.q, b.positions(), freqs(64))
    f = torch.from_numpy(freqs(64)).cuda()
    q, k, v = (b.dev16(x) for x in (b.q, b.nk, b.nv))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    caches = [(b.gk.clone(), b.gv.clone(), b.gs.clone()) for _ in streams]
    got = []
    for st, handle, (kc, vc, sc) in zip(streams, (streams[0], streams[1].cuda_stream), caches):
        st.wait_stream(torch.cuda.current_stream())
        d = B.cache_desc(kc, vc)
        qr = B.pkv_rope_append(d, q, k, v, f, b.gcu, 1, b.gt, b.gctx, b.max_ctx, scales=sc,
                               dev_err=b.err, stream=handle)
        out = B.pkv_paged_attention_decode_scaled(d, sc, qr, b.gt, b.gctx, b.max_ctx, 0.125,
                                                  dev_err=b.err, stream=handle)
        pre = B.pkv_paged_attention_prefill_scaled(d, sc, qr, b.gcu, 1, b.gt, b.gctx, b.max_ctx,
                                                   0.125, dev_err=b.err, stream=handle)
        got.append((qr, out, pre))
    torch.cuda.synchronize()
    assert int(b.err.item()) == 0
    for x, y in zip(*got):
        assert torch.equal(x, y)
    check_rotated(got[0][0], b.q, ref_q, 1.0, W.BF16, "q")
    b.k, b.v, b.scales = (t.cpu().numpy() for t in caches[0])
    b.q = got[0][0].double().cpu().numpy()
    for out in got[0][1:]:
        H.assert_attention_close(H.out_to_double(out), b.attention(0.125), "stream", W.BF16)


def test_scaled_calls_refuse_host_tensors():
    """Every tensor has to be on the GPU: a host address would be read there."""
    b = Batch(155, W.F16, 4, 2, 64, 16, [1, 1], [20, 5])
    f = torch.from_numpy(freqs(64)).cuda()
    good = dict(q=b.dev16(b.q), k=b.dev16(b.nk), v=b.dev16(b.nv), inv_freq=f, cu_seqlens_q=b.gcu,
                block_tables=b.gt, context_lens=b.gctx, scales=b.gs,
                q_out=torch.empty(2, 4, 64, dtype=torch.float16, device="cuda"))
    for name in good:
        with pytest.raises(ValueError):
            B.pkv_rope_append(b.desc, max_q_len=1, max_context_len=21, **dict(good, **{name: good[name].cpu()}))
    args = dict(scales=b.gs, q=good["q"], block_tables=b.gt, context_lens=b.gctx, out=good["q_out"])
    for name in args:
        with pytest.raises(ValueError):
            B.pkv_paged_attention_decode_scaled(b.desc, max_context_len=21, scale=0.1,
                                                **dict(args, **{name: args[name].cpu()}))
    args["cu_seqlens_q"] = b.gcu
    for name in args:
        with pytest.raises(ValueError):
            B.pkv_paged_attention_prefill_scaled(b.desc, max_q_len=1, max_context_len=21, scale=0.1,
                                                 **dict(args, **{name: args[name].cpu()}))
    pairs = torch.tensor([[0, 1]])
    for p, s in ((pairs, b.gs), (pairs.cuda(), b.gs.cpu())):
        with pytest.raises(ValueError):
            B.pkv_copy_blocks_scaled(b.desc, s, p)
