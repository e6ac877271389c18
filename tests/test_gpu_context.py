"""Shared-prefix decode over the scaled cache, attention weights, the decode that
adds its weights, and eviction against the 64-bit oracle.

Bounds, from the arithmetic:
* attention: 2e-3 + 2e-3 |ref|, plus half a bf16 step (harness), as for the scaled
  decode.
* weights: a score is a sum of exact products in fp32, in at most 8 steps of the
  tensor core that may truncate (2^-23 of the sum of magnitudes A each, so 2^-20 A),
  times factors (2^-22 of it), less a maximum (2^-23 of it): it is off by e = 2^-19
  (A + 1) and a weight by a factor within exp(+-e) on top of the exponential (2^-21),
  in the row's sum alike, whose fp32 addition adds 2^-20; in all 3 e + 2^-19 of the
  weight.  Adding rows and the total before: 2^-20 of the result.
* eviction: exact.
Unwritten slots hold 0xFF (NaN codes) and unused scales NaN, so that a read of
either shows.
"""
import numpy as np
import pytest
import torch

import harness as H
import oracle
from oracle import context as OC
from oracle import scaled as OS
from paged_kv_cache_130_gb300 import binding as B
from paged_kv_cache_130_gb300 import workloads as W
from test_gpu_scaled import TD, Batch, freqs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    H.build_library()


class Keys:
    """K of a Batch in 64 bits, by sequence and KV head."""

    def __init__(self, b, k=None, one_scale=None):
        self.b, self.heads, self.k, self.one_scale = b, b.kv, k, one_scale

    def __call__(self, s, h):
        b, c = self.b, int(self.b.ctx[s])
        if self.k is None and self.one_scale is None:
            return OS.gather(b.k, b.scales, 0, b.tables[s], c, h)
        ids = np.asarray(b.tables[s, :-(-c // b.bs)], np.int64)
        x = oracle.decode(oracle.E4M3, np.ascontiguousarray(b.k[ids, h])) * self.one_scale \
            if self.k is None else self.k[ids, h]
        return x.reshape(-1, b.d)[:c]


def weights_close(got, before, add, size, what=""):
    """got = before + add, within the bound above."""
    got = got.double().cpu().numpy()[..., :add.shape[2]]
    e = 2.0 ** -19 * (size + 1)
    ref = before + add
    bound = (3 * e + 2.0 ** -19) * add + 2.0 ** -20 * np.abs(ref) + 1e-30
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.abs(got - ref).max(), (np.abs(got - ref) / bound).max())


def filled(seed, dt, heads, kv, d, bs, ctx, **kw):
    """A Batch whose contexts are all in the cache, one row of q a sequence."""
    b = Batch(seed, dt, heads, kv, d, bs, [1] * len(ctx), np.asarray(ctx) - 1, **kw)
    b.append()
    b.oracle_append()
    return b


# ------------------------------------------------------------------ shared prefixes

class Shared(Batch):
    """Groups of sequences whose tables begin with the same blocks."""

    def __init__(self, seed, dt, heads, kv, d, bs, groups, spread=1.0):
        """groups: [(prefix blocks, [own tokens of each member])]"""
        own = [n for _, m in groups for n in m]
        pre = [p for p, m in groups for _ in m]
        ctx = [n + p * bs for n, p in zip(own, pre)]
        super().__init__(seed, dt, heads, kv, d, bs, [1 if c else 0 for c in ctx],
                         [max(c - 1, 0) for c in ctx], spread=spread)
        self.append()
        self.oracle_append()
        # members read their first one's prefix
        at = 0
        for p, m in groups:
            for i in range(at, at + len(m)):
                self.tables[i, :p] = self.tables[at, :p]
            at += len(m)
        # (blocks that nobody points to any more are poisoned)
        used = np.unique(np.concatenate([self.tables[s, :-(-c // bs)] for s, c in enumerate(ctx)]))
        free = np.setdiff1d(np.arange(self.nb), used)
        self.k[free], self.v[free], self.scales[free] = 0xff, 0xff, np.nan
        self.gk[torch.from_numpy(free)], self.gv[torch.from_numpy(free)] = 0xff, 0xff
        self.gs[torch.from_numpy(free)] = float("nan")
        self.gt.copy_(torch.from_numpy(self.tables))
        self.begin = np.concatenate([[0], np.cumsum([len(m) for _, m in groups])]).astype(np.int32)
        self.prefix = np.array([p for p, _ in groups], np.int32)
        self.q = self.values(len(ctx), heads, 1.0, 0.0)
        self.cu = np.arange(len(ctx) + 1).astype(np.int32)

    def shared(self, scale, **kw):
        a = dict(group_begin=torch.from_numpy(self.begin).cuda(),
                 group_prefix_blocks=torch.from_numpy(self.prefix).cuda(),
                 max_group_size=int(np.diff(self.begin).max()),
                 max_prefix_blocks=int(self.prefix.max()), dev_err=self.err)
        a.update(kw)
        return B.pkv_paged_attention_decode_scaled_shared_prefix(
            self.desc, self.gs, self.dev16(self.q), self.gt, self.gctx, self.max_ctx, scale=scale, **a)


SHARED = [
    # dtype, heads, kv, D, bs, groups
    (W.F16, 4, 4, 64, 16, [(2, [1, 70, 5]), (3, [16, 1])]),
    (W.BF16, 8, 1, 128, 16, [(5, [3, 40, 1, 17, 64, 65])]),                 # 48 rows: tiles of 16
    (W.BF16, 6, 2, 128, 8, [(9, [1, 2, 3, 4, 5]), (0, [33, 7]), (1, [100])]),
    (W.F16, 2, 2, 128, 32, [(4, [0, 0, 5]), (2, [0])]),                     # contexts that are the prefix
    (W.BF16, 16, 1, 64, 16, [(3, [20, 1]), (0, [0]), (2, [9])]),
    (W.F16, 3, 1, 128, 16, [(40, [10] * 11), (1, [700, 3])]),
    (W.BF16, 5, 5, 128, 16, [(1, [1] * 9)] * 7),
    (W.F16, 14, 2, 64, 8, [(130, [5, 300, 1]), (64, [64] * 4)]),
    # more rows than 32: prefixes by a kernel of their own, in runs of keys
    (W.F16, 8, 2, 64, 16, [(150, [3] * 20), (0, [5]), (70, [1, 200] + [2] * 15)]),
    (W.BF16, 16, 1, 128, 32, [(40, [7, 0, 0, 33, 1]), (1, [1] * 3)]),
    (W.BF16, 8, 1, 128, 8, [(200, [4] * 40), (17, [9] * 33)]),              # two CTAs' rows
    (W.F16, 3, 1, 128, 16, [(65, [2] * 90)]),
    # more than 16, of many groups and heads
    (W.F16, 16, 16, 64, 16, [(5, [3] * 17), (0, [9])] + [(2, [1, 20])] * 6),
    (W.BF16, 64, 32, 128, 8, [(70, [2, 0, 33] * 5), (9, [1]), (3, [5, 1]), (1, [8] * 8)]),
]


@pytest.mark.parametrize("i", range(len(SHARED)))
def test_shared_prefix(i):
    dt, h, kv, d, bs, groups = SHARED[i]
    b = Shared(700 + i, dt, h, kv, d, bs, groups)
    out = b.shared(d ** -0.5)
    again = b.shared(d ** -0.5)
    torch.cuda.synchronize()
    assert int(b.err.item()) == 0
    H.assert_attention_close(out.double().cpu().numpy(), b.attention(d ** -0.5), "shared prefix", dt)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


def test_shared_prefix_long_for_its_members():
    """A prefix that many CTAs share, members that each hold a share's worth."""
    b = Shared(720, W.BF16, 8, 2, 128, 16, [(300, [700, 1, 1500, 64]), (0, [2000])])
    out = b.shared(0.09)
    torch.cuda.synchronize()
    assert int(b.err.item()) == 0
    H.assert_attention_close(out.double().cpu().numpy(), b.attention(0.09), "shared prefix", W.BF16)


def test_shared_prefix_without_prefixes_is_the_decode():
    b = Shared(721, W.F16, 4, 2, 64, 16, [(0, [100, 3]), (0, [2000])])
    ref = b.decode(0.125)
    assert torch.equal(b.shared(0.125, max_prefix_blocks=0), ref)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert torch.equal(b.shared(0.125, group_begin=torch.zeros(1, dtype=torch.int32, device="cuda"),
                                group_prefix_blocks=none, max_prefix_blocks=4), ref)
    H.assert_attention_close(b.shared(0.125, max_prefix_blocks=4).double().cpu().numpy(),
                             b.attention(0.125), "no prefix", W.F16)
    assert int(b.err.item()) == 0


@pytest.mark.parametrize("heads,kv,d,members", [(2, 2, 64, 3), (4, 1, 128, 2), (3, 1, 128, 20)])
def test_shared_prefix_nan_reaches_who_sees_it(heads, kv, d, members):
    """A NaN among a member's own values makes that member's output NaN in its column,
    one of the prefix everybody's, and no other."""
    b = Shared(735, W.F16, heads, kv, d, 16, [(4, [70] * members), (0, [50])])
    ref = b.attention(0.125)
    own, common = int(b.tables[1, 5]), int(b.tables[0, 2])
    b.k[common, 0, 3, 7] = 0x40                      # (an ordinary key beside it)
    for pool in (b.v, b.gv):
        pool[own, 0, 9, 11] = 0x7f
        pool[common, 0, 3, 40] = 0xff
    b.gk[common, 0, 3, 7] = 0x40
    ref = b.attention(0.125)
    nan = np.isnan(ref)
    g = heads // kv
    assert nan[1, :g, 11].all() and nan[:members, :g, 40].all() and nan.sum() == g * (members + 1)
    out = b.shared(0.125).double().cpu().numpy()
    assert np.array_equal(np.isnan(out), nan)
    H.assert_attention_close(np.nan_to_num(out), np.nan_to_num(ref), "others", W.F16)
    assert int(b.err.item()) == 0


def zero_rows(out, rows):
    return bool((out[rows] == 0).all())


@pytest.mark.parametrize("case", ["too_long", "negative", "member", "context", "table", "end", "order"])
def test_shared_prefix_entries_that_cannot_be_used(case):
    """Flagged; the sequences concerned get zeros, the others their attention."""
    b = Shared(730, W.F16, 4, 2, 64, 16, [(3, [5, 6, 7]), (2, [8, 9])])
    ref = b.attention(0.125)
    kw, bad, bit = {}, [], B.PKV_DEVERR_PREFIX
    if case == "too_long":
        kw, bad = dict(max_prefix_blocks=2), [0, 1, 2]
    elif case == "negative":
        b.prefix[1], bad = -1, [3, 4]
        kw = dict(max_prefix_blocks=3)
    elif case == "member":
        kw, bad, bit = dict(max_group_size=2), [2], B.PKV_DEVERR_CONTEXT
    elif case == "context":
        b.gctx[1], bad, bit = 40, [1], B.PKV_DEVERR_CONTEXT            # below 3 x 16
    elif case == "table":
        b.gt[1, 1] = b.gt[4, 0]                                        # the first member's is used
    elif case == "end":
        b.begin[2], bad = 9, [3, 4]                                    # past the last sequence
        kw = dict(max_group_size=3)
    else:
        b.begin[1], bad = -4, [0, 1, 2]
        kw = dict(max_group_size=3)
    out = b.shared(0.125, **kw).double().cpu().numpy()
    assert int(b.err.item()) & bit
    assert (out[bad] == 0).all()
    if case != "order":                                                # (the second group then holds all)
        good = [i for i in range(5) if i not in bad]
        H.assert_attention_close(out[good], ref[good], "others", W.F16)


def test_shared_prefix_on_another_stream_and_captured():
    b = Shared(740, W.BF16, 8, 2, 128, 16, [(20, [100, 3, 40])])
    ref = b.shared(0.09)
    side = torch.cuda.Stream()
    q = b.dev16(b.q)
    n = B.pkv_decode_scaled_shared_prefix_workspace_bytes(b.desc, 3, 8, 1, 3, b.max_ctx)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    begin, prefix = torch.from_numpy(b.begin).cuda(), torch.from_numpy(b.prefix).cuda()
    torch.cuda.synchronize()

    def call(stream=None):
        return B.pkv_paged_attention_decode_scaled_shared_prefix(
            b.desc, b.gs, q, b.gt, b.gctx, b.max_ctx, begin, prefix, 3, 20, 0.09, workspace=ws,
            dev_err=b.err, stream=stream)

    assert torch.equal(call(side), ref)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, ref)
    assert int(b.err.item()) == 0


# ------------------------------------------------------------------ weights of a window

WINDOWS = [
    # dtype, heads, kv, D, bs, new, cached, window
    (W.F16, 4, 4, 64, 16, [5, 1, 37], [0, 20, 300], 16),
    (W.BF16, 8, 1, 128, 16, [40, 3, 0, 1], [0, 129, 50, 0], 32),            # 256 rows and less
    (W.BF16, 6, 2, 128, 8, [130, 200], [1, 77], 1),
    (W.F16, 2, 2, 128, 32, [127, 128, 129], [0, 0, 0], 200),                # whole prompts
    (W.BF16, 16, 1, 64, 16, [33, 34], [600, 1], 33),                        # 528 rows: three pairs of tiles
    (W.F16, 17, 1, 128, 16, [23], [1500], 23),                              # 391 rows, several runs of keys
    (W.F16, 1, 1, 64, 8, [1, 1, 1], [0, 511, 1024], 1),                     # single tokens
    (W.BF16, 128, 1, 64, 16, [4], [300], 3),
    (W.F16, 2, 1, 64, 16, [3], [20000], 2),                                 # an item over every CTA
]


def run_weights(b, scale, window, totals, desc=None, scales=None, **kw):
    return B.pkv_attention_weights(b.desc if desc is None else desc, b.dev16(b.q), b.gcu, window, b.gt,
                                   b.gctx, b.max_ctx, scale, totals, scales=scales, dev_err=b.err, **kw)


def some_totals(b, extra=3):
    """A strided view of random totals: rows of other lengths around it."""
    g = torch.Generator().manual_seed(5)
    n = len(b.ctx)
    big = torch.rand(n, b.kv + 1, b.max_ctx + extra, generator=g).cuda()
    return big, big[:, 1:, :b.max_ctx + 1]


@pytest.mark.parametrize("scale_sign", [1, -1])
@pytest.mark.parametrize("i", range(len(WINDOWS)))
def test_attention_weights_scaled(i, scale_sign):
    dt, h, kv, d, bs, new, cached, window = WINDOWS[i]
    b = Batch(800 + i, dt, h, kv, d, bs, new, cached, spread=1.0)
    b.append()
    b.oracle_append()
    big, w = some_totals(b)
    before, around = w.double().cpu().numpy().copy(), big.clone()
    out = run_weights(b, scale_sign * d ** -0.5, window, w, scales=b.gs)
    assert out is w
    torch.cuda.synchronize()
    assert int(b.err.item()) == 0
    add, size = OC.weights(Keys(b), b.q, b.cu, window, b.ctx, scale_sign * d ** -0.5)
    weights_close(w, before[..., :add.shape[2]], add, size, "window")
    # nothing behind a context, nor around the view
    for s, c in enumerate(b.ctx):
        assert torch.equal(w[s, :, c:], around[s, 1:, c:b.max_ctx + 1])
    assert torch.equal(big[:, 0], around[:, 0]) and torch.equal(big[..., -2:], around[..., -2:])
    # again, from the same totals: the same bits
    again = around.clone()
    run_weights(b, scale_sign * d ** -0.5, window, again[:, 1:, :b.max_ctx + 1], scales=b.gs)
    assert torch.equal(again, big)


@pytest.mark.parametrize("cache", [W.F16, W.BF16, W.E4M3])
@pytest.mark.parametrize("i", range(len(WINDOWS)))
def test_attention_weights_other_caches(i, cache):
    """16-bit caches, and E4M3 with one scale."""
    dt, h, kv, d, bs, new, cached, window = WINDOWS[i]
    if cache != W.E4M3:
        dt = cache
    b = Batch(830 + i, dt, h, kv, d, bs, new, cached, fill=False)
    r = np.random.default_rng(i)
    if cache == W.E4M3:
        b.k = r.integers(0, 256, b.k.shape, dtype=np.uint8) & 0xbf         # (at most 1.875)
        b.gk.copy_(torch.from_numpy(b.k))
        desc, keys = B.cache_desc(b.gk, b.gv, 0.75, 0.5), Keys(b, one_scale=0.75)
    else:
        k = torch.from_numpy(r.standard_normal(b.k.shape)).to(TD[dt])
        gk = k.cuda()
        desc, keys = B.cache_desc(gk, torch.zeros_like(gk)), Keys(b, k=k.double().numpy())
    w = torch.zeros(len(b.ctx), kv, b.max_ctx, device="cuda")
    run_weights(b, d ** -0.5, window, w, desc=desc)
    torch.cuda.synchronize()
    assert int(b.err.item()) == 0
    add, size = OC.weights(keys, b.q, b.cu, window, b.ctx, d ** -0.5)
    weights_close(w, 0.0, add, size, "window")


def test_attention_weights_scales_of_any_value_and_wide_scores():
    """Scales that are no powers of two and differ a lot, scores in the hundreds."""
    b = Batch(850, W.BF16, 4, 2, 128, 16, [9, 30], [700, 3], spread=0.0)
    b.append()
    b.oracle_append()
    b.scales *= np.exp(np.random.default_rng(1).uniform(-2, 3, b.scales.shape)).astype(np.float32)
    b.gs.copy_(torch.from_numpy(b.scales))
    w = torch.zeros(2, 2, b.max_ctx, device="cuda")
    run_weights(b, 0.5, 8, w, scales=b.gs)
    add, size = OC.weights(Keys(b), b.q, b.cu, 8, b.ctx, 0.5)
    assert size > 300
    weights_close(w, 0.0, add, size, "wide")


def test_attention_weights_of_unusable_sequences():
    b = Batch(851, W.F16, 4, 2, 64, 16, [5, 6, 7, 3], [0, 30, 9, 100])
    b.append()
    b.oracle_append()
    good, size = OC.weights(Keys(b), b.q, b.cu, 4, b.ctx, 0.125)
    b.gctx[0] = 3                                    # fewer tokens than rows
    b.gctx[2] = b.max_ctx + 1
    w = torch.zeros(4, 2, b.max_ctx, device="cuda")
    run_weights(b, 0.125, 4, w, scales=b.gs)
    assert int(b.err.item()) == B.PKV_DEVERR_CONTEXT
    good[[0, 2]] = 0
    weights_close(w, 0.0, good, size, "others")
    # a bad block: its keys are zeros
    b.gctx.copy_(torch.from_numpy(b.ctx))
    b.err.zero_()
    phys = int(b.tables[3, 2])
    b.gt[3, 2] = b.nb
    b.k[phys] = 0
    ref, size = OC.weights(Keys(b), b.q, b.cu, 4, b.ctx, 0.125)
    w.zero_()
    run_weights(b, 0.125, 4, w, scales=b.gs)
    assert int(b.err.item()) == B.PKV_DEVERR_BLOCK_ID
    weights_close(w, 0.0, ref, size, "bad block")


def test_attention_weights_hidden_nan():
    """A NaN key makes the rows that see it NaN, and no other."""
    b = Batch(852, W.F16, 1, 1, 64, 16, [8], [0])
    b.append()
    b.gk[int(b.tables[0, 0]), 0, 6, 3] = 0x7f
    w = torch.zeros(1, 1, 8, device="cuda")
    run_weights(b, 0.125, 2, w, scales=b.gs)         # rows 6 and 7 see key 6
    assert bool(w[0, 0].isnan().all())
    w.zero_()
    sub = torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    ctx = torch.tensor([6], dtype=torch.int32, device="cuda")
    B.pkv_attention_weights(b.desc, b.dev16(b.q), sub, 2, b.gt, ctx, 8, 0.125, w, scales=b.gs)
    assert bool(w.isfinite().all()) and abs(float(w.sum()) - 2) < 1e-5


# ------------------------------------------------------------------ decode with weights

DECODES = [
    # dtype, heads, kv, D, bs, ctx
    (W.F16, 4, 4, 64, 16, [5, 17, 33, 64]),
    (W.BF16, 8, 1, 128, 16, [1, 1000, 16, 15, 1024]),
    (W.BF16, 6, 2, 128, 8, [300, 7]),
    (W.F16, 2, 2, 128, 32, [1025, 3, 31]),                   # equal shares
    (W.BF16, 16, 1, 64, 16, [4000, 1, 90, 2500]),
    (W.F16, 7, 1, 128, 16, [30000]),                         # one item, many CTAs
    (W.BF16, 10, 5, 128, 32, [1500] * 9),
    (W.F16, 24, 8, 64, 8, [2000, 64, 65, 1030]),
]


@pytest.mark.parametrize("i", range(len(DECODES)))
def test_decode_adds_its_weights(i):
    dt, h, kv, d, bs, ctx = DECODES[i]
    b = filled(860 + i, dt, h, kv, d, bs, ctx, spread=1.0)
    big, w = some_totals(b)
    before, around = w.double().cpu().numpy().copy(), big.clone()
    args = (b.desc, b.gs, b.dev16(b.q), b.gt, b.gctx, b.max_ctx, d ** -0.5)
    out = B.pkv_paged_attention_decode_scaled_weights(*args, w, dev_err=b.err)
    torch.cuda.synchronize()
    assert int(b.err.item()) == 0
    H.assert_attention_close(out.double().cpu().numpy(), b.attention(d ** -0.5), "decode", dt)
    # the attention is that of the decode, bit for bit
    assert torch.equal(out, B.pkv_paged_attention_decode_scaled(*args))
    add, size = OC.weights(Keys(b), b.q, b.cu, 1, b.ctx, d ** -0.5)
    weights_close(w, before[..., :add.shape[2]], add, size, "decode")
    for s, c in enumerate(b.ctx):
        assert torch.equal(w[s, :, c:], around[s, 1:, c:b.max_ctx + 1])
    assert torch.equal(big[:, 0], around[:, 0]) and torch.equal(big[..., -2:], around[..., -2:])
    again = around.clone()
    B.pkv_paged_attention_decode_scaled_weights(*args, again[:, 1:, :b.max_ctx + 1])
    assert torch.equal(again, big)


def test_decode_weights_of_more_sequences_than_a_launch_takes():
    """1,030 sequences, of lengths 0 to 4 (one launch's route) and with one long."""
    r = np.random.default_rng(9)
    for longest in (4, 1100):
        ctx = r.integers(1, 5, 1030)
        ctx[1027] = longest
        b = filled(880, W.F16, 2, 1, 64, 8, ctx)
        b.gctx[5] = 0
        w = torch.zeros(1030, 1, b.max_ctx, device="cuda")
        args = (b.desc, b.gs, b.dev16(b.q), b.gt, b.gctx, b.max_ctx, 0.125)
        out = B.pkv_paged_attention_decode_scaled_weights(*args, w, dev_err=b.err)
        assert int(b.err.item()) == 0
        ref = b.attention(0.125)
        ref[5] = 0
        H.assert_attention_close(out.double().cpu().numpy(), ref, "many", W.F16)
        add, size = OC.weights(Keys(b), b.q, b.cu, 1, b.ctx, 0.125)
        add[5] = 0
        weights_close(w, 0.0, add, size, "many")


@pytest.mark.parametrize("longest", [700, 1700])
def test_decode_weights_of_unusable_sequences_and_blocks(longest):
    b = filled(881, W.BF16, 8, 2, 128, 16, [50, longest, 90, 64])
    add, size = OC.weights(Keys(b), b.q, b.cu, 1, b.ctx, 0.09)
    ref = b.attention(0.09)
    b.gctx[0], b.gctx[3] = -1, b.max_ctx + 5
    b.gt[2, 1] = -7
    w = torch.zeros(4, 2, b.max_ctx, device="cuda")
    out = B.pkv_paged_attention_decode_scaled_weights(
        b.desc, b.gs, b.dev16(b.q), b.gt, b.gctx, b.max_ctx, 0.09, w, dev_err=b.err)
    assert int(b.err.item()) == B.PKV_DEVERR_CONTEXT | B.PKV_DEVERR_BLOCK_ID
    assert zero_rows(out, [0, 3]) and not w[[0, 3]].any()
    assert not w[2, :, 16:32].any() and bool((w[2].sum(-1) - 4).abs().max() < 1e-4)
    weights_close(w[1:2], 0.0, add[1:2], size, "others")
    H.assert_attention_close(out[1:2].double().cpu().numpy(), ref[1:2], "others", W.BF16)


# ------------------------------------------------------------------ eviction

class Evicted:
    """An eviction on the device and in the oracle."""

    def __init__(self, seed, cache, d, bs, kv, ctx, keep, first, last, weights=None, odd_scales=False):
        self.r = r = np.random.default_rng(seed)
        self.ctx, self.keep = np.asarray(ctx, np.int32), np.asarray(keep, np.int32)
        self.kv, self.bs, self.first, self.last, self.cache = kv, bs, first, last, cache
        n = np.minimum(self.ctx, self.keep)
        counts, dcounts = -(-self.ctx // bs), -(-n // bs)
        nb = int(counts.sum() + dcounts.sum()) + 3
        order = r.permutation(nb).astype(np.int32)
        self.tables = np.full((len(ctx), max(1, counts.max())), -1, np.int32)
        self.dst = np.full((len(ctx), max(1, dcounts.max()) + 1), -1, np.int32)
        at = 0
        for i, (a, c) in enumerate(zip(counts, dcounts)):
            self.tables[i, :a] = order[at:at + a]
            self.dst[i, :c] = order[at + a:at + a + c]
            at += a + c
        shape = (nb, kv, bs, d)
        if cache in ("scaled", "e4m3"):
            self.k, self.v = (r.integers(0, 256, shape, dtype=np.uint8) for _ in range(2))
            for c in (self.k, self.v):
                c[c & 0x7f == 0x7f] = 0x38
            self.gk, self.gv = torch.from_numpy(self.k.copy()).cuda(), torch.from_numpy(self.v.copy()).cuda()
        else:
            self.k, self.v = (r.integers(0, 1 << 15, shape).astype(np.int16) for _ in range(2))
            self.gk, self.gv = (torch.from_numpy(x.copy()).cuda().view(cache) for x in (self.k, self.v))
        self.scales = None
        if cache == "scaled":
            e = r.uniform(-3, 3, (nb, kv, 2))
            self.scales = np.exp2(e if odd_scales else np.round(e)).astype(np.float32)
            self.gs = torch.from_numpy(self.scales.copy()).cuda()
        self.max_ctx, self.max_keep = int(self.ctx.max()), int(self.keep.max())
        if weights is None:
            weights = np.exp(2 * r.standard_normal((len(ctx), kv, self.max_ctx + 2))).astype(np.float32)
            weights = np.where(r.random(weights.shape) < 0.3, np.round(weights), weights)
        self.w = weights.astype(np.float32)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def dev(self, x):
        return torch.from_numpy(np.ascontiguousarray(x)).cuda()

    def run(self, **kw):
        a = dict(scales=None if self.scales is None else self.gs, dev_err=self.err)
        a.update(kw)
        return B.pkv_evict(B.cache_desc(self.gk, self.gv), self.dev(self.tables), self.dev(self.ctx),
                           self.max_ctx, self.dev(self.w), self.dev(self.keep), self.max_keep,
                           self.first, self.last, self.dev(self.dst), **a)

    def check(self, lens, out, skip=()):
        torch.cuda.synchronize()
        k, v, sc = self.k.copy(), self.v.copy(), None if self.scales is None else self.scales.copy()
        want = np.zeros(self.w.shape, np.float32)
        n = np.minimum(self.ctx, self.keep)
        for s in range(len(self.ctx)):
            if s in skip:
                continue
            for h in range(self.kv):
                idx = OC.kept(self.w[s, h, :self.ctx[s]], int(n[s]), self.first, self.last)
                want[s, h, :n[s]] = self.w[s, h, idx]
                for b0 in range(0, int(n[s]), self.bs):
                    part, to = idx[b0:b0 + self.bs], int(self.dst[s, b0 // self.bs])
                    src = self.tables[s, part // self.bs]
                    for j, c in enumerate((k, v)):
                        x = c[src, h, part % self.bs]
                        if sc is not None:
                            old = self.scales[src, h, j]
                            sc[to, h, j] = old.max()
                            f = (old / old.max())[:, None]         # fp32, as its rounding
                            y = (oracle.decode(oracle.E4M3, np.ascontiguousarray(x)).astype(np.float32) *
                                 f).astype(np.float32)
                            x = np.where(f == 1, x, oracle.encode_e4m3(y))
                        c[to, h, :len(part)] = x
        gk, gv = (t.view(torch.uint8 if self.k.dtype == np.uint8 else torch.int16).cpu().numpy()
                  for t in (self.gk, self.gv))
        good = [s for s in range(len(self.ctx)) if s not in skip]
        assert np.array_equal(lens.cpu().numpy()[good], n[good])
        got = out.cpu().numpy()
        assert np.array_equal(got[good, :, :self.max_ctx], want[good, :, :self.max_ctx], equal_nan=True)
        assert not got[good][:, :, self.max_ctx:].any()
        assert np.array_equal(gk, k), "K"
        assert np.array_equal(gv, v), "V"
        if sc is not None:
            assert np.array_equal(self.gs.cpu().numpy(), sc)


EVICTIONS = [
    # cache, D, bs, kv, ctx, keep, first, last
    ("scaled", 128, 16, 2, [100, 37, 5, 16], [40, 37, 50, 1], 4, 8),
    ("scaled", 64, 8, 3, [300, 299, 1], [64, 65, 1], 0, 0),
    ("scaled", 128, 32, 1, [5000, 0, 4097], [1000, 10, 4096], 16, 100),      # two CTAs a row
    (torch.float16, 64, 16, 2, [700, 301], [256, 128], 4, 64),
    (torch.bfloat16, 128, 8, 1, [90, 64], [33, 0], 1, 1),
    (torch.bfloat16, 128, 32, 2, [400], [399], 0, 399),
    ("e4m3", 128, 16, 2, [9000, 12], [512, 3], 2, 7),
    ("e4m3", 64, 32, 1, [64, 65, 66], [32, 33, 60], 40, 40),                 # more to keep than stays
    ("scaled", 64, 16, 1, [33000, 40000], [2049, 31000], 4, 32),             # read again in every round
    ("scaled", 64, 16, 2, [2561, 2560, 2049], [2000, 2559, 7], 4, 32),       # CTAs between the least and the most threads
    (torch.float16, 64, 16, 1, [4096, 4095], [1, 4000], 0, 0),
]


@pytest.mark.parametrize("i", range(len(EVICTIONS)))
def test_evict(i):
    e = Evicted(900 + i, *EVICTIONS[i])
    lens, out = e.run()
    assert int(e.err.item()) == 0
    e.check(lens, out)


@pytest.mark.parametrize("kind", ["equal", "zeros", "specials", "neighbours", "falling", "negative"])
def test_evict_ties_and_special_weights(kind):
    r = np.random.default_rng(3)
    w = np.ones((2, 2, 5000), np.float32)
    if kind == "zeros":
        w = np.where(r.random(w.shape) < 0.5, 0.0, -0.0)
    elif kind == "specials":
        w = r.choice([0.0, -0.0, np.nan, np.inf, -np.inf, 1e-45, 3.4e38, 1.0], w.shape)
    elif kind == "neighbours":
        w = np.nextafter(np.float32(1), np.float32(2)) * (r.random(w.shape) < 0.5) + \
            1.0 * (r.random(w.shape) < 0.5)
    elif kind == "falling":
        w = np.broadcast_to(np.arange(5000, 0, -1), w.shape)
    elif kind == "negative":
        w = r.standard_normal(w.shape)
    e = Evicted(950, "e4m3", 64, 16, 2, [4900, 3000], [1201, 2999], 3, 5, weights=np.asarray(w))
    lens, out = e.run()
    assert int(e.err.item()) == 0
    e.check(lens, out)


def test_evict_scales_of_any_value():
    e = Evicted(960, "scaled", 128, 16, 2, [300, 90], [100, 80], 0, 10, odd_scales=True)
    e.check(*e.run())
    assert int(e.err.item()) == 0


def test_evict_into_views_and_given_outputs():
    """Strided totals, longer rows to write, lengths of the caller's."""
    e = Evicted(961, torch.float16, 64, 16, 2, [100, 50], [40, 60], 1, 2)
    big = torch.full((2, 3, e.max_ctx + 60), 7.0, device="cuda")
    lens = torch.full((2,), -5, dtype=torch.int32, device="cuda")
    got, out = e.run(weights_out=big[:, :2, 5:], lens_out=lens)
    assert got is lens
    e.check(lens, out[:, :, :e.max_ctx + 2])
    assert bool((big[:, 2] == 7).all()) and bool((big[:, :, :5] == 7).all())
    assert not bool(out[:, :, e.max_ctx:].any())


def test_evict_unusable_sequences_and_blocks():
    e = Evicted(962, "scaled", 64, 16, 2, [100, 50, 64, 40, 70], [40, 30, 20, 20, 20], 1, 2)
    keep, ctx = e.keep.copy(), e.ctx.copy()
    e.keep = keep.copy()
    e.keep[1], e.ctx[3] = -1, e.max_ctx + 1
    out = torch.full(e.w.shape, 9.0, device="cuda")
    e.tables[2, 0], lost = -3, int(e.tables[2, 0])
    e.dst[4, 1] = 1 << 20
    lens, out = e.run(weights_out=out)
    torch.cuda.synchronize()
    assert int(e.err.item()) == B.PKV_DEVERR_CONTEXT | B.PKV_DEVERR_BLOCK_ID
    assert lens.tolist() == [40, 0, 20, 0, 20]
    assert bool((out[[1, 3]] == 9).all())
    e.keep, e.ctx = keep, ctx
    # nothing of the sequences that cannot be used is written
    for s in (1, 3):
        for t in range(-(-min(ctx[s], keep[s]) // 16)):
            i = int(e.dst[s, t])
            assert np.array_equal(e.gk[i].cpu().numpy(), e.k[i])
    # the bad source block's tokens are left out, whatever the rest
    idx = OC.kept(e.w[2, 0, :64], 20, 1, 2)
    first = idx[:16]
    to = int(e.dst[2, 0])
    here = np.flatnonzero(first // 16 == 0)
    assert len(here) and np.array_equal(e.gk[to, 0].cpu().numpy()[here], e.k[to, 0][here])
    assert lost >= 0


# ------------------------------------------------------------------ positions

def test_rope_append_position_offsets():
    """Rows turn by their place plus the offset, and are stored at their place."""
    r = np.random.default_rng(8)
    f = freqs(64)
    off = np.array([1000, 0, -3], np.int32)
    b = Batch(970, W.BF16, 4, 2, 64, 16, [20, 1, 7], [3, 16, 9])
    q = b.append(f, position_offsets=torch.from_numpy(off).cuda())
    pos = b.positions() + np.repeat(off, b.new)
    from test_gpu_scaled import check_rotated
    check_rotated(q, b.q, OS.rotate(b.q, pos, f), 1.0, W.BF16, "q")
    rk = OS.rotate(b.nk, pos, f)
    place = b.positions()
    seq = np.repeat(np.arange(3), b.new)
    gk, gs = b.gk.cpu().numpy(), b.gs.cpu().numpy()
    phys = b.tables[seq, place // 16]
    sc = gs[phys, :, 0].astype(np.float64)[..., None]
    got = oracle.decode(oracle.E4M3, gk[phys, :, place % 16]) * sc
    e = 2.0 ** -20 * 2 * np.abs(b.nk).max(-1, keepdims=True)
    assert (np.abs(got - rk) <= np.maximum(2.0 ** -4 * (np.abs(rk) + e), 2.0 ** -10 * sc) + e).all()
    c = Batch(970, W.BF16, 4, 2, 64, 16, [20, 1, 7], [3, 16, 9])
    zero = c.append(f, position_offsets=torch.zeros(3, dtype=torch.int32, device="cuda"))
    d = Batch(970, W.BF16, 4, 2, 64, 16, [20, 1, 7], [3, 16, 9])
    assert torch.equal(zero, d.append(f)) and torch.equal(c.gk, d.gk)
    assert r is not None and int(b.err.item()) == 0


# ------------------------------------------------------------------ together

def test_prompt_weighed_evicted_forked_and_decoded():
    """Two prompts are read and weighed, shrink, fork into samples that share what
    stayed and go on at their old positions; later steps weigh and evict again.
    Every attention against the oracle over what is then in the cache."""
    heads, kv, d, bs, f = 8, 2, 64, 16, freqs(64)
    b = Batch(990, W.BF16, heads, kv, d, bs, [300, 217], [0, 0])
    scale = d ** -0.5
    nb = b.nb + 80
    gk, gv = torch.full((nb, kv, bs, d), 0xff, dtype=torch.uint8, device="cuda"), None
    gv = gk.clone()
    gs = torch.full((nb, kv, 2), float("nan"), device="cuda")
    desc = B.cache_desc(gk, gv)
    inv, err = torch.from_numpy(f).cuda(), b.err
    free = list(range(b.nb, nb))
    gt = b.gt
    q = B.pkv_rope_append(desc, b.dev16(b.q), b.dev16(b.nk), b.dev16(b.nv), inv, b.gcu, 300, gt, b.gctx,
                          300, scales=gs, dev_err=err)
    out = B.pkv_paged_attention_prefill_scaled(desc, gs, q, b.gcu, 300, gt, b.gctx, 300, scale, dev_err=err)

    def attention(rows, cu, tables, ctx):
        return OS.attention(gk.cpu().numpy(), gv.cpu().numpy(), gs.cpu().numpy(),
                            rows.double().cpu().numpy(), cu, tables, ctx, scale)

    H.assert_attention_close(out.double().cpu().numpy(), attention(q, b.cu, b.tables, b.ctx), "prompts", W.BF16)
    w = torch.zeros(2, kv, 320, device="cuda")
    B.pkv_attention_weights(desc, q, b.gcu, 16, gt, b.gctx, 300, scale, w, scales=gs, dev_err=err)
    b.k, b.v, b.scales = gk.cpu().numpy(), gv.cpu().numpy(), gs.cpu().numpy()
    b.q = q.double().cpu().numpy()
    add, size = OC.weights(Keys(b), b.q, b.cu, 16, b.ctx, scale)
    weights_close(w, 0.0, add, size, "prompts")
    # down to 112 and 96 tokens: whole blocks, which the samples then share
    keep = torch.tensor([112, 96], dtype=torch.int32, device="cuda")
    dst = np.full((2, 7), -1, np.int32)
    for s, n in enumerate((7, 6)):
        dst[s, :n], free = free[:n], free[n:]
    lens, w = B.pkv_evict(desc, gt, b.gctx, 300, w, keep, 112, 4, 16, torch.from_numpy(dst).cuda(),
                          scales=gs, dev_err=err)
    assert lens.tolist() == [112, 96]
    # three samples each; the weights of what stayed are every sample's own
    tables = np.full((6, 10), -1, np.int32)
    for i in range(6):
        s = i // 3
        n = (7, 6)[s]
        tables[i, :n] = dst[s, :n]
        tables[i, n:n + 2], free = free[:2], free[2:]
    w = w.repeat_interleave(3, 0).contiguous()
    place = np.array([112] * 3 + [96] * 3, np.int32)
    ahead = np.array([300 - 112] * 3 + [217 - 96] * 3, np.int32)
    r = np.random.default_rng(4)
    begin = torch.tensor([0, 3, 6], dtype=torch.int32, device="cuda")
    prefix = torch.tensor([7, 6], dtype=torch.int32, device="cuda")
    t = torch.from_numpy(tables).cuda()
    cu = torch.arange(7, dtype=torch.int32, device="cuda")
    for step in range(3):
        qn, kn, vn = (torch.from_numpy(r.standard_normal((6, m, d))).bfloat16().cuda() for m in (heads, kv, kv))
        place = place + 1
        ctx = torch.from_numpy(place).cuda()
        top = int(place.max())
        qr = B.pkv_rope_append(desc, qn, kn, vn, inv, cu, 1, t, ctx, top, scales=gs, dev_err=err,
                               position_offsets=torch.from_numpy(ahead).cuda())
        want = OS.rotate(qn.double().cpu().numpy(), place - 1 + ahead, f)
        bad = np.abs(qr.double().cpu().numpy() - want) > 2.0 ** -8 * np.abs(want) + 2e-5
        assert not bad.any()
        ref = attention(qr, cu.cpu().numpy(), tables, place)
        got = B.pkv_paged_attention_decode_scaled_shared_prefix(desc, gs, qr, t, ctx, top, begin, prefix,
                                                                3, 7, scale, dev_err=err)
        H.assert_attention_close(got.double().cpu().numpy(), ref, "samples", W.BF16)
        before = w.double().cpu().numpy()
        got = B.pkv_paged_attention_decode_scaled_weights(desc, gs, qr, t, ctx, top, scale, w, dev_err=err)
        H.assert_attention_close(got.double().cpu().numpy(), ref, "samples", W.BF16)
        b.kv, b.ctx, b.tables = kv, place, tables
        b.k, b.scales = gk.cpu().numpy(), gs.cpu().numpy()
        add, size = OC.weights(Keys(b), qr.double().cpu().numpy(), cu.cpu().numpy(), 1, place, scale)
        weights_close(w, before[..., :add.shape[2]], add, size, "samples")
    # the samples part: each keeps what it needs, in blocks of its own
    dst = np.array(free[:30], np.int32).reshape(6, 5)
    keep = torch.full((6,), 70, dtype=torch.int32, device="cuda")
    lens, w2 = B.pkv_evict(desc, t, ctx, top, w, keep, 70, 4, 8, torch.from_numpy(dst).cuda(), scales=gs,
                           dev_err=err)
    assert lens.tolist() == [70] * 6
    host = w.cpu().numpy()
    for s in range(6):
        for h in range(kv):
            idx = OC.kept(host[s, h, :place[s]], 70, 4, 8)
            assert np.array_equal(w2[s, h, :70].cpu().numpy(), host[s, h, idx])
    got = B.pkv_paged_attention_decode_scaled(desc, gs, qr, torch.from_numpy(dst).cuda(), lens, 70, scale,
                                              dev_err=err)
    H.assert_attention_close(got.double().cpu().numpy(),
                             attention(qr, cu.cpu().numpy(), dst, lens.cpu().numpy()), "evicted", W.BF16)
    assert int(err.item()) == 0
