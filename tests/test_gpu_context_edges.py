"""The calls that share, weigh and evict at the edges of what they allow: waits that
run out, infinities and NaN in 16-bit caches, blocks that cannot be used, rows of
very different size, lengths whose products pass 32 bits.  Bounds as in
test_gpu_context."""
import threading

import numpy as np
import pytest
import torch

import harness as H
import oracle
from oracle import context as OC
from oracle import scaled as OS
from paged_kv_cache_130_gb300 import binding as B
from paged_kv_cache_130_gb300 import workloads as W
from test_gpu_context import Evicted, Keys, Shared, run_weights, weights_close
from test_gpu_scaled import TD, Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    H.build_library()
    yield
    B.pkv_testing_set_decode_wait_limit(0)


def sixteen_bit(seed, dt, heads, kv, d, bs, new, cached):
    """A Batch over a 16-bit cache: (batch, K on the device, its descriptor, K in 64 bits)."""
    b = Batch(seed, dt, heads, kv, d, bs, new, cached, fill=False)
    k = torch.from_numpy(np.random.default_rng(seed).standard_normal(b.k.shape)).to(TD[dt])
    gk = k.cuda()
    b.keep = torch.zeros_like(gk)                # (a descriptor keeps no reference itself)
    return b, gk, B.cache_desc(gk, b.keep), k.double().numpy()


# ------------------------------------------------------------------ waits that run out

def weighed(cache, new, cached):
    """(batch, arguments of its weights, keys in 64 bits) over a scaled or 16-bit cache."""
    if cache == "scaled":
        b = Batch(430, W.BF16, 8, 2, 128, 16, new, cached)
        b.append()
        b.oracle_append()
        return b, dict(scales=b.gs), Keys(b)
    b, gk, desc, k = sixteen_bit(430, cache, 8, 2, 128, 16, new, cached)
    b.gk = gk
    return b, dict(desc=desc), Keys(b, k=k)


@pytest.mark.parametrize("cache", ["scaled", W.BF16])
@pytest.mark.parametrize("new,cached", [([40, 1, 100], [3000, 0, 129]), ([3], [5])])
def test_weights_whose_wait_runs_out_flag_it_and_the_next_call_is_right(cache, new, cached):
    b, kw, keys = weighed(cache, new, cached)
    w = torch.zeros(len(new), 2, b.max_ctx, device="cuda")
    B.pkv_testing_set_decode_wait_limit(1)
    try:
        run_weights(b, 0.09, 64, w, **kw)
        torch.cuda.synchronize()
    finally:
        B.pkv_testing_set_decode_wait_limit(0)
    assert int(b.err.item()) & B.PKV_DEVERR_TIMEOUT
    b.err.zero_()
    w.zero_()
    run_weights(b, 0.09, 64, w, **kw)
    assert int(b.err.item()) == 0
    add, size = OC.weights(keys, b.q, b.cu, 64, b.ctx, 0.09)
    weights_close(w, 0.0, add, size, "after a time-out")


@pytest.mark.parametrize("cache", ["scaled", W.BF16])
def test_weights_whose_sums_run_out_leave_the_totals_alone(cache):
    """The limit reaches the pass for the sums only: whenever it runs out, at the first
    wait or on the way, nothing is added; else everything is."""
    b, kw, keys = weighed(cache, [40, 1, 300], [9000, 200, 129])
    before = torch.rand(3, 2, b.max_ctx, device="cuda")
    add, size = OC.weights(keys, b.q, b.cu, 64, b.ctx, 0.09)
    ran_out = []
    for i in range(40):
        w = before.clone()
        b.err.zero_()
        B.pkv_testing_set_decode_wait_limit(int(2 ** (i / 3)))
        try:
            run_weights(b, 0.09, 64, w, **kw)
            torch.cuda.synchronize()
        finally:
            B.pkv_testing_set_decode_wait_limit(0)
        ran_out.append(int(b.err.item()) == B.PKV_DEVERR_TIMEOUT)
        if ran_out[-1]:
            assert torch.equal(w, before), i
        else:
            assert int(b.err.item()) == 0
            weights_close(w, before.double().cpu().numpy()[..., :add.shape[2]], add, size, "all the same")
    assert ran_out[0]
    b.err.zero_()
    w = before.clone()
    run_weights(b, 0.09, 64, w, **kw)
    assert int(b.err.item()) == 0
    weights_close(w, before.double().cpu().numpy()[..., :add.shape[2]], add, size, "after a time-out")


# ------------------------------------------------------------------ infinities in 16-bit caches

INFINITIES = [
    # heads, kv, D, bs, new, cached, window, keys of score -inf, keys of score +inf
    (1, 1, 64, 16, [1], [4], 1, [0], []),
    (4, 2, 64, 8, [3, 5], [40, 7], 2, [0], []),
    (4, 4, 128, 16, [20], [130], 20, [0, 16, 128], []),
    (8, 1, 128, 32, [40], [300], 33, list(range(17)), []),     # 264 rows; a whole column block, and one more
    (2, 2, 64, 16, [9], [380], 8, list(range(130)) + [256], []),       # a whole tile
    (2, 1, 64, 16, [1], [129], 1, list(range(128)), []),       # all but the last two
    (4, 2, 64, 16, [30], [110], 30, [0, 128], [135]),          # rows from 135 on see +inf
    (2, 2, 128, 16, [4], [400], 3, [5], [128]),                # every row does
    (2, 1, 64, 8, [20], [0], 6, [1, 3], [16]),
    (1, 1, 64, 16, [2], [20000], 2, [0, 128, 2560], []),       # an item over every CTA
    # warps of 32 rows each (a row of nobody is zeros, and 0 times an infinity NaN)
    (32, 1, 64, 16, [1], [4], 1, [0], []),                     # five tokens: no column behind the first 16
    (4, 4, 64, 8, [32], [5], 32, [0], []),
    (8, 1, 128, 16, [16], [120], 16, [0, 16, 128], []),        # where tiles and column blocks start
    (16, 1, 64, 16, [8], [250], 8, list(range(128, 145)), []), # an edge tile behind an inner one
    (16, 1, 128, 32, [48], [240], 48, [256], [270]),           # 768 rows; those from 270 on see +inf
    (32, 1, 64, 16, [1], [130], 1, list(range(129)), []),      # a tile of which the rows see two keys
]


@pytest.mark.parametrize("dt", [W.F16, W.BF16])
@pytest.mark.parametrize("i", range(len(INFINITIES)))
def test_weights_of_keys_with_infinite_scores(i, dt):
    """-inf is a weight of 0, and the others keep theirs; a row that sees +inf is NaN
    where it sees a key, and reaches no other."""
    h, kv, d, bs, new, cached, window, low, high = INFINITIES[i]
    b, gk, desc, k = sixteen_bit(440 + i, dt, h, kv, d, bs, new, cached)
    b.q[..., 0] = 0.25 + np.abs(b.q[..., 0])
    b.q = b.dev16(b.q).double().cpu().numpy()
    finite = k.copy()
    for keys, value in ((low, -np.inf), (high, np.inf)):
        for s, c in enumerate(b.ctx):
            for t in keys:
                if t < c:
                    k[b.tables[s, t // bs], :, t % bs, 0] = value
                    finite[b.tables[s, t // bs], :, t % bs, 0] = 0.0
    gk.copy_(torch.from_numpy(k))
    w = torch.zeros(len(new), kv, b.max_ctx, device="cuda")
    run_weights(b, 0.125, window, w, desc=desc)
    assert int(b.err.item()) == 0
    _, size = OC.weights(Keys(b, k=finite), b.q, b.cu, window, b.ctx, 0.125)
    with np.errstate(invalid="ignore"):
        add, _ = OC.weights(Keys(b, k=k), b.q, b.cu, window, b.ctx, 0.125)
    nan = np.isnan(add)
    assert nan.any() == bool(high) and np.array_equal(w.isnan().cpu().numpy(), nan)
    weights_close(w.nan_to_num(0.0), 0.0, np.nan_to_num(add), size, "infinite scores")


@pytest.mark.parametrize("dt", [W.F16, W.BF16])
def test_weights_nan_in_a_sixteen_bit_cache(dt):
    """A NaN key makes the rows that see it NaN where they see a key; behind a row's
    position, behind a context or in a block of nobody it reaches nothing."""
    b, gk, desc, k = sixteen_bit(460, dt, 4, 2, 64, 16, [12, 3], [190, 40])
    used = np.unique(np.concatenate([b.tables[s, :-(-c // 16)] for s, c in enumerate(b.ctx)]))
    k[np.setdiff1d(np.arange(b.nb), used)] = np.nan
    for s, c in enumerate(b.ctx):                             # slots behind the last token
        k[b.tables[s, (c - 1) // 16], :, c % 16 or 16:] = np.nan
    k[b.tables[0, 195 // 16], 1, 195 % 16, 7] = np.nan        # rows at 195 and later see it
    gk.copy_(torch.from_numpy(k))
    w = torch.zeros(2, 2, b.max_ctx, device="cuda")
    run_weights(b, 0.125, 12, w, desc=desc)
    assert int(b.err.item()) == 0
    got = w.isnan().cpu().numpy()
    want = np.zeros_like(got)
    want[0, 1, :202] = True
    assert np.array_equal(got, want)
    add, size = OC.weights(Keys(b, k=np.nan_to_num(k)), b.q, b.cu, 12, b.ctx, 0.125)
    add[0, 1, :202] = 0
    weights_close(w.nan_to_num(0.0), 0.0, add, size, "others")


@pytest.mark.parametrize("dt", [W.F16, W.BF16])
def test_weights_of_bad_blocks_in_a_sixteen_bit_cache(dt):
    """Their keys are zeros, and get the weight of such a key."""
    b, gk, desc, k = sixteen_bit(461, dt, 4, 2, 64, 8, [9, 4], [150, 5])
    for (s, j), bad in {(0, 0): -1, (0, 16): b.nb, (0, 17): 1 << 30, (1, 1): b.nb + 7}.items():
        k[b.tables[s, j]] = 0.0
        b.gt[s, j] = bad
    w = torch.zeros(2, 2, b.max_ctx, device="cuda")
    run_weights(b, 0.125, 5, w, desc=desc)
    assert int(b.err.item()) == B.PKV_DEVERR_BLOCK_ID
    add, size = OC.weights(Keys(b, k=k), b.q, b.cu, 5, b.ctx, 0.125)
    weights_close(w, 0.0, add, size, "bad blocks")


# ------------------------------------------------------------------ shared prefixes

BAD_BLOCKS = [
    # dtype, heads, kv, D, bs, members, prefix blocks, their own tokens, bad blocks of the prefix
    (W.F16, 4, 2, 64, 16, 3, 10, [20, 1, 7], [0, 4]),                        # shares, 6 rows
    (W.BF16, 8, 1, 128, 16, 4, 10, [20, 1, 7, 0], [9]),                      # shares, 32 rows
    (W.BF16, 8, 1, 128, 16, 5, 10, [20, 1, 7, 0, 3], [9]),                   # the kernel of the prefixes, 40
    (W.F16, 16, 2, 64, 16, 9, 70, [3] * 9, list(range(32, 64))),             # a run of bad blocks only
    (W.BF16, 8, 2, 128, 8, 12, 140, [1, 30] * 6, list(range(16)) + [40, 139]),   # first a tile of them
    (W.F16, 8, 1, 64, 32, 6, 40, [2] * 6, list(range(0, 40, 2))),
    (W.BF16, 3, 1, 128, 16, 20, 6, [5, 70] * 10, list(range(6))),            # all of them
    (W.F16, 3, 1, 128, 16, 2, 6, [5, 70], list(range(6))),
    (W.F16, 4, 4, 64, 16, 40, 9, [4] * 40, [3]),
]


@pytest.mark.parametrize("odd_scales", [False, True])
@pytest.mark.parametrize("i", range(len(BAD_BLOCKS)))
def test_bad_blocks_of_a_shared_prefix_contribute_nothing(i, odd_scales):
    """On either side of the rule that gives prefixes a kernel of their own, as in the
    plain decode: the attention over the tokens that are there."""
    dt, h, kv, d, bs, members, blocks, own, bad = BAD_BLOCKS[i]
    b = Shared(470 + i, dt, h, kv, d, bs, [(blocks, own), (2, [9, 1])])
    if odd_scales:
        b.scales *= np.random.default_rng(i).uniform(1, 2, b.scales.shape).astype(np.float32)
        b.gs.copy_(torch.from_numpy(b.scales))
    for n, j in enumerate(bad):
        b.gt[:members, j] = (-1, b.nb, 1 << 30)[n % 3]
    out = b.shared(0.125)
    assert int(b.err.item()) == B.PKV_DEVERR_BLOCK_ID
    # the reference: tables without those blocks
    stay = [j for j in range(b.tables.shape[1]) if j not in bad]
    tables = b.tables.copy()
    tables[:members] = -1
    tables[:members, :len(stay)] = b.tables[:members][:, stay]
    ctx = b.ctx.copy()
    ctx[:members] -= bs * len(bad)
    ref = OS.attention(b.k, b.v, b.scales, b.q, b.cu, tables, ctx, 0.125)
    H.assert_attention_close(out.double().cpu().numpy(), ref, "bad prefix blocks", dt)


# ------------------------------------------------------------------ lengths whose products pass 32 bits

@pytest.mark.parametrize("heads,ctx,size", [
    (128, (1 << 24) + 500, 20),                 # a power of two for each row of q
    (100, (1 << 31) // 100 + 700, 0),           # rows that do not fill a tile
])
def test_weights_of_keys_far_behind_the_window(heads, ctx, size):
    """Millions of tokens of a few blocks, one row of many heads: tokens x heads passes
    32 bits for the first ones."""
    r = np.random.default_rng(7)
    kinds, d, bs = 128, 64, 32
    k = r.integers(0, 256, (4, 1, bs, d), dtype=np.uint8) & 0xb7       # (at most 0.9375)
    q = r.standard_normal((1, heads, d))
    q[0, heads // 2] *= 2.0 ** -size
    gq = torch.from_numpy(q).bfloat16().cuda()
    gk = torch.from_numpy(k).cuda()
    gv = torch.zeros_like(gk)
    gs = torch.ones(4, 1, 2, device="cuda")
    table = (torch.arange(-(-ctx // bs), dtype=torch.int32, device="cuda") % 4).view(1, -1)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    w = torch.zeros(1, 1, ctx, device="cuda")
    lens = torch.tensor([ctx], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    B.pkv_attention_weights(B.cache_desc(gk, gv), gq, cu, 1, table, lens, ctx, 0.25, w, scales=gs, dev_err=err)
    assert int(err.item()) == 0
    x = gq[0].double().cpu().numpy()
    keys = oracle.decode(oracle.E4M3, k).reshape(kinds, d)
    s = 0.25 * x @ keys.T
    p = np.exp(s - s.max(1, keepdims=True))
    counts = np.full(kinds, ctx // kinds) + (np.arange(kinds) < ctx % kinds)
    add = (p / (p * counts).sum(1, keepdims=True)).sum(0)
    add = np.tile(add, -(-ctx // kinds))[None, None, :ctx]
    weights_close(w, 0.0, add, 0.25 * (abs(x) @ abs(keys).T).max(), "far")


# ------------------------------------------------------------------ rows of very different size

@pytest.mark.parametrize("exact", [True, False])
def test_weights_of_small_elements_beside_a_large_one(exact):
    """bf16 rows of a tile share a power of two while their largest elements lie within
    2^12 of each other: a row's elements from 2^-18 of its largest on are exact, smaller
    ones off by 2^-26 of it at most.  Here a row's large element meets keys of 0, and the
    small ones decide."""
    b = Batch(480, W.BF16, 4, 2, 64, 16, [20], [300])
    b.append()
    b.oracle_append()
    b.k[..., 0] = 0
    b.gk.copy_(torch.from_numpy(b.k))
    r = np.random.default_rng(1)
    low = -18 if exact else -24
    q = r.choice([-1.0, 1.0], b.q.shape) * (1 + r.integers(0, 128, b.q.shape) / 128) * \
        2.0 ** r.integers(low, -15 if exact else -20, b.q.shape)
    q[..., 0] = 1.0                             # (the row's largest: up to 2^-12 of the tile's)
    q[7, 1, 0] = 2.0 ** 12
    b.q = q
    assert np.array_equal(b.dev16(q).double().cpu().numpy(), q)
    scale = 2.0 ** (12 if exact else 17)
    w = torch.zeros(1, 2, b.max_ctx, device="cuda")
    run_weights(b, scale, 20, w, scales=b.gs)
    assert int(b.err.item()) == 0
    keys = Keys(b)
    add, size = OC.weights(keys, b.q, b.cu, 20, b.ctx, scale)
    if not exact:
        # what the elements lose moves a score by 2^-26 of the row's largest times the
        # key's magnitudes; the bound of a score is 2^-19 (size + 1)
        lost = scale * 2.0 ** -26 * max(np.abs(keys(0, h)).sum(1).max() for h in range(2))
        assert lost < 0.2
        size += lost * 2.0 ** 19
    weights_close(w, 0.0, add, size, "small elements")


# ------------------------------------------------------------------ totals in any order

def by_head(n, kv, tokens):
    """Totals [n, kv, tokens] that lie head by head."""
    return torch.rand(kv, n, tokens, device="cuda").transpose(0, 1)


def test_totals_that_lie_head_by_head():
    """Rows that do not overlap, the KV heads outside the sequences."""
    b = Batch(490, W.F16, 4, 2, 64, 16, [5, 1, 9], [100, 40, 3])
    b.append()
    b.oracle_append()
    w = by_head(3, 2, b.max_ctx + 1)
    assert w.stride(1) > w.stride(0) > b.max_ctx
    dense = w.contiguous()
    run_weights(b, 0.125, 4, w, scales=b.gs)
    run_weights(b, 0.125, 4, dense, scales=b.gs)
    assert torch.equal(w, dense)
    one = Batch(491, W.F16, 4, 2, 64, 16, [1, 1, 1], [100, 40, 3])
    one.append()
    args = (one.desc, one.gs, one.dev16(one.q), one.gt, one.gctx, one.max_ctx, 0.125)
    for t in (w, dense):
        B.pkv_paged_attention_decode_scaled_weights(*args, t, dev_err=one.err)
    assert torch.equal(w, dense)
    e = Evicted(492, "scaled", 64, 16, 2, [100, 37, 5], [40, 37, 50], 4, 8)
    lens, out = e.run(weights_out=by_head(3, 2, e.max_ctx + 2))
    e.check(lens, out)
    assert int(b.err.item()) == int(one.err.item()) == int(e.err.item()) == 0


# ------------------------------------------------------------------ calls at once

def test_calls_of_several_threads_at_once():
    """Four threads, each on a stream and with tensors of its own, make every call again
    and again: the results are those of one call after the other."""
    jobs = []
    for i in range(4):
        s = Shared(500 + i, W.F16, 8, 2, 64, 16, [(40, [3] * 10), (0, [5])])     # 40 rows: both kernels
        b, kw, _ = weighed(W.BF16 if i % 2 else "scaled", [40, 1], [500 + i, 129])
        n = torch.zeros(2, 2, b.max_ctx, device="cuda")
        e = Evicted(510 + i, torch.float16, 64, 16, 2, [700, 301], [256, 128], 4, 64)
        t = torch.zeros(11, 2, s.max_ctx, device="cuda")

        def work(s=s, b=b, kw=kw, n=n, e=e, t=t):
            a = s.shared(0.125)
            run_weights(b, 0.09, 16, n.zero_(), **kw)
            B.pkv_paged_attention_decode_scaled_weights(s.desc, s.gs, s.dev16(s.q), s.gt, s.gctx, s.max_ctx,
                                                        0.125, t.zero_(), dev_err=s.err)
            return [a, n.clone(), t.clone()] + list(e.run())

        want = work()
        torch.cuda.synchronize()
        jobs.append((work, want, s, b, e))
    wrong, start = [], threading.Barrier(4)

    def go(i):
        try:
            work, want = jobs[i][:2]
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait(30)
                for _ in range(20):
                    got = work()
                    torch.cuda.current_stream().synchronize()
                    wrong.extend(i for x, y in zip(got, want) if not torch.equal(x, y))
        except Exception as ex:                      # (a thread's own failure is the test's)
            wrong.append(ex)

    threads = [threading.Thread(target=go, args=(i,)) for i in range(4)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert not wrong
    assert all(int(x.err.item()) == 0 for j in jobs for x in j[2:])


# ------------------------------------------------------------------ evictions with bad blocks

@pytest.mark.parametrize("cache", ["scaled", "e4m3", torch.bfloat16])
def test_evict_with_bad_blocks_and_unusable_sequences_in_full(cache):
    """Every byte of the pools, the scales, totals and lengths: the usable sequence and
    the good blocks are as without the others, what a bad block holds or would hold is
    left out, and nothing else changes."""
    e = Evicted(520, cache, 64, 16, 2, [100, 50, 64, 40, 70], [40, 30, 33, 20, 20], 1, 2, odd_scales=True)
    keep, ctx, tables, dst = e.keep.copy(), e.ctx.copy(), e.tables.copy(), e.dst.copy()
    e.keep[1], e.ctx[3] = -1, e.max_ctx + 1
    e.tables[2, 0], e.tables[2, 3] = -3, 1 << 20               # (its first token stays in any case)
    e.dst[4, 1] = len(e.k)
    out = torch.full(e.w.shape, 9.0, device="cuda")
    lens, got = e.run(weights_out=out)
    torch.cuda.synchronize()
    assert int(e.err.item()) == B.PKV_DEVERR_CONTEXT | B.PKV_DEVERR_BLOCK_ID
    assert lens.tolist() == [40, 0, 33, 0, 20]
    k, v, sc = e.k.copy(), e.v.copy(), None if e.scales is None else e.scales.copy()
    want = np.full(e.w.shape, 9.0, np.float32)
    for s, n in ((0, 40), (2, 33), (4, 20)):
        want[s] = 0
        for h in range(2):
            idx = OC.kept(e.w[s, h, :ctx[s]], n, 1, 2)
            want[s, h, :n] = e.w[s, h, idx]
            for b0 in range(0, n, 16):
                part = idx[b0:b0 + 16]
                slot = np.arange(len(part))
                if (s, b0) == (4, 16):
                    continue                                   # the destination that is not there
                if s == 2:
                    there = (part // 16 != 0) & (part // 16 != 3)
                    part, slot = part[there], slot[there]
                src, to = tables[s, part // 16], int(dst[s, b0 // 16])
                for j, (pool, old) in enumerate(((k, e.k), (v, e.v))):
                    x = old[src, h, part % 16]
                    if sc is not None and len(part):
                        was = e.scales[src, h, j]
                        sc[to, h, j] = was.max()
                        f = (was / was.max())[:, None]         # fp32, as its rounding
                        y = (oracle.decode(oracle.E4M3, np.ascontiguousarray(x)).astype(np.float32) * f)
                        x = np.where(f == 1, x, oracle.encode_e4m3(y.astype(np.float32)))
                    pool[to, h, slot] = x
    bits = torch.uint8 if e.k.dtype == np.uint8 else torch.int16
    assert np.array_equal(e.gk.view(bits).cpu().numpy(), k) and np.array_equal(e.gv.view(bits).cpu().numpy(), v)
    assert sc is None or np.array_equal(e.gs.cpu().numpy(), sc)
    assert np.array_equal(got.cpu().numpy(), want)


# ------------------------------------------------------------------ prefixes with a kernel of their own

def test_prefix_kernel_on_another_stream_in_graphs_and_twice_over_a_workspace():
    """80 rows of a group over 1,600 tokens (runs of 512 keys): the shares' kernel starts
    beside the prefixes' and waits at its end, and the reduce behind both.  Two batches
    over one workspace, on a stream of their own and in graphs that are replayed in
    turn, give the bits that each gives alone."""
    pair = [Shared(530, W.BF16, 8, 1, 128, 16, [(100, [100, 3, 40, 1, 0, 9, 64, 65, 2, 500])]),
            Shared(531, W.BF16, 8, 1, 128, 16, [(33, [7] * 8), (70, [1, 300])])]
    calls, want = [], []
    for b in pair:
        n, groups = len(b.ctx), len(b.prefix)
        size = int(np.diff(b.begin).max())
        assert 8 * size > 32
        calls.append(dict(cache=b.desc, scales=b.gs, q=b.dev16(b.q), block_tables=b.gt, context_lens=b.gctx,
                          max_context_len=b.max_ctx, group_begin=torch.from_numpy(b.begin).cuda(),
                          group_prefix_blocks=torch.from_numpy(b.prefix).cuda(), max_group_size=size,
                          max_prefix_blocks=int(b.prefix.max()), scale=0.09, dev_err=b.err,
                          out=torch.empty(n, 8, 128, dtype=torch.bfloat16, device="cuda")))
        calls[-1]["need"] = B.pkv_decode_scaled_shared_prefix_workspace_bytes(b.desc, n, 8, groups, size, b.max_ctx)
        want.append(b.shared(0.09))
        H.assert_attention_close(want[-1].double().cpu().numpy(), b.attention(0.09), "prefix kernel", W.BF16)
    ws = torch.empty(max(c.pop("need") for c in calls), dtype=torch.uint8, device="cuda")
    fn = B.pkv_paged_attention_decode_scaled_shared_prefix
    torch.cuda.synchronize()

    def right():
        torch.cuda.synchronize()
        for c, x in zip(calls, want):
            assert torch.equal(c["out"], x)
            c["out"].zero_()
        ws.fill_(0xff)                                        # (NaN wherever a partial is not written again)

    side = torch.cuda.Stream()
    for _ in range(20):
        for c in calls:
            fn(**c, workspace=ws, stream=side)
    right()
    for _ in range(20):
        for c in calls:
            fn(**c, workspace=ws)
    right()
    graphs = []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fn(**c, workspace=ws)
        graphs.append(g)
    for _ in range(20):
        for g in graphs:
            g.replay()
    right()
    both = torch.cuda.CUDAGraph()
    with torch.cuda.graph(both):
        for c in calls:
            fn(**c, workspace=ws)
    for _ in range(20):
        both.replay()
    right()
    assert all(int(b.err.item()) == 0 for b in pair)


# ------------------------------------------------------------------ a scale of 0

def test_a_scale_of_zero_weighs_every_token_alike():
    """Every call: the mean over the tokens, weights of 1 / their number."""
    for members in (3, 10):                                    # 12 rows a group, and 40: shares, own kernel
        s = Shared(540 + members, W.F16, 8, 2, 64, 16, [(40, [3] * members), (0, [5])])
        H.assert_attention_close(s.shared(0.0).double().cpu().numpy(), s.attention(0.0), "scale 0", W.F16)
        w = torch.zeros(members + 1, 2, s.max_ctx, device="cuda")
        B.pkv_paged_attention_decode_scaled_weights(s.desc, s.gs, s.dev16(s.q), s.gt, s.gctx, s.max_ctx, 0.0, w,
                                                    dev_err=s.err)
        add, size = OC.weights(Keys(s), s.q, s.cu, 1, s.ctx, 0.0)
        assert size == 0.0
        weights_close(w, 0.0, add, size, "scale 0")
        assert int(s.err.item()) == 0
    for cache in ("scaled", W.F16, W.BF16):
        b, kw, keys = weighed(cache, [40, 1], [300, 129])
        w = torch.zeros(2, 2, b.max_ctx, device="cuda")
        run_weights(b, 0.0, 33, w, **kw)
        add, size = OC.weights(keys, b.q, b.cu, 33, b.ctx, 0.0)
        weights_close(w, 0.0, add, size, "scale 0")
        assert int(b.err.item()) == 0
