"""How the scaled-cache calls and the rotary append treat what surrounds them:
streams, memory they allocate, and arguments they refuse."""
import pytest
import torch

import harness as H
from test_gpu_scaled import Batch, freqs

from paged_kv_cache_130_gb300 import binding as B
from paged_kv_cache_130_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    H.build_library()


def pool_of(address):
    """Handle of the stream whose memory pool holds an address."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= address < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not torch's memory")


def scaled_calls(b, f, stream):
    """Every call that allocates, on `stream`: name -> a function that makes it."""
    q, k, v = (b.dev16(x) for x in (b.q, b.nk, b.nv))
    kw = dict(dev_err=b.err, stream=stream)
    return dict(
        rope=lambda: B.pkv_rope_append(b.desc, q, k, v, f, b.gcu, b.max_new, b.gt, b.gctx,
                                       b.max_ctx, scales=b.gs, **kw),
        decode=lambda: B.pkv_paged_attention_decode_scaled(b.desc, b.gs, q, b.gt, b.gctx,
                                                           b.max_ctx, 0.125, **kw),
        prefill=lambda: B.pkv_paged_attention_prefill_scaled(b.desc, b.gs, q, b.gcu, b.max_new,
                                                             b.gt, b.gctx, b.max_ctx, 0.125, **kw))


@pytest.mark.parametrize("as_number", [False, True])
def test_what_a_call_on_another_stream_allocates_is_that_streams(as_number, monkeypatch):
    """Outputs and workspace come from the pool of the stream they are written
    on: a block of the current stream's could still be read there."""
    b = Batch(300, W.BF16, 8, 2, 64, 16, [1, 1, 1], [1500, 30, 1200])
    f = torch.from_numpy(freqs(64)).cuda()
    side = torch.cuda.Stream()
    calls = scaled_calls(b, f, side.cuda_stream if as_number else side)
    torch.cuda.synchronize()
    made = []
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made.append(empty(*a, **k)) or made[-1])
    for name, call in calls.items():
        out = call()
        assert pool_of(out.data_ptr()) == side.cuda_stream, name
        torch.cuda.synchronize()
    assert made and all(pool_of(t.data_ptr()) == side.cuda_stream for t in made)
    assert int(b.err.item()) == 0


def test_a_call_on_another_stream_leaves_memory_in_use_alone():
    """The current stream is busy and then reads tensors that their owner has let
    go of; calls on another stream that could get that memory must not write it."""
    b = Batch(301, W.BF16, 8, 2, 64, 16, [1, 1, 1], [1500, 30, 1200])
    f = torch.from_numpy(freqs(64)).cuda()
    side = torch.cuda.Stream()
    calls = scaled_calls(b, f, side)
    torch.cuda.synchronize()
    like = calls["decode"]()
    calls["prefill"]()
    torch.cuda.synchronize()
    for name in ("decode", "prefill"):
        xs = [torch.full_like(like, float(i)) for i in range(8)]
        ys = [torch.empty_like(like) for _ in xs]
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)                       # ~10 ms
        for x, y in zip(xs, ys):
            y.copy_(x)
        del x, xs
        outs = [calls[name]() for _ in range(8)]
        torch.cuda.synchronize()
        assert all((y == i).all() for i, y in enumerate(ys))
        # (bits: the last token's K and V are not written, and read as NaN)
        bits = [o.view(torch.int16) for o in outs]
        assert all(torch.equal(x, bits[0]) for x in bits)


def test_calls_on_another_stream_in_a_captured_graph():
    """A capture that forks to another stream and joins it again."""
    b = Batch(302, W.BF16, 8, 2, 64, 16, [1, 1, 1], [1500, 30, 1200])
    b.oracle_append()
    b.upload()
    f = torch.from_numpy(freqs(64)).cuda()
    side = torch.cuda.Stream()
    calls = scaled_calls(b, f, side)
    side.wait_stream(torch.cuda.current_stream())
    want = [calls[n]() for n in ("decode", "prefill")]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        got = [calls[n]() for n in ("decode", "prefill")]
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        for t in got:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(want, got))
    assert int(b.err.item()) == 0


class Elsewhere:
    """A tensor as it would look on another GPU."""

    def __init__(self, t):
        self._t = t

    def get_device(self):
        return self._t.get_device() + 1

    def __getattr__(self, name):
        return getattr(self._t, name)


def arguments():
    """name of a call -> (function, arguments that it takes without complaint)"""
    b = Batch(310, W.F16, 4, 2, 64, 16, [1, 1], [20, 5])
    q = b.dev16(b.q)
    f = torch.from_numpy(freqs(64)).cuda()
    common = dict(cache=b.desc, scales=b.gs, q=q, block_tables=b.gt, context_lens=b.gctx,
                  max_context_len=21, dev_err=b.err)
    attend = dict(common, scale=0.125, out=torch.empty_like(q))
    n = B.pkv_decode_scaled_workspace_bytes(b.desc, 2, 4, 21, 16)
    return dict(
        rope=(B.pkv_rope_append, dict(common, k=b.dev16(b.nk), v=b.dev16(b.nv), inv_freq=f,
                                      cu_seqlens_q=b.gcu, max_q_len=1, q_out=torch.empty_like(q))),
        decode=(B.pkv_paged_attention_decode_scaled,
                dict(attend, partition_size=16,
                     workspace=torch.empty(n, dtype=torch.uint8, device="cuda"))),
        prefill=(B.pkv_paged_attention_prefill_scaled,
                 dict(attend, cu_seqlens_q=b.gcu, max_q_len=1)),
        copy=(B.pkv_copy_blocks_scaled,
              dict(caches=b.desc, scales=b.gs, dev_err=b.err,
                   block_pairs=torch.tensor([[0, 1]], device="cuda"))))


def elsewhere(name, value):
    if name not in ("cache", "caches"):
        return Elsewhere(value)
    c = B.CacheDesc(*(getattr(value, f) for f, _ in B.CacheDesc._fields_))
    c.device = value.device + 1
    return c


@pytest.mark.parametrize("call", ["rope", "decode", "prefill", "copy"])
@pytest.mark.parametrize("where", ["host", "gpu"])
def test_every_tensor_has_to_be_on_the_current_device(call, where):
    fn, good = arguments()[call]
    fn(**good)
    torch.cuda.synchronize()
    for name, value in good.items():
        if isinstance(value, torch.Tensor):
            bad = value.cpu() if where == "host" else elsewhere(name, value)
        elif isinstance(value, B.CacheDesc):
            if where == "host":
                t = torch.zeros(value.num_blocks, value.num_kv_heads, value.block_size,
                                value.head_dim, dtype=torch.uint8)
                bad = B.cache_desc(t, t)
            else:
                bad = elsewhere(name, value)
        else:
            continue
        what = "the cache" if name in ("cache", "caches") else name
        with pytest.raises(ValueError, match="%s must be on the current CUDA device" % what):
            fn(**dict(good, **{name: bad}))


@pytest.mark.parametrize("name", ["caches", "scales", "dst", "dst_scales", "block_pairs"])
def test_a_pool_of_another_gpu_is_refused(name):
    """Between two pools: host memory may take part, another GPU's not."""
    _, good = arguments()["copy"]
    k = torch.zeros(good["caches"].num_blocks, 2, 16, 64, dtype=torch.uint8, device="cuda")
    good = dict(good, dst=B.cache_desc(k, k.clone()), dst_scales=torch.ones_like(good["scales"]))
    B.pkv_copy_blocks_scaled(**good)
    torch.cuda.synchronize()
    bad = good[name]
    if isinstance(bad, torch.Tensor):
        bad = Elsewhere(bad)
    else:
        bad = elsewhere("cache", bad)
    with pytest.raises(ValueError, match="must be on the current CUDA device"):
        B.pkv_copy_blocks_scaled(**dict(good, **{name: bad}))


@pytest.mark.parametrize("call,name,change,error,match", [
    ("rope", "k", lambda t: t.float(), TypeError, "k must be float16 or bfloat16"),
    ("rope", "k", lambda t: t.bfloat16(), ValueError, "k and v must be alike"),
    ("rope", "k", lambda t: t[:, :1], ValueError, "k and v must be alike"),
    ("rope", "v", lambda t: t[:1], ValueError, "k and v must be alike"),
    ("rope", "v", lambda t: t.transpose(0, 1).contiguous().transpose(0, 1), ValueError,
     "v must be .tokens, heads, head_dim. with dense heads"),
    ("rope", "q", lambda t: t[:1], ValueError, "q must be alike k"),
    ("rope", "q", lambda t: t.bfloat16(), ValueError, "q must be alike k"),
    ("rope", "q", lambda t: t[:, :, ::2], ValueError, "q must be alike k"),
    ("rope", "q", lambda t: t.transpose(0, 1).contiguous().transpose(0, 1), ValueError,
     "q must be .tokens, heads, head_dim. with dense heads"),
    ("rope", "q_out", lambda t: t[:1], ValueError, "q_out must be dense and like q"),
    ("rope", "q_out", lambda t: t.bfloat16(), ValueError, "q_out must be dense and like q"),
    ("rope", "inv_freq", lambda t: t.float(), ValueError, "inv_freq must be contiguous float64"),
    ("rope", "inv_freq", lambda t: t[::2], ValueError, "inv_freq must be contiguous float64"),
    ("rope", "cu_seqlens_q", lambda t: t[:2], ValueError, "cu_seqlens_q needs num_seqs"),
    ("rope", "block_tables", lambda t: t[:1], ValueError, "block_tables num_seqs rows"),
    ("decode", "q", lambda t: t.float(), TypeError, "q must be float16 or bfloat16"),
    ("decode", "q", lambda t: t[:1], ValueError, "do not fit together"),
    ("decode", "q", lambda t: t[:, :, :32], ValueError, "do not fit together"),
    ("decode", "out", lambda t: t[:, :2], ValueError, "out must be dense and like q"),
    ("decode", "block_tables", lambda t: t[:1], ValueError, "do not fit together"),
    ("prefill", "q", lambda t: t.float(), TypeError, "q must be float16 or bfloat16"),
    ("prefill", "q", lambda t: t[:, :, :32], ValueError, "do not fit together"),
    ("prefill", "out", lambda t: t.bfloat16(), ValueError, "out must be dense and like q"),
    ("prefill", "cu_seqlens_q", lambda t: t[:2], ValueError, "do not fit together"),
    ("copy", "block_pairs", lambda t: t.int(), ValueError, "block_pairs must be contiguous int64"),
    ("copy", "scales", lambda t: [t, t], ValueError, "one array of scales per layer"),
] + [(call, "scales", change, ValueError, "scales must be contiguous float32")
     for call in ("rope", "decode", "prefill", "copy")
     for change in (lambda t: t[:3], lambda t: t.half(), lambda t: t.double(), lambda t: t[..., :1])
] + [(call, name, change, ValueError, "%s must be contiguous int32" % name)
     for call in ("rope", "decode", "prefill")
     for name in ("block_tables", "context_lens", "cu_seqlens_q")
     if call != "decode" or name != "cu_seqlens_q"
     for change in (lambda t: t.long(), lambda t: torch.stack([t, t], -1)[..., 0])
] + [(call, "dev_err", lambda t: t.long(), ValueError, "dev_err must be int32")
     for call in ("rope", "decode", "prefill", "copy")])
def test_what_the_binding_refuses(call, name, change, error, match):
    """One argument changed at a time: the refusal is that argument's own."""
    fn, good = arguments()[call]
    fn(**good)
    torch.cuda.synchronize()
    args = dict(good)
    if call == "copy" and name == "scales" and match.startswith("one array"):
        args["caches"] = [args["caches"]]
    args[name] = change(args[name])
    if name == "k" and match.startswith("k must"):
        args["v"] = args["v"].float()
    if name in ("q",) and "out" in args:
        args["out"] = None
    with pytest.raises(error, match=match):
        fn(**args)


def test_more_sequences_than_a_grid_has_rows():
    """70,000 sequences: a prompt of one token each, appended and prefilled, and
    decoded; each attends to itself alone, so its output is its stored V."""
    n, kv, bs, d = 70000, 1, 8, 64
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(n, 4, d, generator=g, device="cuda").half()
    q, k, v = x[:, :2], x[:, 2:3], x[:, 3:]
    codes = [torch.full((n, kv, bs, d), 0xff, dtype=torch.uint8, device="cuda") for _ in range(2)]
    sc = torch.full((n, kv, 2), float("nan"), device="cuda")
    desc = B.cache_desc(*codes)
    tables = torch.randperm(n, generator=g, device="cuda").int()[:, None].contiguous()
    ctx = torch.ones(n, dtype=torch.int32, device="cuda")
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    qr = B.pkv_rope_append(desc, q, k, v, None, cu, 1, tables, ctx, 1, scales=sc, dev_err=err)
    pre = B.pkv_paged_attention_prefill_scaled(desc, sc, qr, cu, 1, tables, ctx, 1, 0.125, dev_err=err)
    dec = B.pkv_paged_attention_decode_scaled(desc, sc, qr, tables, ctx, 1, 0.125, dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.equal(qr, q)
    ids = tables[:, 0].long()
    stored = codes[1][ids, 0, 0].view(torch.float8_e4m3fn).double() * sc[ids, 0, 1:].double()
    # half an E4M3 step of the value, or half a subnormal step
    off = (stored - v[:, 0].double()).abs()
    assert (off <= torch.maximum(2.0 ** -4 * v[:, 0].double().abs(), 2.0 ** -10 * sc[ids, 0, 1:].double())).all()
    assert (codes[1][:, :, 1:] == 0xff).all()
    # a single weight of 1 (over a sum of 1): the value itself, in fp16
    for out in (pre, dec):
        assert torch.equal(out[:, 0], stored.half()) and torch.equal(out[:, 1], stored.half())


def test_copy_of_more_pairs_and_layers_than_one_launch_takes():
    n, layers = 66000, 65
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randint(0, 256, (2 * n, 1, 8, 64), dtype=torch.uint8, device="cuda", generator=g)
    v, s = k.flip(0), torch.rand(2 * n, 1, 2, device="cuda", generator=g)
    order = torch.randperm(2 * n, device="cuda", generator=g)
    pairs = order.view(2, n).t().contiguous()
    B.pkv_copy_blocks_scaled(B.cache_desc(k, v), s, pairs)
    for t in (k, v, s):
        assert torch.equal(t[pairs[:, 1]], t[pairs[:, 0]])
    ks = torch.randint(0, 256, (layers, 6, 1, 8, 64), dtype=torch.uint8, device="cuda", generator=g)
    vs, ss = ks.flip(0), torch.rand(layers, 6, 1, 2, device="cuda", generator=g)
    before = [t.clone() for t in (ks, vs, ss)]
    B.pkv_copy_blocks_scaled([B.cache_desc(a, b) for a, b in zip(ks, vs)], list(ss),
                             torch.tensor([[1, 4], [2, 5]], device="cuda"))
    for t, u in zip((ks, vs, ss), before):
        u[:, 4:] = u[:, 1:3].clone()
        assert torch.equal(t, u)


@pytest.mark.parametrize("kv,heads,d,bs,cached,partition", [
    (8, 8, 64, 16, 20, 0), (8, 64, 128, 16, 1300, 0), (32, 32, 128, 32, 40, 0), (4, 16, 64, 32, 600, 64)])
def test_decode_right_behind_an_append_that_raises_scales(kv, heads, d, bs, cached, partition):
    """The decode starts while the append before it ends: it has to see the raised
    scales and re-rounded codes that other SMs wrote.  Every new token is twice the
    one before, so every append but a block's first rewrites whole blocks."""
    n, steps = 48, 40
    g = torch.Generator(device="cuda").manual_seed(kv)
    width = -(-(cached + steps) // bs)
    nb = n * width
    codes = [torch.randint(0, 0x60, (nb, kv, bs, d), dtype=torch.uint8, device="cuda", generator=g)
             for _ in range(2)]
    sc = torch.full((nb, kv, 2), 2.0 ** -12, device="cuda")
    desc = B.cache_desc(*codes)
    tables = torch.randperm(nb, device="cuda", generator=g).int().view(n, width).contiguous()
    f = torch.from_numpy(freqs(d)).cuda()
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    ctx = torch.empty(n, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(1, B.pkv_decode_scaled_workspace_bytes(desc, n, heads, cached + steps, partition)),
                     dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = torch.randn(n, heads + 2 * kv, d, device="cuda", generator=g)
    qkv = x.bfloat16()
    out = torch.empty(n, heads, d, dtype=torch.bfloat16, device="cuda")
    args = (tables, ctx, cached + steps, d ** -0.5, partition)

    def step():
        qr = B.pkv_rope_append(desc, qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:], f,
                               cu, 1, tables, ctx, cached + steps, scales=sc, dev_err=err)
        B.pkv_paged_attention_decode_scaled(desc, sc, qr, *args, workspace=ws, out=out)
        return qr

    ctx.fill_(cached + 1)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qr = step()
    for i in range(steps):
        ctx.fill_(cached + i + 1)
        qkv[:, heads:] = (x[:, heads:] * 2.0 ** (i % bs - 8)).bfloat16()
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()                              # the two launches side by side
        torch.cuda.synchronize()
        again = B.pkv_paged_attention_decode_scaled(desc, sc, qr, *args, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), again.view(torch.int16)), i
    assert int(err.item()) == 0 and not out.isnan().any()
