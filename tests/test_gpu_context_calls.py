"""How the calls that share, weigh and evict treat what surrounds them: streams,
memory they allocate, graphs, arguments they refuse; and their less common
paths."""
import numpy as np
import pytest
import torch

import harness as H
from oracle import context as OC
from paged_kv_cache_130_gb300 import binding as B
from paged_kv_cache_130_gb300 import workloads as W
from test_gpu_context import Evicted, Keys, filled, run_weights, weights_close
from test_gpu_scaled import Batch, freqs
from test_gpu_scaled_calls import Elsewhere, elsewhere, pool_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    H.build_library()


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def arguments(longest=1500):
    """name of a call -> (function, arguments that it takes without complaint)"""
    b = filled(400, W.F16, 4, 2, 64, 16, [longest, 40, 700])
    b.desc.caches = b.gk, b.gv                # (a descriptor keeps no reference itself)
    q = b.dev16(b.q)
    common = dict(cache=b.desc, block_tables=b.gt, context_lens=b.gctx, max_context_len=b.max_ctx,
                  dev_err=b.err, scales=b.gs)
    attend = dict(common, q=q, scale=0.125)
    w = torch.rand(3, 2, b.max_ctx, device="cuda")

    def ws(n):
        return torch.empty(n, dtype=torch.uint8, device="cuda")

    free = torch.arange(b.nb, dtype=torch.int32, device="cuda")
    used = torch.cat([b.gt[i, :-(-int(c) // 16)] for i, c in enumerate(b.ctx)])
    free = free[~torch.isin(free, used)][:3].view(3, 1).contiguous()
    return dict(
        shared=(B.pkv_paged_attention_decode_scaled_shared_prefix,
                dict(attend, group_begin=i32(0, 1, 3), group_prefix_blocks=i32(0, 0),
                     max_group_size=2, max_prefix_blocks=2, out=torch.empty_like(q),
                     workspace=ws(B.pkv_decode_scaled_shared_prefix_workspace_bytes(
                         b.desc, 3, 4, 2, 2, b.max_ctx)))),
        weights=(B.pkv_attention_weights,
                 dict(attend, cu_seqlens_q=b.gcu, window=1, weights=w,
                      workspace=ws(B.pkv_attention_weights_workspace_bytes(b.desc, 3, 4, 1, b.max_ctx)))),
        decode=(B.pkv_paged_attention_decode_scaled_weights,
                dict(attend, weights=w, out=torch.empty_like(q),
                     workspace=ws(B.pkv_decode_scaled_weights_workspace_bytes(b.desc, 3, 4, b.max_ctx)))),
        evict=(B.pkv_evict,
               dict(common, weights=w, keep_lens=i32(16, 10, 3), max_keep_len=16, keep_first=1,
                    keep_last=2, dst_tables=free, weights_out=torch.empty_like(w),
                    lens_out=torch.empty_like(b.gctx),
                    workspace=ws(B.pkv_evict_workspace_bytes(b.desc, 3, 16, b.max_ctx)))))


CALLS = ["shared", "weights", "decode", "evict"]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("where", ["host", "gpu"])
def test_every_tensor_has_to_be_on_the_current_device(call, where):
    fn, good = arguments()[call]
    fn(**good)
    torch.cuda.synchronize()
    assert int(good["dev_err"].item()) == 0
    for name, value in good.items():
        if isinstance(value, torch.Tensor):
            bad = value.cpu() if where == "host" else Elsewhere(value)
        elif isinstance(value, B.CacheDesc):
            if where == "host":
                t = torch.zeros(value.num_blocks, 2, 16, 64, dtype=torch.uint8)
                bad = B.cache_desc(t, t)
            else:
                bad = elsewhere(name, value)
        else:
            continue
        what = "the cache" if name == "cache" else name
        with pytest.raises(ValueError, match="%s must be on the current CUDA device" % what):
            fn(**dict(good, **{name: bad}))


@pytest.mark.parametrize("call,name,change,error,match", [
    (call, "q", lambda t: t.float(), TypeError, "q must be float16 or bfloat16")
    for call in CALLS[:3]
] + [(call, "q", lambda t: t[:, :, :32], ValueError, "do not fit together") for call in CALLS[:3]
] + [(call, "out", lambda t: t[:, :2], ValueError, "out must be dense and like q") for call in ("shared", "decode")
] + [(call, "block_tables", lambda t: t[:1], ValueError, "do not fit together") for call in CALLS
] + [(call, name, lambda t: t.long(), ValueError, "%s must be contiguous int32" % name)
     for call, names in (("shared", ("block_tables", "context_lens", "group_begin", "group_prefix_blocks")),
                         ("weights", ("block_tables", "context_lens", "cu_seqlens_q")),
                         ("decode", ("block_tables", "context_lens")),
                         ("evict", ("block_tables", "context_lens", "keep_lens", "dst_tables", "lens_out")))
     for name in names
] + [(call, "scales", lambda t: t[:3], ValueError, "scales must be contiguous float32") for call in CALLS
] + [(call, "dev_err", lambda t: t.long(), ValueError, "dev_err must be int32") for call in CALLS
] + [(call, "weights", change, ValueError, "weights must be")
     for call in ("weights", "decode", "evict")
     for change in (lambda t: t.double(), lambda t: t[:2], lambda t: t[:, :1], lambda t: t[..., :-1],
                    lambda t: t.transpose(1, 2).contiguous().transpose(1, 2), lambda t: t[0])
] + [("evict", "weights_out", lambda t: t[:2], ValueError, "weights_out must be"),
     ("evict", "weights_out", lambda t: t[..., :15], ValueError, "weights_out must be"),
     ("evict", "lens_out", lambda t: t[:2], ValueError, "lens_out needs num_seqs"),
     ("evict", "keep_lens", lambda t: t[:2], ValueError, "do not fit together"),
     ("evict", "dst_tables", lambda t: t[:2], ValueError, "do not fit together"),
     ("shared", "group_begin", lambda t: t[:2], ValueError, "group_begin needs num_groups"),
     ("weights", "cu_seqlens_q", lambda t: t[:3], ValueError, "do not fit together"),
     ("weights", "weights", lambda t: t[:1].expand(3, 2, t.shape[2]), B.PkvError, "invalid"),
     ("evict", "workspace", lambda t: t[:100], B.PkvError, "workspace"),
     ("decode", "workspace", lambda t: t[256:], B.PkvError, "workspace"),
     ("shared", "workspace", lambda t: t[:256], B.PkvError, "workspace"),
     ("weights", "workspace", lambda t: t[16:], B.PkvError, "workspace")])
def test_what_the_binding_refuses(call, name, change, error, match):
    """One argument changed at a time: the refusal is that argument's own."""
    fn, good = arguments(200)[call]
    args = dict(good, **{name: change(good[name])})
    if name == "q" and "out" in args:
        args["out"] = None
    with pytest.raises(error, match=match):
        fn(**args)


def test_evict_refuses_its_input_as_its_output():
    fn, good = arguments(200)["evict"]
    with pytest.raises(ValueError, match="weights_out must not be weights"):
        fn(**dict(good, weights_out=good["weights"]))
    with pytest.raises(B.PkvError, match="invalid"):
        fn(**dict(good, weights_out=good["weights"][:]))


def test_evict_refuses_lengths_that_it_reads_as_its_output():
    fn, good = arguments(200)["evict"]
    for name in ("context_lens", "keep_lens"):
        with pytest.raises(ValueError, match="lens_out must not be"):
            fn(**dict(good, lens_out=good[name]))
        with pytest.raises(B.PkvError, match="invalid"):
            fn(**dict(good, lens_out=good[name][:]))


def test_position_offsets_are_checked():
    b = Batch(401, W.F16, 4, 2, 64, 16, [2, 1], [3, 0])
    for bad in (i32(1), torch.zeros(2, dtype=torch.int64, device="cuda"), torch.zeros(2, dtype=torch.int32)):
        with pytest.raises(ValueError, match="position_offsets"):
            b.append(freqs(64), position_offsets=bad)


@pytest.mark.parametrize("as_number", [False, True])
def test_what_a_call_on_another_stream_allocates_is_that_streams(as_number, monkeypatch):
    side = torch.cuda.Stream()
    calls = arguments()
    torch.cuda.synchronize()
    made = []
    empty, like = torch.empty, torch.empty_like
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made.append(empty(*a, **k)) or made[-1])
    monkeypatch.setattr(torch, "empty_like", lambda *a, **k: made.append(like(*a, **k)) or made[-1])
    for call, (fn, good) in calls.items():
        args = dict(good, stream=side.cuda_stream if as_number else side)
        for name in ("out", "workspace", "weights_out", "lens_out"):
            args.pop(name, None)
        made.clear()
        fn(**args)
        assert made and all(pool_of(t.data_ptr()) == side.cuda_stream for t in made), call
        torch.cuda.synchronize()
        assert int(good["dev_err"].item()) == 0


@pytest.mark.parametrize("longest", [900, 1500])
def test_calls_in_captured_graphs_that_share_a_workspace(longest):
    """Each call captured twice over one workspace, the graphs replayed in turn: what
    one leaves there does not reach the other; totals grow by the same each time."""
    for call, (fn, good) in arguments(longest).items():
        others = dict(good)
        if "q" in good:
            others["q"] = torch.randn_like(good["q"])
        if "out" in good:
            others["out"] = torch.empty_like(good["out"])
        if call == "evict":
            others["weights"] = torch.rand_like(good["weights"])
            others["weights_out"] = torch.empty_like(good["weights"])
            others["lens_out"] = torch.empty_like(good["lens_out"])
        if call in ("weights", "decode"):
            good["weights"].zero_()
            others["weights"] = torch.zeros_like(good["weights"])

        def results(a):
            return [a[n].clone() for n in ("out", "weights", "weights_out", "lens_out") if n in a]

        def reset():
            for a in (good, others):
                if call in ("weights", "decode"):
                    a["weights"].zero_()

        want = []
        for a in (good, others):
            fn(**a)
            want.append(results(a))
        torch.cuda.synchronize()
        graphs = []
        for a in (good, others):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                fn(**a)
            graphs.append(g)
        for _ in range(2):
            reset()
            for g in graphs:
                g.replay()
            torch.cuda.synchronize()
            for a, x in zip((good, others), want):
                for y, z in zip(results(a), x):
                    assert torch.equal(y, z), call
        assert int(good["dev_err"].item()) == 0


def test_weights_of_more_sequences_than_a_launch_takes():
    """1,100 sequences, one of them long."""
    ctx = np.random.default_rng(2).integers(1, 9, 1100)
    ctx[600] = 700
    b = filled(410, W.BF16, 2, 1, 64, 8, ctx)
    b.gctx[1090] = 0                                     # (fewer tokens than rows)
    w = torch.zeros(1100, 1, b.max_ctx, device="cuda")
    run_weights(b, 0.125, 1, w, scales=b.gs)
    assert int(b.err.item()) == B.PKV_DEVERR_CONTEXT
    add, size = OC.weights(Keys(b), b.q, b.cu, 1, b.ctx, 0.125)
    add[1090] = 0
    weights_close(w, 0.0, add, size, "many")


@pytest.mark.parametrize("spread", [6, 30])
def test_weights_of_rows_of_very_different_size(spread):
    """bf16 rows over E4M3 codes become fp16 times a power of two: of all rows where
    they are alike, of each row (2^-30 and zero among them) where they are not."""
    b = Batch(411, W.BF16, 4, 2, 128, 16, [40], [300])
    b.append()
    b.oracle_append()
    e = np.random.default_rng(3).integers(-spread, 1, b.q.shape[:2])
    b.q = b.q * 2.0 ** e[..., None]
    b.q[-3] = 0.0
    b.q[-1, 0, 5] = 2.0 ** 12
    w = torch.zeros(1, 2, b.max_ctx, device="cuda")
    run_weights(b, 0.09, 40, w, scales=b.gs)
    add, size = OC.weights(Keys(b), b.q, b.cu, 40, b.ctx, 0.09)
    weights_close(w, 0.0, add, size, "rows")
    assert int(b.err.item()) == 0


@pytest.mark.parametrize("heads", [1, 16])
def test_weights_whose_scores_leave_any_reference_behind(heads):
    """The first key of every tile scores far below the others, by far more than the
    sum's range; and the row's largest comes last."""
    b = Batch(412, W.F16, heads, 1, 64, 16, [20], [500], spread=0.0)
    b.nv[:] = b.nk[:] = 0
    b.append()
    b.oracle_append()
    one = np.zeros((heads, 64))
    one[:, 0] = 1.0
    b.q[:] = one
    codes = b.k
    codes[:] = 0
    scales = np.ones_like(b.scales)
    for t in range(520):
        # scores from -448 to 448, the lowest where a tile starts
        code = 0xfe if t % 128 == 0 else (0x7e if t == 519 else 0x30 + t % 16)
        codes[b.tables[0, t // 16], 0, t % 16, 0] = code
    b.scales = scales.astype(np.float32)
    b.gk.copy_(torch.from_numpy(codes))
    b.gs.copy_(torch.from_numpy(b.scales))
    w = torch.zeros(1, 1, b.max_ctx, device="cuda")
    run_weights(b, 1.0, 20, w, scales=b.gs)
    add, size = OC.weights(Keys(b), b.q, b.cu, 20, b.ctx, 1.0)
    assert size >= 448
    weights_close(w, 0.0, add, size, "references")
    assert int(b.err.item()) == 0


def test_evict_of_a_row_over_eight_blocks_of_a_cluster():
    e = Evicted(420, "e4m3", 64, 16, 2, [20000, 17], [3000, 5], 4, 64)
    e.check(*e.run())
    assert int(e.err.item()) == 0


def test_evict_of_many_sequences():
    r = np.random.default_rng(5)
    e = Evicted(421, torch.float16, 64, 8, 1, r.integers(0, 60, 700), r.integers(0, 40, 700), 2, 3)
    e.check(*e.run())
    assert int(e.err.item()) == 0


def test_evict_of_empty_contexts():
    """No context has a token: lengths of zero, rows of zeros, or no rows at all."""
    e = Evicted(422, "scaled", 64, 16, 2, [0, 0], [5, 0], 1, 1)
    lens, out = e.run()
    assert lens.tolist() == [0, 0] and not out.any() and int(e.err.item()) == 0
    none = torch.zeros(2, 2, 0, device="cuda")
    lens, out = B.pkv_evict(B.cache_desc(e.gk, e.gv), e.dev(e.tables), e.dev(e.ctx), 0, none,
                            e.dev(e.keep), 5, 1, 1, e.dev(e.dst), scales=e.gs, dev_err=e.err)
    torch.cuda.synchronize()
    assert lens.tolist() == [0, 0] and out.shape == (2, 2, 0) and int(e.err.item()) == 0
