"""The calls that share, weigh and evict at the edges of what they allow: waits that
run out, infinities and NaN in 16-bit caches, blocks that cannot be used, rows of
very different size, lengths whose products pass 32 bits.  Bounds as in
test_gpu_context."""
import numpy as np
import pytest
import torch

import harness as H
from oracle import context as OC
from paged_kv_cache_130_gb300 import binding as B
from paged_kv_cache_130_gb300 import workloads as W
from test_gpu_context import Keys, run_weights, weights_close
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
