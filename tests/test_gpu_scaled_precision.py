"""The scaled-cache calls where precision is lost first, against the 64-bit
oracle.

Bounds, from the arithmetic (eps = 2^-11, half a step of fp16):
* a weight times its block's scale is rounded to fp16: eps of itself, or half of
  the subnormal step, which is 2^-31 of the largest weight in the prefill (the
  weights are held times 2^6) and 2^-30 of the largest weight times the largest
  scale in the decode (times at least 2^5); so the sum over N tokens is off by
  eps sum p |v| + N 2^-30 max |v| at most;
* an fp32 sum of products, the exponential and the final division: 2^-18 of
  sum p |v|, and of the scores, which are below 2^5 here: another 2^-18;
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


def assert_within(got, b, scale, what):
    """got against the oracle's attention, each output to the bound above."""
    ref, absum, vmax = attention_and_sizes(b, scale)
    n = float(b.ctx.max())
    half = torch.finfo(TD[b.dt]).eps / 2
    err = (EPS + 2.0 ** -17) * absum + n * 2.0 ** -30 * vmax
    bound = err + half * (np.abs(ref) + err) + (2.0 ** -25 if b.dt == W.F16 else 0.0)
    got = H.out_to_double(got)
    ratio = np.abs(got - ref) / np.maximum(bound, 1e-300)
    ratio = np.where((got == ref), 0.0, ratio)
    assert (ratio <= 1).all(), (what, float(ratio.max()), np.abs(got - ref).max())


def attention_and_sizes(b, scale):
    """(attention, sum of p |v|, largest |v| of the context) per output."""
    ref = b.attention(scale)
    v, vmax = b.v, np.zeros(ref.shape)
    b.v = v & 0x7f
    absum = b.attention(scale)
    b.v = v
    G = b.heads // b.kv
    for s, c in enumerate(b.ctx):
        for h in range(b.kv):
            if c:
                x = np.abs(OS.gather(v, b.scales, 1, b.tables[s], int(c), h)).max()
                vmax[b.cu[s]:b.cu[s + 1], h * G:(h + 1) * G] = x
    return ref, absum, vmax


@pytest.mark.parametrize("dt,bs,n", [(W.F16, 16, 32768), (W.BF16, 32, 131072)])
def test_faint_weights_behind_one_large_one(dt, bs, n):
    """One key 17.5 nats above all others, whose V is 0: what the others bring
    is the output, and grows with the context."""
    b = Batch(200, dt, 2, 1, 64, bs, [1], [0])
    b.nb = n // bs
    b.tables = b.r.permutation(b.nb).astype(np.int32)[None]
    shape = (b.nb, 1, bs, 64)
    b.k, b.v = np.zeros(shape, np.uint8), np.full(shape, 0x7e, np.uint8)      # 0 and 448
    b.scales = np.ones((b.nb, 1, 2), np.float32)
    first = b.tables[0, 0]
    b.k[first, 0, 5, 0] = 0x38                                               # 1
    b.v[first, 0, 5] = 0
    b.q[...] = 0
    b.q[..., 0] = 1
    b.ctx = np.array([n], np.int32)
    b.upload()
    assert 0.3 < b.attention(17.5).max() < 2
    assert_within(b.prefill(17.5), b, 17.5, "prefill")
    assert_within(b.decode(17.5), b, 17.5, "decode")
    assert int(b.err.item()) == 0
