"""Host-side refusals of the scaled-cache calls and the rotary append: every call
here fails a check before any launch, so no pointer is dereferenced."""
import ctypes

import pytest
import torch

from paged_kv_cache_130_gb300 import binding as B
from paged_kv_cache_130_gb300 import build as pkv_build

INVALID, UNSUPPORTED, WORKSPACE = B.PKV_ERR_INVALID_ARG, B.PKV_ERR_UNSUPPORTED, B.PKV_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return B.load()


def _desc(**kw):
    d = dict(k_cache=0x10000, v_cache=0x20000, num_blocks=64, num_kv_heads=8, block_size=16,
             head_dim=128, cache_dtype=B.PKV_FP8_E4M3, k_scale=0.0, v_scale=0.0)
    d.update(kw)
    return B.CacheDesc(**d)


ROPE = dict(scales=0x1000, q=0x2000, qs=8192, k=0x3000, ks=1024, v=0x4000, vs=1024,
            dtype=B.PKV_BF16, heads=64, inv=0x5000, rot=128, inter=0, m=1.0, seqs=2, cu=0x6000,
            total=4, maxq=2, bt=0x7000, mb=8, ctx=0x8000, maxc=100, err=None, out=0x9000,
            stream=None)


@pytest.mark.parametrize("desc,kw,want", [
    (dict(head_dim=96), {}, UNSUPPORTED),
    (dict(block_size=64), {}, UNSUPPORTED),
    (dict(cache_dtype=B.PKV_BF16), {}, UNSUPPORTED),          # scales beside a 16-bit cache
    (dict(cache_dtype=7), {}, INVALID),
    (dict(), dict(scales=None), INVALID),                      # one scale, but it is 0
    (dict(cache_dtype=B.PKV_F16), dict(scales=None), UNSUPPORTED),   # bf16 into fp16
    (dict(), dict(scales=0x1004), INVALID),
    (dict(), dict(rot=24), UNSUPPORTED),
    (dict(), dict(rot=144), INVALID),
    (dict(), dict(rot=-16), INVALID),
    (dict(), dict(m=float("nan")), INVALID),
    (dict(), dict(m=float("inf")), INVALID),
    (dict(), dict(inv=None), INVALID),
    (dict(), dict(inv=0x5004), INVALID),
    (dict(), dict(ks=1020), INVALID),
    (dict(), dict(ks=1028), INVALID),
    (dict(), dict(qs=8184), INVALID),
    (dict(), dict(q=0x2008), INVALID),
    (dict(), dict(v=0x4004), INVALID),
    (dict(), dict(out=None), INVALID),
    (dict(), dict(dtype=B.PKV_FP8_E4M3), INVALID),
    (dict(), dict(cu=None), INVALID),
    (dict(), dict(bt=None), INVALID),
    (dict(), dict(ctx=None), INVALID),
    (dict(), dict(mb=0), INVALID),
    (dict(), dict(mb=1 << 30), INVALID),
    (dict(), dict(maxc=(1 << 31) - 1), INVALID),
    (dict(), dict(total=-1), INVALID),
    (dict(), dict(heads=0), INVALID),
    (dict(), dict(seqs=0), B.PKV_OK),
    (dict(), dict(total=0), B.PKV_OK),
])
def test_rope_append_checks(lib, desc, kw, want):
    a = dict(ROPE, **kw)
    assert lib.pkv_rope_append(ctypes.byref(_desc(**desc)), *a.values()) == want


DECODE = dict(scales=0x1000, q=0x2000, dtype=B.PKV_BF16, seqs=4, heads=64, bt=0x3000, mb=64,
              ctx=0x4000, maxc=1000, scale=0.1, part=64, ws=0x10000, ws_bytes=1 << 30, err=None,
              out=0x5000, stream=None)


@pytest.mark.parametrize("desc,kw,want", [
    (dict(cache_dtype=B.PKV_F16), {}, UNSUPPORTED),
    (dict(head_dim=256), {}, UNSUPPORTED),
    (dict(num_kv_heads=7), {}, INVALID),
    (dict(num_kv_heads=2), {}, UNSUPPORTED),                  # 32 heads per KV head
    (dict(), dict(scales=None), INVALID),
    (dict(), dict(q=None), INVALID),
    (dict(), dict(out=0x5002), INVALID),
    (dict(), dict(part=24), INVALID),
    (dict(block_size=8), dict(part=24), INVALID),
    (dict(block_size=32), dict(part=48), INVALID),
    (dict(), dict(part=-16), INVALID),
    (dict(), dict(ws=None), WORKSPACE),
    (dict(), dict(ws=0x10010), WORKSPACE),
    (dict(), dict(ws_bytes=1024), WORKSPACE),
    (dict(), dict(bt=None), INVALID),
    (dict(), dict(maxc=-1), INVALID),
    (dict(), dict(dtype=9), INVALID),
    (dict(), dict(seqs=0), B.PKV_OK),
])
def test_decode_scaled_checks(lib, desc, kw, want):
    a = dict(DECODE, **kw)
    assert lib.pkv_paged_attention_decode_scaled(ctypes.byref(_desc(**desc)), *a.values()) == want


PREFILL = dict(scales=0x1000, q=0x2000, dtype=B.PKV_BF16, seqs=2, heads=64, cu=0x3000, total=10,
               maxq=6, bt=0x4000, mb=64, ctx=0x5000, maxc=1000, scale=0.1, err=None, out=0x6000,
               stream=None)


@pytest.mark.parametrize("desc,kw,want", [
    (dict(cache_dtype=B.PKV_BF16), {}, UNSUPPORTED),
    (dict(block_size=12), {}, UNSUPPORTED),
    (dict(num_kv_heads=6), {}, INVALID),
    (dict(num_kv_heads=1), dict(heads=129), UNSUPPORTED),
    (dict(), dict(scales=None), INVALID),
    (dict(), dict(q=0x2004), INVALID),
    (dict(), dict(cu=None), INVALID),
    (dict(), dict(mb=0), INVALID),
    (dict(), dict(maxc=(1 << 31) - 1), INVALID),
    (dict(), dict(total=-1), INVALID),
    (dict(), dict(total=0), B.PKV_OK),
    (dict(), dict(maxq=0), B.PKV_OK),
])
def test_prefill_scaled_checks(lib, desc, kw, want):
    a = dict(PREFILL, **kw)
    assert lib.pkv_paged_attention_prefill_scaled(ctypes.byref(_desc(**desc)), *a.values()) == want


def test_workspace_follows_the_partition(lib):
    d = _desc()
    assert B.pkv_decode_scaled_workspace_bytes(d, 4, 64, 1000, 1008) == 0
    ml = -(-4 * 4 * 64 * 16 // 256) * 256
    assert B.pkv_decode_scaled_workspace_bytes(d, 4, 64, 1000, 64) == 2 * ml + 4 * 4 * 64 * 16 * 128
    # the library's choice: one partition, without a workspace, for contexts up
    # to 1,024 tokens; equal shares beyond, with a workspace that the batch does
    # not change
    assert B.pkv_decode_scaled_partition_size(d, 4, 64, 500) == 512
    assert B.pkv_decode_scaled_workspace_bytes(d, 4, 64, 500) == 0
    assert B.pkv_decode_scaled_partition_size(d, 900, 64, 1024) == 1024
    assert B.pkv_decode_scaled_partition_size(d, 4, 64, 1025) == 0
    n = B.pkv_decode_scaled_workspace_bytes(d, 4, 64, 2000)
    assert n > 0 and n == B.pkv_decode_scaled_workspace_bytes(d, 900, 64, 100000)
    p = B.pkv_decode_scaled_partition_size(d, 2000, 64, 100000)
    assert p > 0 and p % 32 == 0
    assert B.pkv_decode_scaled_workspace_bytes(d, 0, 64, 1000) == 0


def _copy(lib, src, ss, dst=None, ds=None, layers=1, pairs=0x1000, n=1):
    ptr = ctypes.c_void_p * layers
    return lib.pkv_copy_blocks_scaled(ctypes.byref(src), ptr(*[ss] * layers),
                                      ctypes.byref(dst) if dst else None,
                                      ptr(*[ds] * layers) if ds else None, layers, pairs, n, None,
                                      None)


def test_copy_scaled_checks(lib):
    assert _copy(lib, _desc(cache_dtype=B.PKV_F16), 0x1000) == UNSUPPORTED
    assert _copy(lib, _desc(), None) == INVALID
    assert _copy(lib, _desc(), 0x1004) == INVALID
    assert _copy(lib, _desc(), 0x1000, _desc()) == INVALID           # dst without its scales
    assert _copy(lib, _desc(), 0x1000, _desc(block_size=32), 0x2000) == INVALID
    assert _copy(lib, _desc(), 0x1000, pairs=None) == INVALID
    assert _copy(lib, _desc(), 0x1000, n=-1) == INVALID
    assert _copy(lib, _desc(), 0x1000, n=0) == B.PKV_OK


def test_binding_checks():
    """Shapes and types that the binding refuses before it calls the library."""
    d = _desc(num_blocks=4, num_kv_heads=2, head_dim=64)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    t = torch.zeros(1, 4, dtype=torch.int32)
    c = torch.zeros(1, dtype=torch.int32)
    s = torch.zeros(4, 2, 2)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    f = torch.zeros(32, dtype=torch.float64)
    good = dict(q=q, k=k, v=k, inv_freq=f, cu_seqlens_q=i, max_q_len=3, block_tables=t,
                context_lens=c, max_context_len=3, scales=s)
    for bad in (dict(k=k.half()), dict(v=k[:2]), dict(q=q.transpose(0, 1)), dict(q=q[:, :, ::2]),
                dict(inv_freq=f.float()), dict(cu_seqlens_q=i[:1]), dict(scales=s[:3]),
                dict(scales=s.half()), dict(block_tables=t.long()), dict(q_out=q[:2]),
                dict(k=torch.zeros(3, 1, 64, dtype=torch.bfloat16))):
        with pytest.raises((ValueError, TypeError)):
            B.pkv_rope_append(d, **dict(good, **bad))
    with pytest.raises(ValueError):
        B.pkv_paged_attention_decode_scaled(d, s, q, t, c, 3, 0.1)
    with pytest.raises(ValueError):
        B.pkv_copy_blocks_scaled([d, d], [s], torch.zeros(1, 2, dtype=torch.int64))


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -float("inf")])
def test_attention_scale_has_to_be_finite(lib, scale):
    """The prefill would answer a NaN with numbers."""
    a = dict(DECODE, scale=scale)
    assert lib.pkv_paged_attention_decode_scaled(ctypes.byref(_desc()), *a.values()) == INVALID
    a = dict(PREFILL, scale=scale)
    assert lib.pkv_paged_attention_prefill_scaled(ctypes.byref(_desc()), *a.values()) == INVALID
