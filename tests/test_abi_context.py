"""Host-side refusals of the calls that share, weigh and evict: every call here
fails a check before any launch (or has nothing to do), so no pointer is
dereferenced."""
import ctypes

import pytest
import torch

from paged_kv_cache_130_gb300 import binding as B
from paged_kv_cache_130_gb300 import build as pkv_build

INVALID, UNSUPPORTED, WORKSPACE = B.PKV_ERR_INVALID_ARG, B.PKV_ERR_UNSUPPORTED, B.PKV_ERR_WORKSPACE
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return B.load()


def _desc(**kw):
    d = dict(k_cache=0x10000, v_cache=0x20000, num_blocks=64, num_kv_heads=8, block_size=16,
             head_dim=128, cache_dtype=B.PKV_FP8_E4M3, k_scale=0.0, v_scale=0.0)
    d.update(kw)
    return B.CacheDesc(**d)


SHARED = dict(scales=0x1000, q=0x2000, dtype=B.PKV_BF16, seqs=4, heads=64, bt=0x3000, mb=64,
              ctx=0x4000, maxc=1000, groups=2, begin=0x6000, prefix=0x7000, size=3, blocks=10,
              scale=0.1, ws=0x100000, ws_bytes=1 << 40, err=None, out=0x5000, stream=None)


@pytest.mark.parametrize("desc,kw,want", [
    (dict(cache_dtype=B.PKV_F16), {}, UNSUPPORTED),
    (dict(head_dim=256), {}, UNSUPPORTED),
    (dict(num_kv_heads=7), {}, INVALID),
    (dict(num_kv_heads=2), {}, UNSUPPORTED),                  # 32 heads per KV head
    (dict(), dict(scales=None), INVALID),
    (dict(), dict(scales=0x1004), INVALID),
    (dict(), dict(q=None), INVALID),
    (dict(), dict(q=0x2008), INVALID),
    (dict(), dict(out=0x5002), INVALID),
    (dict(), dict(bt=None), INVALID),
    (dict(), dict(ctx=None), INVALID),
    (dict(), dict(begin=None), INVALID),
    (dict(), dict(prefix=None), INVALID),
    (dict(), dict(groups=-1), INVALID),
    (dict(), dict(size=-1), INVALID),
    (dict(), dict(size=0), INVALID),
    (dict(), dict(blocks=-1), INVALID),
    (dict(), dict(blocks=65), INVALID),                       # more than a table holds
    (dict(), dict(blocks=63), INVALID),                       # 1,008 tokens of 1,000
    (dict(), dict(maxc=-1), INVALID),
    (dict(), dict(maxc=(1 << 31) - 1), INVALID),
    (dict(), dict(dtype=B.PKV_FP8_E4M3), INVALID),
    (dict(), dict(scale=NAN), INVALID),
    (dict(), dict(scale=-INF), INVALID),
    (dict(), dict(seqs=-1), INVALID),
    (dict(), dict(seqs=2000, groups=49), UNSUPPORTED),        # 2,049 entries
    (dict(), dict(ws=None), WORKSPACE),
    (dict(), dict(ws=0x100010), WORKSPACE),
    (dict(), dict(ws_bytes=1 << 20), WORKSPACE),
    (dict(), dict(seqs=0), B.PKV_OK),
    (dict(), dict(seqs=0, groups=0), B.PKV_OK),
])
def test_shared_prefix_checks(lib, desc, kw, want):
    a = dict(SHARED, **kw)
    fn = lib.pkv_paged_attention_decode_scaled_shared_prefix
    assert fn(ctypes.byref(_desc(**desc)), *a.values()) == want


WEIGHTS = dict(scales=0x1000, q=0x2000, dtype=B.PKV_BF16, seqs=2, heads=64, cu=0x3000, total=10,
               window=6, bt=0x4000, mb=64, ctx=0x5000, maxc=1000, scale=0.1, w=0x8000, seq=8000,
               head=1000, ws=0x100000, ws_bytes=1 << 40, err=None, stream=None)


@pytest.mark.parametrize("desc,kw,want", [
    (dict(cache_dtype=B.PKV_BF16), {}, UNSUPPORTED),          # scales beside a 16-bit cache
    (dict(cache_dtype=B.PKV_F16), dict(scales=None), UNSUPPORTED),   # bf16 rows over fp16
    (dict(), dict(scales=None), INVALID),                     # one scale, but it is 0
    (dict(k_scale=3e38, v_scale=1.0), dict(scales=None, scale=4.0), INVALID),   # their product
    (dict(block_size=12), {}, UNSUPPORTED),
    (dict(num_kv_heads=6), {}, INVALID),
    (dict(num_kv_heads=1), dict(heads=129), UNSUPPORTED),
    (dict(), dict(scales=0x1002), INVALID),
    (dict(), dict(q=0x2004), INVALID),
    (dict(), dict(q=None), INVALID),
    (dict(), dict(cu=None), INVALID),
    (dict(), dict(bt=None), INVALID),
    (dict(), dict(mb=0), INVALID),
    (dict(), dict(ctx=None), INVALID),
    (dict(), dict(window=-1), INVALID),
    (dict(), dict(total=-1), INVALID),
    (dict(), dict(w=None), INVALID),
    (dict(), dict(w=0x8002), INVALID),
    (dict(), dict(head=999), INVALID),                        # rows that overlap
    (dict(), dict(seq=7999), INVALID),
    (dict(), dict(seq=0), INVALID),
    (dict(), dict(head=-1000), INVALID),
    (dict(), dict(scale=NAN), INVALID),
    (dict(), dict(scale=INF), INVALID),
    (dict(), dict(maxc=(1 << 31) - 1), INVALID),
    (dict(), dict(dtype=5), INVALID),
    (dict(), dict(ws=None), WORKSPACE),
    (dict(), dict(ws=0x100080), WORKSPACE),
    (dict(), dict(ws_bytes=1000), WORKSPACE),
    (dict(), dict(seqs=0), B.PKV_OK),
    (dict(), dict(total=0), B.PKV_OK),
    (dict(), dict(window=0), B.PKV_OK),
])
def test_attention_weights_checks(lib, desc, kw, want):
    a = dict(WEIGHTS, **kw)
    assert lib.pkv_attention_weights(ctypes.byref(_desc(**desc)), *a.values()) == want


DECODE = dict(scales=0x1000, q=0x2000, dtype=B.PKV_BF16, seqs=4, heads=64, bt=0x3000, mb=64,
              ctx=0x4000, maxc=1000, scale=0.1, w=0x8000, seq=8000, head=1000, ws=0x100000,
              ws_bytes=1 << 40, err=None, out=0x5000, stream=None)


@pytest.mark.parametrize("desc,kw,want", [
    (dict(cache_dtype=B.PKV_F16), {}, UNSUPPORTED),
    (dict(head_dim=96), {}, UNSUPPORTED),
    (dict(num_kv_heads=2), {}, UNSUPPORTED),
    (dict(num_kv_heads=7), {}, INVALID),
    (dict(), dict(scales=None), INVALID),
    (dict(), dict(q=None), INVALID),
    (dict(), dict(out=None), INVALID),
    (dict(), dict(bt=None), INVALID),
    (dict(), dict(mb=0), INVALID),
    (dict(), dict(w=None), INVALID),
    (dict(), dict(w=0x8001), INVALID),
    (dict(), dict(head=900), INVALID),
    (dict(), dict(seq=100), INVALID),
    (dict(), dict(scale=NAN), INVALID),
    (dict(), dict(dtype=9), INVALID),
    (dict(), dict(maxc=-1), INVALID),
    (dict(), dict(ws=None), WORKSPACE),
    (dict(), dict(ws_bytes=1 << 16), WORKSPACE),
    (dict(), dict(ws=0x100001), WORKSPACE),
    (dict(), dict(seqs=0), B.PKV_OK),
])
def test_decode_weights_checks(lib, desc, kw, want):
    a = dict(DECODE, **kw)
    assert lib.pkv_paged_attention_decode_scaled_weights(ctypes.byref(_desc(**desc)),
                                                         *a.values()) == want


EVICT = dict(scales=0x1000, seqs=2, bt=0x2000, mb=64, ctx=0x3000, maxc=1000, w=0x8000, seq=8000,
             head=1000, keep=0x4000, maxk=100, first=4, last=8, dst=0x5000, md=7, wo=0x900000,
             wo_seq=8000, wo_head=1000, wo_len=1000, lens=0x6000, ws=0x100000, ws_bytes=1 << 40,
             err=None, stream=None)


@pytest.mark.parametrize("desc,kw,want", [
    (dict(cache_dtype=B.PKV_F16), {}, UNSUPPORTED),           # scales beside a 16-bit cache
    (dict(), dict(scales=None), INVALID),                     # one scale, but it is 0
    (dict(head_dim=80), {}, UNSUPPORTED),
    (dict(), dict(scales=0x1004), INVALID),
    (dict(), dict(maxk=-1), INVALID),
    (dict(), dict(first=-1), INVALID),
    (dict(), dict(last=-1), INVALID),
    (dict(), dict(md=6), INVALID),                            # 96 of 100 tokens
    (dict(), dict(md=-1), INVALID),
    (dict(), dict(maxk=1 << 30, md=62), INVALID),             # 992 of 1,000
    (dict(), dict(wo_len=99), INVALID),
    (dict(), dict(wo_len=-1), INVALID),
    (dict(), dict(bt=None), INVALID),
    (dict(), dict(ctx=None), INVALID),
    (dict(), dict(keep=None), INVALID),
    (dict(), dict(dst=None), INVALID),
    (dict(), dict(lens=None), INVALID),
    (dict(), dict(w=None), INVALID),
    (dict(), dict(head=999), INVALID),
    (dict(), dict(wo=None), INVALID),
    (dict(), dict(wo=0x8000), INVALID),                       # the weights themselves
    (dict(), dict(wo_head=999), INVALID),
    (dict(), dict(wo_seq=7000), INVALID),
    (dict(), dict(maxc=(1 << 31) - 1), INVALID),
    (dict(), dict(ws=None), WORKSPACE),
    (dict(), dict(ws=0x100040), WORKSPACE),
    (dict(), dict(ws_bytes=4 * 2 * 8 * 100 - 1), WORKSPACE),
    (dict(), dict(seqs=0), B.PKV_OK),
])
def test_evict_checks(lib, desc, kw, want):
    a = dict(EVICT, **kw)
    assert lib.pkv_evict(ctypes.byref(_desc(**desc)), *a.values()) == want


@pytest.mark.parametrize("lens", [0x3000, 0x3004, 0x2ffc, 0x4000, 0x4004])
def test_evict_reads_no_lengths_that_it_writes(lib, lens):
    """lens_out over context_lens or keep_lens of two sequences."""
    a = dict(EVICT, lens=lens)
    assert lib.pkv_evict(ctypes.byref(_desc()), *a.values()) == INVALID


def test_workspaces(lib):
    d = _desc()
    assert B.pkv_evict_workspace_bytes(d, 2, 100, 1000) == 2 * 8 * 100 * 4
    assert B.pkv_evict_workspace_bytes(d, 2, 1000, 100) == 2 * 8 * 100 * 4      # no more than there is
    assert B.pkv_evict_workspace_bytes(d, 0, 100, 1000) == 0
    # scores of every token and query head, the latter to a power of two
    a, b = (B.pkv_decode_scaled_weights_workspace_bytes(d, 4, h, 1000) for h in (24, 32))
    assert a > 4 * 8 * 1000 * 4 * 4 and b - a < 1 << 12
    # launches of 1,024 sequences share it
    n = B.pkv_decode_scaled_weights_workspace_bytes(d, 1024, 64, 5000)
    assert n == B.pkv_decode_scaled_weights_workspace_bytes(d, 100000, 64, 5000)
    # a window holds no more rows than a context has tokens
    n = B.pkv_attention_weights_workspace_bytes(d, 2, 64, 100, 100)
    assert n > 0 and n == B.pkv_attention_weights_workspace_bytes(d, 2, 64, 1 << 30, 100)
    assert B.pkv_attention_weights_workspace_bytes(d, 2, 64, 0, 100) == 0
    # without groups, or with what the call refuses: that of the plain decode
    plain = B.pkv_decode_scaled_workspace_bytes(d, 4, 64, 5000)
    assert B.pkv_decode_scaled_shared_prefix_workspace_bytes(d, 4, 64, 0, 0, 5000) == plain
    assert B.pkv_decode_scaled_shared_prefix_workspace_bytes(d, 4, 64, 2, 2, 5000) > plain


def test_binding_checks():
    """Shapes that the binding refuses before it calls the library."""
    d = _desc(num_blocks=4, num_kv_heads=2, head_dim=64)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    t, c = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    s, w = torch.zeros(4, 2, 2), torch.zeros(3, 2, 10)
    for call in (lambda: B.pkv_paged_attention_decode_scaled_weights(d, s, q, t, c, 10, 0.1, w),
                 lambda: B.pkv_attention_weights(d, q, torch.zeros(4, dtype=torch.int32), 1, t, c, 10, 0.1, w),
                 lambda: B.pkv_evict(d, t, c, 10, w, c, 5, 0, 0, t),
                 lambda: B.pkv_paged_attention_decode_scaled_shared_prefix(
                     d, s, q, t, c, 10, c[:2], c[:1], 3, 1, 0.1)):
        with pytest.raises(ValueError, match="must be on the current CUDA device"):
            call()


def test_windows_of_more_rows_than_32_bits_hold(lib):
    """min(window, max_context_len) x query heads of a KV head beyond 2^30."""
    d = _desc(num_kv_heads=1)
    a = dict(WEIGHTS, heads=128, window=(1 << 23) + 1, maxc=1 << 30, ws=None)
    assert lib.pkv_attention_weights(ctypes.byref(d), *a.values()) == UNSUPPORTED
    assert B.pkv_attention_weights_workspace_bytes(d, 2, 128, a["window"], a["maxc"]) == 0
    a = dict(a, maxc=1 << 23, seq=1 << 23, head=1 << 23)              # (no more rows than a context has)
    assert lib.pkv_attention_weights(ctypes.byref(d), *a.values()) == WORKSPACE
    assert B.pkv_attention_weights_workspace_bytes(d, 2, 128, a["window"], a["maxc"]) > 1 << 37


@pytest.mark.parametrize("seq,head,want", [
    (1000, 2000, WORKSPACE),                                   # head by head (the next check's answer)
    (1500, 2500, WORKSPACE),
    (8000, 1000, WORKSPACE),
    (1000, 1999, INVALID),
    (999, 5000, INVALID),
    (1000, 1000, INVALID),
    (-1000, 2000, INVALID),
    (1 << 62, 1 << 62, INVALID),                               # (the same row, modulo 2^64 in bytes)
    (1 << 62, 1 << 60, INVALID),
])
def test_totals_of_either_order(lib, seq, head, want):
    """Two sequences, eight heads, rows of 1,000."""
    for fn, args in ((lib.pkv_attention_weights, WEIGHTS),
                     (lib.pkv_paged_attention_decode_scaled_weights, dict(DECODE, seqs=2)),
                     (lib.pkv_evict, EVICT)):
        a = dict(args, seq=seq, head=head, ws=None)
        assert fn(ctypes.byref(_desc()), *a.values()) == want
    a = dict(EVICT, wo_seq=seq, wo_head=head, ws=None)
    assert lib.pkv_evict(ctypes.byref(_desc()), *a.values()) == want
