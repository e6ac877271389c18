"""Thin ctypes binding of libpkv.so (include/pkv.h).

Argument marshalling only: tensors become device pointers, torch dtypes become
pkv_dtype codes, the stream defaults to torch's current stream, and a non-zero
status raises :class:`PkvError`.  Every step of the computation runs in the
library's CUDA kernels; there is no other path.  When the library has not been
built the first call raises.

The functions carry the C names.  Caches are described by :class:`CacheDesc`
(``pkv_cache_desc``); :func:`cache_desc` fills one from two torch tensors.
"""
import ctypes
import os
import re

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libpkv.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "pkv.h")

PKV_F16, PKV_BF16, PKV_FP8_E4M3 = 0, 1, 2
PKV_OK, PKV_ERR_INVALID_ARG, PKV_ERR_UNSUPPORTED, PKV_ERR_WORKSPACE, PKV_ERR_CUDA = range(5)
PKV_ERR_SCRATCH_LIMIT = 5
PKV_STATIC_SCRATCH_BYTES = 32 << 20
PKV_DEVERR_SLOT, PKV_DEVERR_BLOCK_ID, PKV_DEVERR_CONTEXT, PKV_DEVERR_COPY_PAIR = 1, 2, 4, 8
PKV_DEVERR_TIMEOUT = 16
PKV_DEVERR_PREFIX = 32
PKV_DEVERR_SCHED = 64


class PkvError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__("%s: %s (status %d)" % (where, pkv_status_string(status), status))


class CacheDesc(ctypes.Structure):
    _fields_ = [("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
                ("num_blocks", ctypes.c_int64), ("num_kv_heads", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("cache_dtype", ctypes.c_int32), ("k_scale", ctypes.c_float),
                ("v_scale", ctypes.c_float)]
    device = None          # of the caches (-1: host), where cache_desc made it


_lib = None


def library_path():
    return LIB_PATH


def load():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("libpkv.so is not built (%s); run paged_kv_cache_130_gb300.build.build()"
                           % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    dp = ctypes.POINTER(CacheDesc)
    sigs = {
        "pkv_status_string": (ctypes.c_char_p, [i32]),
        "pkv_kv_append": (i32, [dp, vp, vp, i32, vp, i64, vp, vp]),
        "pkv_copy_blocks": (i32, [dp, i32, vp, i64, vp, vp]),
        "pkv_decode_partition_size": (i32, [dp, i32, i32, i32, i32]),
        "pkv_decode_workspace_bytes": (ctypes.c_size_t, [dp, i32, i32, i32, i32]),
        "pkv_paged_attention_decode": (i32, [dp, vp, i32, i32, i32, vp, i32, vp, i32, f32, i32,
                                             vp, ctypes.c_size_t, vp, vp, vp]),
        "pkv_paged_attention_partitions": (i32, [dp, vp, i32, i32, i32, vp, i32, vp, i32, f32,
                                                 i32, vp, ctypes.c_size_t, vp, vp, vp]),
        "pkv_lse_reduce": (i32, [i32, i32, i32, vp, i32, i32, vp, ctypes.c_size_t, i32, vp, vp]),
        "pkv_paged_attention_decode_static_ws": (i32, [dp, vp, i32, i32, i32, vp, i32, vp, i32,
                                                       f32, i32, vp, vp, vp]),
        "pkv_shared_prefix_workspace_bytes": (ctypes.c_size_t, [dp, i32, i32, i32, i32]),
        "pkv_swap_blocks": (i32, [dp, dp, i32, vp, i64, vp, vp]),
        "pkv_block_hashes": (i32, [vp, vp, i32, i64, i32, vp, vp, i64, vp, vp, vp]),
        "pkv_paged_attention_prefill": (i32, [dp, vp, i32, i32, i32, vp, i32, i32, vp, i32,
                                              vp, i32, f32, vp, vp, vp]),
        "pkv_paged_attention_decode_shared_prefix": (i32, [dp, vp, i32, i32, i32, vp, i32, vp,
                                                           i32, i32, vp, vp, i32, i32, f32, i32,
                                                           vp, ctypes.c_size_t, vp, vp, vp]),
        "pkv_rope_append": (i32, [dp, vp, vp, i64, vp, i64, vp, i64, i32, i32, vp, i32, i32, f32,
                                  i32, vp, i32, i32, vp, i32, vp, i32, vp, vp, vp]),
        "pkv_decode_scaled_partition_size": (i32, [dp, i32, i32, i32, i32]),
        "pkv_decode_scaled_workspace_bytes": (ctypes.c_size_t, [dp, i32, i32, i32, i32]),
        "pkv_paged_attention_decode_scaled": (i32, [dp, vp, vp, i32, i32, i32, vp, i32, vp, i32,
                                                    f32, i32, vp, ctypes.c_size_t, vp, vp, vp]),
        "pkv_paged_attention_prefill_scaled": (i32, [dp, vp, vp, i32, i32, i32, vp, i32, i32, vp,
                                                     i32, vp, i32, f32, vp, vp, vp]),
        "pkv_copy_blocks_scaled": (i32, [dp, ctypes.POINTER(vp), dp, ctypes.POINTER(vp), i32, vp,
                                         i64, vp, vp]),
        "pkv_rope_append_at": (i32, [dp, vp, vp, i64, vp, i64, vp, i64, i32, i32, vp, i32, i32,
                                     f32, i32, vp, i32, i32, vp, i32, vp, i32, vp, vp, vp, vp]),
        "pkv_decode_scaled_shared_prefix_workspace_bytes": (ctypes.c_size_t, [dp, i32, i32, i32,
                                                                              i32, i32]),
        "pkv_paged_attention_decode_scaled_shared_prefix": (i32, [
            dp, vp, vp, i32, i32, i32, vp, i32, vp, i32, i32, vp, vp, i32, i32, f32, vp,
            ctypes.c_size_t, vp, vp, vp]),
        "pkv_attention_weights_workspace_bytes": (ctypes.c_size_t, [dp, i32, i32, i32, i32]),
        "pkv_attention_weights": (i32, [dp, vp, vp, i32, i32, i32, vp, i32, i32, vp, i32, vp, i32,
                                        f32, vp, i64, i64, vp, ctypes.c_size_t, vp, vp]),
        "pkv_decode_scaled_weights_workspace_bytes": (ctypes.c_size_t, [dp, i32, i32, i32]),
        "pkv_paged_attention_decode_scaled_weights": (i32, [
            dp, vp, vp, i32, i32, i32, vp, i32, vp, i32, f32, vp, i64, i64, vp, ctypes.c_size_t,
            vp, vp, vp]),
        "pkv_evict_workspace_bytes": (ctypes.c_size_t, [dp, i32, i32, i32]),
        "pkv_evict": (i32, [dp, vp, i32, vp, i32, vp, i32, vp, i64, i64, vp, i32, i32, i32, vp,
                            i32, vp, i64, i64, i32, vp, vp, ctypes.c_size_t, vp, vp]),
        "pkv_testing_set_decode_wait_limit": (ctypes.c_uint32, [ctypes.c_uint32]),
        "pkv_testing_set_shared_prefix_path": (i32, [i32]),
        "pkv_testing_stream_copy": (i32, [vp, vp, i64, vp]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def header_functions():
    """Names of the functions include/pkv.h declares."""
    with open(HEADER_PATH) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", " ", text, flags=re.S)
    return sorted(set(re.findall(r"\b(pkv_[a-z_0-9]+)\s*\(", text)))


# ------------------------------------------------------------------ helpers

def dtype_code(t):
    if t == torch.float16:
        return PKV_F16
    if t == torch.bfloat16:
        return PKV_BF16
    if t in (torch.uint8, getattr(torch, "float8_e4m3fn", None)):
        return PKV_FP8_E4M3
    raise TypeError("unsupported element type %s" % t)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


# the current device and its current stream as plain numbers; the public call
# makes a Stream object each time, several microseconds of a small call
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None and _raw_device is not None:
            return ctypes.c_void_p(_raw_stream(_raw_device()))
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _allocate(make, stream):
    """make(), a tensor that a call on `stream` writes.  With an explicit stream it
    comes from that stream's pool: memory from the current stream's may still be
    read there, by work queued before its last owner let go of it, and the call
    does not wait for that.  The caller reads the tensor on the current stream, so
    its memory is not handed out again before that stream is done either."""
    if stream is None:
        return make()
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    here = torch.cuda.current_stream()
    with torch.cuda.stream(torch.cuda.ExternalStream(handle)):
        t = make()
    if here.cuda_stream != handle:
        t.record_stream(here)
    return t


def _check(status, where):
    if status != PKV_OK:
        raise PkvError(status, where)


def _dense(t, name):
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def cache_desc(k_cache, v_cache, k_scale=1.0, v_scale=1.0):
    """Descriptor of one layer's caches, each [num_blocks, num_kv_heads, block_size, head_dim]."""
    _dense(k_cache, "k_cache")
    _dense(v_cache, "v_cache")
    if k_cache.shape != v_cache.shape or k_cache.dtype != v_cache.dtype or k_cache.dim() != 4 or \
            k_cache.device != v_cache.device:
        raise ValueError("k_cache and v_cache must be alike, 4-D")
    nb, hkv, bs, d = k_cache.shape
    desc = CacheDesc(k_cache.data_ptr(), v_cache.data_ptr(), nb, hkv, bs, d,
                     dtype_code(k_cache.dtype), float(k_scale), float(v_scale))
    desc.device = k_cache.get_device()
    return desc


# ------------------------------------------------------------------ entry points

def pkv_status_string(status):
    return load().pkv_status_string(int(status)).decode()


def pkv_kv_append(cache, k, v, slot_mapping, dev_err=None, stream=None):
    _dense(k, "k")
    _dense(v, "v")
    _dense(slot_mapping, "slot_mapping")
    if slot_mapping.dtype != torch.int64 or k.shape != v.shape:
        raise ValueError("slot_mapping must be int64 and k, v alike")
    _check(load().pkv_kv_append(ctypes.byref(cache), _ptr(k), _ptr(v), dtype_code(k.dtype),
                                _ptr(slot_mapping), slot_mapping.numel(), _ptr(dev_err),
                                _stream(stream)), "pkv_kv_append")


def pkv_copy_blocks(caches, block_pairs, dev_err=None, stream=None):
    if isinstance(caches, CacheDesc):
        caches = [caches]
    arr = (CacheDesc * len(caches))(*caches)
    _dense(block_pairs, "block_pairs")
    if block_pairs.dtype != torch.int64:
        raise ValueError("block_pairs must be int64 [n, 2]")
    n = block_pairs.numel() // 2
    _check(load().pkv_copy_blocks(arr, len(caches), _ptr(block_pairs), n, _ptr(dev_err),
                                  _stream(stream)), "pkv_copy_blocks")


def pkv_decode_partition_size(cache, num_seqs, num_heads, max_context_len, requested=0):
    return int(load().pkv_decode_partition_size(ctypes.byref(cache), int(num_seqs),
                                                int(num_heads), int(max_context_len),
                                                int(requested)))


def pkv_decode_workspace_bytes(cache, num_seqs, num_heads, max_context_len, partition_size=0):
    return int(load().pkv_decode_workspace_bytes(ctypes.byref(cache), num_seqs, num_heads,
                                                 max_context_len, partition_size))


def _decode_common(fn, where, cache, q, block_tables, context_lens, max_context_len, scale,
                   partition_size, workspace, dev_err, out, stream):
    _dense(q, "q")
    _dense(block_tables, "block_tables")
    _dense(context_lens, "context_lens")
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError("block_tables and context_lens must be int32")
    s, h, d = q.shape
    if out is None:
        out = _allocate(lambda: torch.empty_like(q), stream)
    need = pkv_decode_workspace_bytes(cache, s, h, max_context_len, partition_size)
    if workspace is None and need > 0:
        workspace = _allocate(lambda: torch.empty(need, dtype=torch.uint8, device=q.device),
                              stream)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(fn(ctypes.byref(cache), _ptr(q), dtype_code(q.dtype), s, h, _ptr(block_tables),
              block_tables.shape[1], _ptr(context_lens), int(max_context_len), float(scale),
              int(partition_size), _ptr(workspace), ws_bytes, _ptr(dev_err), _ptr(out),
              _stream(stream)), where)
    return out


def pkv_paged_attention_decode(cache, q, block_tables, context_lens, max_context_len, scale,
                               partition_size=0, workspace=None, dev_err=None, out=None,
                               stream=None):
    return _decode_common(load().pkv_paged_attention_decode, "pkv_paged_attention_decode",
                          cache, q, block_tables, context_lens, max_context_len, scale,
                          partition_size, workspace, dev_err, out, stream)


def pkv_paged_attention_partitions(cache, q, block_tables, context_lens, max_context_len, scale,
                                   partition_size=0, workspace=None, dev_err=None, out=None,
                                   stream=None):
    return _decode_common(load().pkv_paged_attention_partitions,
                          "pkv_paged_attention_partitions", cache, q, block_tables,
                          context_lens, max_context_len, scale, partition_size, workspace,
                          dev_err, out, stream)


def pkv_lse_reduce(num_seqs, num_heads, head_dim, context_lens, max_context_len, partition_size,
                   workspace, out, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(load().pkv_lse_reduce(num_seqs, num_heads, head_dim, _ptr(context_lens),
                                 int(max_context_len), int(partition_size), _ptr(workspace),
                                 ws_bytes, dtype_code(out.dtype), _ptr(out), _stream(stream)),
           "pkv_lse_reduce")
    return out


def pkv_paged_attention_decode_static_ws(cache, q, block_tables, context_lens, max_context_len,
                                         scale, partition_size=0, dev_err=None, out=None,
                                         stream=None):
    """Decode without a caller workspace: for callers that cannot allocate
    device memory (an engine that has reserved the GPU's memory for its own
    cache pool, or a latency-critical path where cudaMalloc may synchronise).
    The partials live in the library's static 32 MiB device array; calls that
    overlap on the GPU race on it, so keep them on one stream."""
    _dense(q, "q")
    _dense(block_tables, "block_tables")
    _dense(context_lens, "context_lens")
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError("block_tables and context_lens must be int32")
    s, h, d = q.shape
    if out is None:
        out = _allocate(lambda: torch.empty_like(q), stream)
    _check(load().pkv_paged_attention_decode_static_ws(
        ctypes.byref(cache), _ptr(q), dtype_code(q.dtype), s, h, _ptr(block_tables),
        block_tables.shape[1], _ptr(context_lens), int(max_context_len), float(scale),
        int(partition_size), _ptr(dev_err), _ptr(out), _stream(stream)),
        "pkv_paged_attention_decode_static_ws")
    return out


def pkv_testing_set_decode_wait_limit(tries):
    """Polls per bounded wait of the streaming decode kernel and of attention
    weights for later calls (0: the kernel's own limit); a testing aid.  Returns
    the previous setting."""
    return int(load().pkv_testing_set_decode_wait_limit(int(tries)))


def pkv_testing_set_shared_prefix_path(path):
    """Route of later shared-prefix decode calls (0: the library's choice,
    1: the single pass, 2: prefix kernel + partitions + reduce); a testing
    aid.  Returns the previous setting."""
    r = int(load().pkv_testing_set_shared_prefix_path(int(path)))
    if r < 0:
        raise ValueError("path must be 0, 1 or 2")
    return r


def pkv_shared_prefix_workspace_bytes(cache, num_seqs, num_heads, max_context_len,
                                      partition_size=0):
    return int(load().pkv_shared_prefix_workspace_bytes(ctypes.byref(cache), num_seqs,
                                                        num_heads, max_context_len,
                                                        partition_size))


def pkv_paged_attention_decode_shared_prefix(cache, q, block_tables, context_lens,
                                             max_context_len, group_begin, group_prefix_blocks,
                                             max_group_size, max_prefix_blocks, scale,
                                             partition_size=0, workspace=None, dev_err=None,
                                             out=None, stream=None):
    """Decode where the sequences [group_begin[i], group_begin[i+1]) share their
    first group_prefix_blocks[i] blocks (int32 device tensors); the two
    max_* arguments are host upper bounds."""
    _dense(q, "q")
    _dense(block_tables, "block_tables")
    _dense(context_lens, "context_lens")
    _dense(group_begin, "group_begin")
    _dense(group_prefix_blocks, "group_prefix_blocks")
    for t, name in ((block_tables, "block_tables"), (context_lens, "context_lens"),
                    (group_begin, "group_begin"), (group_prefix_blocks, "group_prefix_blocks")):
        if t.dtype != torch.int32:
            raise ValueError("%s must be int32" % name)
    num_groups = group_prefix_blocks.numel()
    if group_begin.numel() != num_groups + 1:
        raise ValueError("group_begin needs num_groups + 1 entries")
    s, h, d = q.shape
    if out is None:
        out = _allocate(lambda: torch.empty_like(q), stream)
    need = pkv_shared_prefix_workspace_bytes(cache, s, h, max_context_len, partition_size)
    if workspace is None and need > 0:
        workspace = _allocate(lambda: torch.empty(need, dtype=torch.uint8, device=q.device),
                              stream)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load().pkv_paged_attention_decode_shared_prefix(
        ctypes.byref(cache), _ptr(q), dtype_code(q.dtype), s, h, _ptr(block_tables),
        block_tables.shape[1], _ptr(context_lens), int(max_context_len), num_groups,
        _ptr(group_begin), _ptr(group_prefix_blocks), int(max_group_size),
        int(max_prefix_blocks), float(scale), int(partition_size), _ptr(workspace), ws_bytes,
        _ptr(dev_err), _ptr(out), _stream(stream)), "pkv_paged_attention_decode_shared_prefix")
    return out


def pkv_paged_attention_prefill(cache, q, cu_seqlens_q, max_q_len, block_tables, context_lens,
                                max_context_len, scale, dev_err=None, out=None, stream=None):
    """Causal prefill of q [total_q, num_heads, head_dim]: sequence s owns rows
    [cu_seqlens_q[s], cu_seqlens_q[s+1]), the last tokens of its context."""
    _dense(q, "q")
    for t, name in ((cu_seqlens_q, "cu_seqlens_q"), (block_tables, "block_tables"),
                    (context_lens, "context_lens")):
        _dense(t, name)
        if t.dtype != torch.int32:
            raise ValueError("%s must be int32" % name)
    total, h, d = q.shape
    num_seqs = context_lens.numel()
    if cu_seqlens_q.numel() != num_seqs + 1:
        raise ValueError("cu_seqlens_q needs num_seqs + 1 entries")
    if out is None:
        out = _allocate(lambda: torch.empty_like(q), stream)
    _check(load().pkv_paged_attention_prefill(
        ctypes.byref(cache), _ptr(q), dtype_code(q.dtype), num_seqs, h, _ptr(cu_seqlens_q),
        total, int(max_q_len), _ptr(block_tables), block_tables.shape[1], _ptr(context_lens),
        int(max_context_len), float(scale), _ptr(dev_err), _ptr(out), _stream(stream)),
        "pkv_paged_attention_prefill")
    return out


def pkv_swap_blocks(src, dst, block_pairs, dev_err=None, stream=None):
    """Move blocks src[l][pairs[i, 0]] -> dst[l][pairs[i, 1]] for every layer;
    `src` / `dst` are CacheDesc lists (device or pinned host pools)."""
    if isinstance(src, CacheDesc):
        src, dst = [src], [dst]
    if len(src) != len(dst):
        raise ValueError("src and dst need one descriptor per layer")
    a = (CacheDesc * len(src))(*src)
    b = (CacheDesc * len(dst))(*dst)
    _dense(block_pairs, "block_pairs")
    if block_pairs.dtype != torch.int64:
        raise ValueError("block_pairs must be int64 [n, 2]")
    _check(load().pkv_swap_blocks(a, b, len(src), _ptr(block_pairs), block_pairs.numel() // 2,
                                  _ptr(dev_err), _stream(stream)), "pkv_swap_blocks")


def pkv_testing_stream_copy(dst, src, stream=None):
    """Copy src into dst (same byte size) with SM loads and stores: the
    measurement reference for copies over a link (device <-> pinned host)."""
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != nbytes:
        raise ValueError("dst and src must have the same byte size")
    _check(load().pkv_testing_stream_copy(_ptr(dst), _ptr(src), nbytes, _stream(stream)),
           "pkv_testing_stream_copy")
    return dst


def pkv_block_hashes(token_ids, cu_seqlens, block_size, block_offsets=None, parent_hashes=None,
                     hashes=None, dev_err=None, stream=None):
    """Chained SHA-256 of every full block; returns uint8 [total_blocks, 32].
    `block_offsets` (int64 [num_seqs]) defaults to the running count of full
    blocks, which needs the lengths on the host (one device-to-host copy)."""
    _dense(token_ids, "token_ids")
    _dense(cu_seqlens, "cu_seqlens")
    if token_ids.dtype != torch.int32 or cu_seqlens.dtype != torch.int32:
        raise ValueError("token_ids and cu_seqlens must be int32")
    num_seqs = cu_seqlens.numel() - 1
    if block_offsets is None:
        full = torch.diff(cu_seqlens.to(torch.int64)) // block_size
        block_offsets = torch.cumsum(full, 0) - full
        total_blocks = int(full.sum().item())
        if stream is not None:
            # (read there after the caller's view of it is gone)
            block_offsets.record_stream(torch.cuda.ExternalStream(
                stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)))
    else:
        _dense(block_offsets, "block_offsets")
        total_blocks = hashes.shape[0] if hashes is not None else None
        if total_blocks is None:
            raise ValueError("pass `hashes` together with `block_offsets`")
    if hashes is None:
        hashes = _allocate(lambda: torch.empty((max(total_blocks, 1), 32), dtype=torch.uint8,
                                               device=token_ids.device), stream)
    if parent_hashes is not None:
        _dense(parent_hashes, "parent_hashes")
    _check(load().pkv_block_hashes(_ptr(token_ids), _ptr(cu_seqlens), num_seqs,
                                   token_ids.numel(), int(block_size), _ptr(parent_hashes),
                                   _ptr(block_offsets), total_blocks, _ptr(hashes), _ptr(dev_err),
                                   _stream(stream)), "pkv_block_hashes")
    return hashes[:total_blocks]


# ------------------------------------------------------------------ scaled cache
#
# A decode step's calls take a few microseconds on the GPU, as long as the
# marshalling of their arguments: these functions look at each tensor once and
# hand plain numbers to ctypes.

_I32, _F32, _F64 = torch.int32, torch.float32, torch.float64
_CODES = {torch.float16: PKV_F16, torch.bfloat16: PKV_BF16}


def _here(t, name):
    """The current CUDA device, where a call runs; t must be on it."""
    dev = t.get_device()
    if dev < 0 or dev != (_raw_device() if _raw_device is not None else
                          torch.cuda.current_device()):
        raise ValueError("%s must be on the current CUDA device" % name)
    return dev


def _handle(stream, dev):
    """Handle of `stream`, or of device dev's current one."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(dev)
    return _stream(stream)


def _refuse(t, dev, name, what):
    """The error of a tensor that is not `what` on device dev."""
    if t.get_device() != dev:
        what = "on the current CUDA device"
    return ValueError("%s must be %s" % (name, what))


def _elsewhere(cache, dev):
    """Whether cache_desc made it on another device than dev."""
    return cache.device != dev and cache.device is not None


def _i32(t, name, dev):
    """Address of a dense int32 tensor on device dev."""
    if t.dtype is not _I32 or not t.is_contiguous() or t.get_device() != dev:
        raise _refuse(t, dev, name, "contiguous int32")
    return t.data_ptr()


def _err_flag(t, dev):
    """Address of the word that device checks set bits in."""
    if t.dtype is not _I32 or t.numel() < 1 or t.get_device() != dev:
        raise _refuse(t, dev, "dev_err", "int32 with an element")
    return t.data_ptr()


def _scales_of(cache, scales, dev):
    """Address of a layer's scales, float32 [num_blocks, num_kv_heads, 2]."""
    if scales.dtype is not _F32 or not scales.is_contiguous() or scales.get_device() != dev or \
            scales.numel() != 2 * cache.num_blocks * cache.num_kv_heads:
        raise _refuse(scales, dev, "scales", "contiguous float32 [num_blocks, num_kv_heads, 2]")
    return scales.data_ptr()


def _code16(t, name):
    c = _CODES.get(t.dtype)
    if c is None:
        raise TypeError("%s must be float16 or bfloat16" % name)
    return c


def _token_rows(t, name, n, h, d):
    """Elements between the tokens of t [n, h, d], whose heads lie side by side
    (a slice of a fused projection will do)."""
    a, b, c = t.stride()
    if c != 1 or (h > 1 and b != d):
        raise ValueError("%s must be [tokens, heads, head_dim] with dense heads" % name)
    return a if n > 1 else h * d


def _like(t, ref, name, dev):
    if t.shape != ref.shape or t.dtype is not ref.dtype or not t.is_contiguous() or \
            t.get_device() != dev:
        raise _refuse(t, dev, name, "dense and like q")
    return t


def pkv_rope_append(cache, q, k, v, inv_freq, cu_seqlens_q, max_q_len, block_tables, context_lens,
                    max_context_len, interleaved=False, mscale=1.0, scales=None, dev_err=None,
                    q_out=None, stream=None, position_offsets=None):
    """Rotate q and K by their positions and append K and V; returns the rotated
    q (None without q).  `inv_freq` is a float64 device tensor of rot_dim / 2
    radians per position (rope.inv_freq computes it), or None to rotate
    nothing; with `scales` the cache is a scaled one.  `position_offsets` (int32
    [num_seqs]): how far positions are ahead of places in the context, as after
    an eviction (pkv_rope_append_at)."""
    dev = _here(k, "k")
    if _elsewhere(cache, dev):
        raise ValueError("the cache must be on the current CUDA device")
    code = _code16(k, "k")
    rows, kv, d = shape = k.shape
    if kv != cache.num_kv_heads or d != cache.head_dim or v.shape != shape or \
            v.dtype is not k.dtype:
        raise ValueError("k and v must be alike and fit the cache")
    if v.get_device() != dev:
        raise _refuse(v, dev, "v", "")
    qp = qo = None
    qs = heads = 0
    if q is not None:
        rows_q, heads, d_q = q.shape
        if rows_q != rows or d_q != d or q.dtype is not k.dtype or q.get_device() != dev:
            raise _refuse(q, dev, "q", "alike k in its tokens, head_dim and type")
        qs = _token_rows(q, "q", rows, heads, d)
        if q_out is None:
            # (dense: q is, but for the space between tokens)
            q_out = torch.empty_like(q) if stream is None else \
                _allocate(lambda: torch.empty_like(q), stream)
        else:
            _like(q_out, q, "q_out", dev)
        qp, qo = q.data_ptr(), q_out.data_ptr()
    rot, fp = 0, None
    if inv_freq is not None:
        if inv_freq.dtype is not _F64 or not inv_freq.is_contiguous() or \
                inv_freq.get_device() != dev:
            raise _refuse(inv_freq, dev, "inv_freq", "contiguous float64")
        rot, fp = 2 * inv_freq.numel(), inv_freq.data_ptr()
    num_seqs = context_lens.numel()
    n_tables, width = block_tables.shape
    if cu_seqlens_q.numel() != num_seqs + 1 or n_tables != num_seqs:
        raise ValueError("cu_seqlens_q needs num_seqs + 1 entries, block_tables num_seqs rows")
    offsets = None
    if position_offsets is not None:
        offsets = _i32(position_offsets, "position_offsets", dev)
        if position_offsets.numel() != num_seqs:
            raise ValueError("position_offsets needs num_seqs entries")
    st = (_lib or load()).pkv_rope_append_at(
        ctypes.byref(cache), None if scales is None else _scales_of(cache, scales, dev), qp, qs,
        k.data_ptr(), _token_rows(k, "k", rows, kv, d), v.data_ptr(),
        _token_rows(v, "v", rows, kv, d), code, heads, fp, rot, interleaved, mscale, num_seqs,
        _i32(cu_seqlens_q, "cu_seqlens_q", dev), rows, max_q_len,
        _i32(block_tables, "block_tables", dev), width, _i32(context_lens, "context_lens", dev),
        max_context_len, offsets, None if dev_err is None else _err_flag(dev_err, dev), qo,
        _handle(stream, dev))
    if st:
        raise PkvError(st, "pkv_rope_append")
    return q_out if q is not None else None


def pkv_decode_scaled_partition_size(cache, num_seqs, num_heads, max_context_len, requested=0):
    return int(load().pkv_decode_scaled_partition_size(ctypes.byref(cache), num_seqs, num_heads,
                                                       max_context_len, requested))


def pkv_decode_scaled_workspace_bytes(cache, num_seqs, num_heads, max_context_len,
                                      partition_size=0):
    return int(load().pkv_decode_scaled_workspace_bytes(ctypes.byref(cache), num_seqs, num_heads,
                                                        max_context_len, partition_size))


def pkv_paged_attention_decode_scaled(cache, scales, q, block_tables, context_lens,
                                      max_context_len, scale, partition_size=0, workspace=None,
                                      dev_err=None, out=None, stream=None):
    """Decode over a scaled cache; arguments as pkv_paged_attention_decode."""
    dev = _here(q, "q")
    if _elsewhere(cache, dev):
        raise ValueError("the cache must be on the current CUDA device")
    s, h, d = q.shape
    n_tables, width = block_tables.shape
    if d != cache.head_dim or context_lens.numel() != s or n_tables != s or not q.is_contiguous():
        raise ValueError("q (dense), block_tables and context_lens do not fit together")
    if out is not None:
        _like(out, q, "out", dev)
    elif stream is None:
        out = torch.empty_like(q)
    else:
        out = _allocate(lambda: torch.empty_like(q), stream)
    wp, ws_bytes = None, 0
    if workspace is None:
        need = pkv_decode_scaled_workspace_bytes(cache, s, h, max_context_len, partition_size)
        if need > 0:
            workspace = _allocate(
                lambda: torch.empty(need, dtype=torch.uint8, device=q.device), stream)
    if workspace is not None:
        if workspace.get_device() != dev:
            raise _refuse(workspace, dev, "workspace", "")
        wp, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    st = (_lib or load()).pkv_paged_attention_decode_scaled(
        ctypes.byref(cache), _scales_of(cache, scales, dev), q.data_ptr(), _code16(q, "q"), s, h,
        _i32(block_tables, "block_tables", dev), width, _i32(context_lens, "context_lens", dev),
        max_context_len, scale, partition_size, wp, ws_bytes,
        None if dev_err is None else _err_flag(dev_err, dev), out.data_ptr(),
        _handle(stream, dev))
    if st:
        raise PkvError(st, "pkv_paged_attention_decode_scaled")
    return out


def pkv_paged_attention_prefill_scaled(cache, scales, q, cu_seqlens_q, max_q_len, block_tables,
                                       context_lens, max_context_len, scale, dev_err=None,
                                       out=None, stream=None):
    """Causal attention over a scaled cache; arguments as
    pkv_paged_attention_prefill."""
    dev = _here(q, "q")
    if _elsewhere(cache, dev):
        raise ValueError("the cache must be on the current CUDA device")
    total, h, d = q.shape
    num_seqs = context_lens.numel()
    n_tables, width = block_tables.shape
    if d != cache.head_dim or cu_seqlens_q.numel() != num_seqs + 1 or n_tables != num_seqs or \
            not q.is_contiguous():
        raise ValueError("q (dense), cu_seqlens_q, block_tables and context_lens do not fit "
                         "together")
    if out is not None:
        _like(out, q, "out", dev)
    elif stream is None:
        out = torch.empty_like(q)
    else:
        out = _allocate(lambda: torch.empty_like(q), stream)
    st = (_lib or load()).pkv_paged_attention_prefill_scaled(
        ctypes.byref(cache), _scales_of(cache, scales, dev), q.data_ptr(), _code16(q, "q"),
        num_seqs, h, _i32(cu_seqlens_q, "cu_seqlens_q", dev), total, max_q_len,
        _i32(block_tables, "block_tables", dev), width, _i32(context_lens, "context_lens", dev),
        max_context_len, scale, None if dev_err is None else _err_flag(dev_err, dev),
        out.data_ptr(), _handle(stream, dev))
    if st:
        raise PkvError(st, "pkv_paged_attention_prefill_scaled")
    return out


def pkv_copy_blocks_scaled(caches, scales, block_pairs, dst=None, dst_scales=None, dev_err=None,
                           stream=None):
    """Copy blocks with their scales: inside one pool, or with `dst` and
    `dst_scales` from one pool to another (device or pinned host memory)."""
    if isinstance(caches, CacheDesc):
        caches, scales = [caches], [scales]
        if dst is not None:
            dst, dst_scales = [dst], [dst_scales]
    n = len(caches)
    if len(scales) != n or (dst is None) != (dst_scales is None) or \
            (dst is not None and (len(dst) != n or len(dst_scales) != n)):
        raise ValueError("one array of scales per layer, and as many layers on both sides")
    if block_pairs.dtype is not torch.int64 or not block_pairs.is_contiguous():
        raise ValueError("block_pairs must be contiguous int64 [n, 2]")
    if dst is None:
        dev = _here(block_pairs, "block_pairs")
    else:
        # a pool may be in pinned host memory (which the library checks), and so
        # may the pairs; what is on a GPU is on this one
        dev = _raw_device() if _raw_device is not None else torch.cuda.current_device()
        if block_pairs.is_cuda and block_pairs.get_device() != dev:
            raise _refuse(block_pairs, dev, "block_pairs", "")
    for c in caches if dst is None else (*caches, *dst):
        if _elsewhere(c, dev) and (dst is None or c.device != -1):
            raise ValueError("the cache must be on the current CUDA device")

    def addresses(descs, ts):
        return ptrs(*[_scales_of(c, t, -1 if dst is not None and not t.is_cuda else dev)
                      for c, t in zip(descs, ts)])

    ptrs = ctypes.c_void_p * n
    a, a_s = (CacheDesc * n)(*caches), addresses(caches, scales)
    b = b_s = None
    if dst is not None:
        b, b_s = (CacheDesc * n)(*dst), addresses(dst, dst_scales)
    st = (_lib or load()).pkv_copy_blocks_scaled(
        a, a_s, b, b_s, n, block_pairs.data_ptr(), block_pairs.numel() // 2,
        None if dev_err is None else _err_flag(dev_err, dev), _handle(stream, dev))
    if st:
        raise PkvError(st, "pkv_copy_blocks_scaled")


# ------------------------------------------------------------------ long contexts
#
# Shared prefixes over the scaled cache, attention weights, eviction.

def _workspace(workspace, need, dev, stream, device):
    """The caller's scratch, or `need` bytes: (tensor, address, bytes)."""
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=device) if stream is None else \
            _allocate(lambda: torch.empty(need, dtype=torch.uint8, device=device), stream)
    elif workspace.get_device() != dev:
        raise _refuse(workspace, dev, "workspace", "")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _out_like(out, q, dev, stream):
    if out is not None:
        return _like(out, q, "out", dev)
    return torch.empty_like(q) if stream is None else _allocate(lambda: torch.empty_like(q), stream)


def _totals(t, name, num_seqs, kv_heads, least, dev):
    """Address and strides of a [num_seqs, kv_heads, >= least] float32 tensor of
    dense rows."""
    if t.dtype is not _F32 or t.dim() != 3 or t.get_device() != dev or t.stride(2) != 1 and \
            t.shape[2] > 1:
        raise _refuse(t, dev, name, "float32 [num_seqs, num_kv_heads, tokens] with dense rows")
    n, h, w = t.shape
    if n != num_seqs or h != kv_heads or w < least:
        raise ValueError("%s must be [num_seqs, num_kv_heads, at least %d]" % (name, least))
    return t.data_ptr(), t.stride(0), t.stride(1)


def pkv_decode_scaled_shared_prefix_workspace_bytes(cache, num_seqs, num_heads, num_groups,
                                                    max_group_size, max_context_len):
    return int(load().pkv_decode_scaled_shared_prefix_workspace_bytes(
        ctypes.byref(cache), num_seqs, num_heads, num_groups, max_group_size, max_context_len))


def pkv_paged_attention_decode_scaled_shared_prefix(cache, scales, q, block_tables, context_lens,
                                                    max_context_len, group_begin,
                                                    group_prefix_blocks, max_group_size,
                                                    max_prefix_blocks, scale, workspace=None,
                                                    dev_err=None, out=None, stream=None):
    """Decode over a scaled cache where the sequences [group_begin[i],
    group_begin[i+1]) share their first group_prefix_blocks[i] blocks; arguments
    as pkv_paged_attention_decode_shared_prefix."""
    dev = _here(q, "q")
    if _elsewhere(cache, dev):
        raise ValueError("the cache must be on the current CUDA device")
    s, h, d = q.shape
    n_tables, width = block_tables.shape
    groups = group_prefix_blocks.numel()
    if d != cache.head_dim or context_lens.numel() != s or n_tables != s or not q.is_contiguous():
        raise ValueError("q (dense), block_tables and context_lens do not fit together")
    if group_begin.numel() != groups + 1:
        raise ValueError("group_begin needs num_groups + 1 entries")
    code = _code16(q, "q")
    out = _out_like(out, q, dev, stream)
    need = 0 if workspace is not None else pkv_decode_scaled_shared_prefix_workspace_bytes(
        cache, s, h, groups, max_group_size, max_context_len)
    workspace, wp, ws_bytes = _workspace(workspace, need, dev, stream, q.device)
    st = (_lib or load()).pkv_paged_attention_decode_scaled_shared_prefix(
        ctypes.byref(cache), _scales_of(cache, scales, dev), q.data_ptr(), code, s, h,
        _i32(block_tables, "block_tables", dev), width, _i32(context_lens, "context_lens", dev),
        max_context_len, groups, _i32(group_begin, "group_begin", dev),
        _i32(group_prefix_blocks, "group_prefix_blocks", dev), max_group_size, max_prefix_blocks,
        scale, wp, ws_bytes, None if dev_err is None else _err_flag(dev_err, dev), out.data_ptr(),
        _handle(stream, dev))
    if st:
        raise PkvError(st, "pkv_paged_attention_decode_scaled_shared_prefix")
    return out


def pkv_attention_weights_workspace_bytes(cache, num_seqs, num_heads, window, max_context_len):
    return int(load().pkv_attention_weights_workspace_bytes(ctypes.byref(cache), num_seqs,
                                                            num_heads, window, max_context_len))


def pkv_attention_weights(cache, q, cu_seqlens_q, window, block_tables, context_lens,
                          max_context_len, scale, weights, scales=None, workspace=None,
                          dev_err=None, stream=None):
    """Add the attention weights of each sequence's last `window` rows of q, summed
    over rows and the query heads of a KV head, to `weights` (float32 [num_seqs,
    num_kv_heads, at least max_context_len]); returns `weights`.  Any cache: with
    `scales` a scaled one."""
    dev = _here(q, "q")
    if _elsewhere(cache, dev):
        raise ValueError("the cache must be on the current CUDA device")
    total, h, d = q.shape
    num_seqs = context_lens.numel()
    n_tables, width = block_tables.shape
    if d != cache.head_dim or cu_seqlens_q.numel() != num_seqs + 1 or n_tables != num_seqs or \
            not q.is_contiguous():
        raise ValueError("q (dense), cu_seqlens_q, block_tables and context_lens do not fit "
                         "together")
    code = _code16(q, "q")
    at, seq, head = _totals(weights, "weights", num_seqs, cache.num_kv_heads, max_context_len, dev)
    need = 0 if workspace is not None else pkv_attention_weights_workspace_bytes(
        cache, num_seqs, h, window, max_context_len)
    workspace, wp, ws_bytes = _workspace(workspace, need, dev, stream, q.device)
    st = (_lib or load()).pkv_attention_weights(
        ctypes.byref(cache), None if scales is None else _scales_of(cache, scales, dev),
        q.data_ptr(), code, num_seqs, h, _i32(cu_seqlens_q, "cu_seqlens_q", dev), total, window,
        _i32(block_tables, "block_tables", dev), width, _i32(context_lens, "context_lens", dev),
        max_context_len, scale, at, seq, head, wp, ws_bytes,
        None if dev_err is None else _err_flag(dev_err, dev), _handle(stream, dev))
    if st:
        raise PkvError(st, "pkv_attention_weights")
    return weights


def pkv_decode_scaled_weights_workspace_bytes(cache, num_seqs, num_heads, max_context_len):
    return int(load().pkv_decode_scaled_weights_workspace_bytes(ctypes.byref(cache), num_seqs,
                                                                num_heads, max_context_len))


def pkv_paged_attention_decode_scaled_weights(cache, scales, q, block_tables, context_lens,
                                              max_context_len, scale, weights, workspace=None,
                                              dev_err=None, out=None, stream=None):
    """Decode over a scaled cache that adds each token's weight, summed over the
    query heads of its KV head, to `weights`; returns the attention's output."""
    dev = _here(q, "q")
    if _elsewhere(cache, dev):
        raise ValueError("the cache must be on the current CUDA device")
    s, h, d = q.shape
    n_tables, width = block_tables.shape
    if d != cache.head_dim or context_lens.numel() != s or n_tables != s or not q.is_contiguous():
        raise ValueError("q (dense), block_tables and context_lens do not fit together")
    code = _code16(q, "q")
    at, seq, head = _totals(weights, "weights", s, cache.num_kv_heads, max_context_len, dev)
    out = _out_like(out, q, dev, stream)
    need = 0 if workspace is not None else pkv_decode_scaled_weights_workspace_bytes(
        cache, s, h, max_context_len)
    workspace, wp, ws_bytes = _workspace(workspace, need, dev, stream, q.device)
    st = (_lib or load()).pkv_paged_attention_decode_scaled_weights(
        ctypes.byref(cache), _scales_of(cache, scales, dev), q.data_ptr(), code, s, h,
        _i32(block_tables, "block_tables", dev), width, _i32(context_lens, "context_lens", dev),
        max_context_len, scale, at, seq, head, wp, ws_bytes,
        None if dev_err is None else _err_flag(dev_err, dev), out.data_ptr(), _handle(stream, dev))
    if st:
        raise PkvError(st, "pkv_paged_attention_decode_scaled_weights")
    return out


def pkv_evict_workspace_bytes(cache, num_seqs, max_keep_len, max_context_len):
    return int(load().pkv_evict_workspace_bytes(ctypes.byref(cache), num_seqs, max_keep_len,
                                                max_context_len))


def pkv_evict(cache, block_tables, context_lens, max_context_len, weights, keep_lens, max_keep_len,
              keep_first, keep_last, dst_tables, scales=None, weights_out=None, lens_out=None,
              workspace=None, dev_err=None, stream=None):
    """Keep, for every KV head, the tokens of largest weight: at most keep_lens[s]
    of a context, its first and last ones among them, in the blocks of
    `dst_tables`.  Returns (new lengths, their weights, of the shape of `weights`
    unless `weights_out` is given)."""
    dev = _here(context_lens, "context_lens")
    if _elsewhere(cache, dev):
        raise ValueError("the cache must be on the current CUDA device")
    num_seqs = context_lens.numel()
    n_tables, width = block_tables.shape
    n_dst, dst_width = dst_tables.shape
    if n_tables != num_seqs or n_dst != num_seqs or keep_lens.numel() != num_seqs:
        raise ValueError("block_tables, dst_tables, keep_lens and context_lens do not fit together")
    kv = cache.num_kv_heads
    most = min(max_keep_len, max_context_len)
    at, seq, head = _totals(weights, "weights", num_seqs, kv, max_context_len, dev)

    if weights_out is None:
        weights_out = torch.empty_like(weights, memory_format=torch.contiguous_format) \
            if stream is None else \
            _allocate(lambda: torch.empty(weights.shape, dtype=_F32, device=weights.device), stream)
    elif weights_out is weights:
        raise ValueError("weights_out must not be weights")
    to, to_seq, to_head = _totals(weights_out, "weights_out", num_seqs, kv, most, dev)
    if lens_out is None:
        lens_out = torch.empty_like(context_lens) if stream is None else \
            _allocate(lambda: torch.empty_like(context_lens), stream)
    elif lens_out.numel() != num_seqs:
        raise ValueError("lens_out needs num_seqs entries")
    elif lens_out is context_lens or lens_out is keep_lens:
        raise ValueError("lens_out must not be context_lens or keep_lens")
    need = 0 if workspace is not None else pkv_evict_workspace_bytes(cache, num_seqs, max_keep_len,
                                                                     max_context_len)
    workspace, wp, ws_bytes = _workspace(workspace, need, dev, stream, weights.device)
    st = (_lib or load()).pkv_evict(
        ctypes.byref(cache), None if scales is None else _scales_of(cache, scales, dev), num_seqs,
        _i32(block_tables, "block_tables", dev), width, _i32(context_lens, "context_lens", dev),
        max_context_len, at, seq, head, _i32(keep_lens, "keep_lens", dev), max_keep_len, keep_first,
        keep_last, _i32(dst_tables, "dst_tables", dev), dst_width, to, to_seq, to_head,
        weights_out.shape[2], _i32(lens_out, "lens_out", dev), wp, ws_bytes,
        None if dev_err is None else _err_flag(dev_err, dev), _handle(stream, dev))
    if st:
        raise PkvError(st, "pkv_evict")
    return lens_out, weights_out
