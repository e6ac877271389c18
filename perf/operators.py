"""The operators of the 8-bit paged cache with a scale per block and KV head,
as a program of plain torch operations and as calls of the library.

Four operators, the steps of one layer of a serving engine:

* ``rope_append``: rotary positions on the new tokens' q and K, K and V written
  into the paged cache (E4M3 codes with a power-of-two scale per block and KV
  head, or the cache of the input type);
* ``decode``: one query token per sequence attends over the scaled cache;
* ``prefill``: causal attention of prompts and chunks over the scaled cache;
* ``copy``: copy-on-write of blocks with their scales, every layer.

Codes are held as ``torch.float8_e4m3fn`` tensors [num_blocks, kv_heads,
block_size, head_dim], scales as float32 [num_blocks, kv_heads, 2] (K, V); a
value is its code times its scale.
"""
import math
import random

import torch

own = False

F8 = torch.float8_e4m3fn
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
F8_MAX = 448.0
SQRT2_32 = float(torch.tensor(math.sqrt(2.0), dtype=torch.float32))


# ------------------------------------------------------------------ cases

def _rope(name, **kw):
    c = dict(name=name, op="rope_append", num_seqs=1, new_lo=1, new_hi=1, cached_lo=0, cached_hi=0,
             heads=8, kv_heads=8, dim=128, block=16, dtype="bf16", cache="scaled", rot=128,
             layout="half", scaling="none", lens=1)
    c.update(kw)
    return c


def _decode(name, **kw):
    c = dict(name=name, op="decode", num_seqs=1, ctx_lo=1, ctx_hi=1, heads=8, kv_heads=8, dim=128,
             block=16, dtype="bf16", lens=1)
    c.update(kw)
    return c


def _prefill(name, **kw):
    c = dict(name=name, op="prefill", num_seqs=1, new_lo=1, new_hi=1, cached_lo=0, cached_hi=0,
             heads=8, kv_heads=8, dim=128, block=16, dtype="bf16", lens=1)
    c.update(kw)
    return c


def _copy(name, **kw):
    c = dict(name=name, op="copy", layers=1, pairs=1, kv_heads=8, dim=128, block=16, pool=64, lens=1)
    c.update(kw)
    return c


def listed():
    return [
        # one decode step of a small model: four short sequences, launch latency
        _rope("rope_append_tiny_step", num_seqs=4, cached_lo=4, cached_hi=63, heads=8, kv_heads=8,
              dim=64, dtype="f16", rot=64),
        # one decode step of a Llama-2-70B layer, 64 sequences, part-filled blocks
        _rope("rope_append_gqa_step", num_seqs=64, cached_lo=1023, cached_hi=4095, heads=64,
              kv_heads=8, scaling="linear"),
        # whole prompts of a Llama-2-7B layer
        _rope("rope_append_prompts", num_seqs=8, new_lo=512, new_hi=2048, heads=32, kv_heads=32),
        # a chunk after a long cached context, interleaved pairs, half of the
        # head rotated, frequencies interpolated for long contexts, cache kept in bf16
        _rope("rope_append_chunk_16bit", num_seqs=4, new_lo=512, new_hi=512, cached_lo=100000,
              cached_hi=130000, heads=64, kv_heads=8, cache="same", rot=64, layout="interleaved",
              scaling="yarn"),
        # one decode step of a small model: latency
        _decode("decode_tiny", num_seqs=4, ctx_lo=5, ctx_hi=64, dim=64, dtype="f16"),
        # a Llama-2-70B layer's decode step
        _decode("decode_gqa", num_seqs=64, ctx_lo=1024, ctx_hi=4096, heads=64, kv_heads=8),
        # a Llama-2-7B layer over long contexts, block size 32
        _decode("decode_long", num_seqs=16, ctx_lo=8192, ctx_hi=32768, heads=32, kv_heads=32,
                block=32),
        # a short question after a cached conversation: few rows, latency
        _prefill("prefill_short", num_seqs=1, new_lo=37, new_hi=37, cached_lo=300, cached_hi=300,
                 heads=32, kv_heads=8, dtype="f16"),
        # whole prompts of a Llama-2-7B layer
        _prefill("prefill_prompts", num_seqs=8, new_lo=512, new_hi=2048, heads=32, kv_heads=32),
        # chunks of a Llama-2-70B layer after a cached context
        _prefill("prefill_gqa_chunk", num_seqs=4, new_lo=512, new_hi=512, cached_lo=1024,
                 cached_hi=4096, heads=64, kv_heads=8),
        # the copy-on-write of a few diverging samples in one layer: latency
        _copy("copy_few", layers=1, pairs=5, kv_heads=8, dim=64, pool=64),
        # 16 prompts with 6 samples each diverge at once, 32 layers
        _copy("copy_parallel_sampling", layers=32, pairs=80, kv_heads=32, pool=256),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope_append", "decode", "prefill", "copy"])
    dim, block = rng.choice([64, 128, 128]), rng.choice([8, 16, 16, 32])
    dtype, lens = rng.choice(["f16", "bf16"]), rng.randrange(1, 1 << 20)
    kv = rng.choice([1, 2, 4, 5, 8, 16, 32])
    group = rng.choice([1, 1, 2, 3, 4, 7, 8, 16])
    if kv * group > 64:
        group = max(1, 64 // kv)
    heads = kv * group
    if op == "rope_append":
        tokens = _log_int(rng, 1, 8000)
        seqs = min(tokens, _log_int(rng, 1, 64))
        hi = max(1, tokens // seqs)
        lo = rng.randint(1, hi)
        cached = _log_int(rng, 1, 130000 if seqs <= 4 else 4000) - 1
        rot = rng.choice([16, 32, dim // 2, dim, dim])
        c = _rope("", num_seqs=seqs, new_lo=lo, new_hi=hi, cached_lo=cached // 2, cached_hi=cached,
                  heads=heads, kv_heads=kv, dim=dim, block=block, dtype=dtype,
                  cache=rng.choice(["scaled", "scaled", "same"]), rot=rot,
                  layout=rng.choice(["half", "interleaved"]),
                  scaling=rng.choice(["none", "linear", "yarn"]), lens=lens)
    elif op == "decode":
        seqs = _log_int(rng, 1, 64)
        total = _log_int(rng, seqs, 300000 * 32 * 128 // (kv * dim))
        hi = max(1, min(40000, total // seqs))
        c = _decode("", num_seqs=seqs, ctx_lo=max(1, hi // rng.randint(1, 8)), ctx_hi=hi, heads=heads,
                    kv_heads=kv, dim=dim, block=block, dtype=dtype, lens=lens)
    elif op == "prefill":
        seqs = _log_int(rng, 1, 8)
        new = _log_int(rng, 1, 1500)
        cached = rng.choice([0, _log_int(rng, 1, 3000)])
        if seqs * new * (new + cached) * heads > 4 * 512 * 4000 * 64:
            seqs = 1
        c = _prefill("", num_seqs=seqs, new_lo=max(1, new // rng.randint(1, 4)), new_hi=new,
                     cached_lo=cached // 2, cached_hi=cached, heads=heads, kv_heads=kv, dim=dim,
                     block=block, dtype=dtype, lens=lens)
    else:
        pairs = _log_int(rng, 1, 100)
        c = _copy("", layers=_log_int(rng, 1, 20), pairs=pairs, kv_heads=kv, dim=dim, block=block,
                  pool=2 * pairs + rng.randint(0, 50), lens=lens)
    del c["name"]
    return c


def _lengths(case):
    """(new tokens, tokens after the step) of every sequence."""
    r = random.Random(case["lens"])
    if case["op"] == "decode":
        return [1] * case["num_seqs"], [r.randint(case["ctx_lo"], case["ctx_hi"])
                                        for _ in range(case["num_seqs"])]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["num_seqs"])]
    ctx = [n + r.randint(case["cached_lo"], case["cached_hi"]) for n in new]
    return new, ctx


def work(case):
    if case["op"] == "copy":
        per = case["kv_heads"] * case["block"] * case["dim"] + 4 * case["kv_heads"]
        return {"bytes": 2 * 2 * per * case["pairs"] * case["layers"] + 16 * case["pairs"],
                "flops": 0}
    new, ctx = _lengths(case)
    H, K, D, bs = case["heads"], case["kv_heads"], case["dim"], case["block"]
    rows = sum(new)
    if case["op"] == "rope_append":
        scaled = case["cache"] == "scaled"
        touched = sum((c - 1) // bs - (c - n) // bs + 1 for n, c in zip(new, ctx))
        return {"bytes": rows * (H * D * 4 + K * D * 4 + K * D * 2 * (1 if scaled else 2)) +
                touched * (4 + (8 * K if scaled else 0)),
                "flops": rows * (H + K) * case["rot"] * 3}
    blocks = sum(-(-c // bs) for c in ctx)
    cache = sum(ctx) * K * D * 2 + blocks * (8 * K + 4)
    pairs = sum(n * (c - n) + n * (n + 1) // 2 for n, c in zip(new, ctx))
    return {"bytes": cache + rows * H * D * 4, "flops": 4 * pairs * H * D}


# ------------------------------------------------------------------ inputs

def _power_of_two(bound):
    """The smallest power of two s >= 2^-126 with bound <= 448 s (bound finite, >= 0)."""
    m, e = torch.frexp(bound)                     # bound = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-126)
    return torch.ldexp(torch.ones_like(bound), torch.where(bound > 0, e, torch.full_like(e, -126)))


def _random_cache(g, nb, K, bs, D):
    """Codes and scales of a cache of normal values whose size varies by KV head
    and channel (keys have a few channels far larger than the rest)."""
    dev = "cuda"
    scales = torch.empty(nb, K, 2, device=dev)
    out = []
    for i in range(2):
        codes = torch.empty(nb, K, bs, D, device=dev, dtype=F8)
        mag = torch.exp(0.5 * torch.randn(1, K, 1, 1, generator=g, device=dev))
        if i == 0:
            mag = mag * (1 + 3 * (torch.rand(1, K, 1, D, generator=g, device=dev) < 0.03))
        step = max(1, (1 << 27) // (K * bs * D))
        for j in range(0, nb, step):
            x = torch.randn(min(step, nb - j), K, bs, D, generator=g, device=dev) * mag
            s = _power_of_two(x.abs().amax((2, 3)))
            scales[j:j + step, :, i] = s
            codes[j:j + step] = (x / s[:, :, None, None]).to(F8)
        out.append(codes)
    return out[0], out[1], scales


def _inv_freq(case):
    """(inverse frequencies in 64 bits, factor on the rotated part): base 10000,
    as they are, positions divided by 4, or interpolated by parts (yarn) for a
    context 32 times the trained 4096 tokens."""
    r = case["rot"]
    f = 10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)
    if case["scaling"] == "linear":
        return f / 4, 1.0
    if case["scaling"] == "yarn":
        turns = 4096 * f / (2 * math.pi)
        keep = ((turns - 1) / (32 - 1)).clamp(0, 1)       # 1: kept, 0: divided by 32
        return f * keep + f / 32 * (1 - keep), 0.1 * math.log(32) + 1
    return f, 1.0


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = "cuda"
    if case["op"] == "copy":
        L, nb, K, bs, D = case["layers"], case["pool"], case["kv_heads"], case["block"], case["dim"]
        k, v, scales = _random_cache(g, L * nb, K, bs, D)
        order = torch.randperm(nb, generator=g, device=dev)
        n = case["pairs"]
        # sources may repeat (several samples leave one shared block)
        src = order[torch.randint(0, nb - n, (n,), generator=g, device=dev)]
        s = dict(case=case, k=k.view(L, nb, K, bs, D), v=v.view(L, nb, K, bs, D),
                 scales=scales.view(L, nb, K, 2),
                 pairs=torch.stack([src, order[nb - n:]], 1).contiguous())
        if own:  # the layers' descriptors, which an engine makes once
            import paged_kv_cache_130_gb300 as P
            s["P"] = P
            s["descs"] = [P.cache_desc(s["k"][i], s["v"][i]) for i in range(L)]
            s["layer_scales"] = [s["scales"][i] for i in range(L)]
        return s
    new, ctx = _lengths(case)
    S, H, K, D, bs = case["num_seqs"], case["heads"], case["kv_heads"], case["dim"], case["block"]
    dt = DTYPES[case["dtype"]]
    counts = [-(-c // bs) for c in ctx]
    nb = sum(counts) + 8
    order = torch.randperm(nb, generator=g, device=dev).to(torch.int32)
    tables = torch.full((S, max(counts)), -1, dtype=torch.int32, device=dev)
    at = 0
    for i, n in enumerate(counts):
        tables[i, :n] = order[at:at + n]
        at += n
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    rows = cu[-1]
    s = dict(case=case, tables=tables, ctx=torch.tensor(ctx, dtype=torch.int32, device=dev),
             cu=torch.tensor(cu, dtype=torch.int32, device=dev), max_new=max(new),
             max_ctx=max(ctx), scale=1 / math.sqrt(D))
    if case["op"] == "rope_append":
        # the fused projection's output: q, k and v of a token side by side
        qkv = torch.randn(rows, H + 2 * K, D, generator=g, device=dev)
        qkv = (qkv * torch.exp(0.5 * torch.randn(1, H + 2 * K, 1, generator=g, device=dev))).to(dt)
        s["q"], s["new_k"], s["new_v"] = qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:]
        f, s["mscale"] = _inv_freq(case)
        s["inv_freq"] = f.to(dev)
        if case["cache"] == "same":
            s["k"] = torch.randn(nb, K, bs, D, generator=g, device=dev).to(dt)
            s["v"] = torch.randn(nb, K, bs, D, generator=g, device=dev).to(dt)
            s["scales"] = None
        else:
            s["k"], s["v"], s["scales"] = _random_cache(g, nb, K, bs, D)
    else:
        s["k"], s["v"], s["scales"] = _random_cache(g, nb, K, bs, D)
        s["q"] = torch.randn(rows, H, D, generator=g, device=dev).to(dt)
    if own:  # the descriptor and the workspace, which an engine keeps
        import paged_kv_cache_130_gb300 as P
        s["P"] = P
        s["desc"] = P.cache_desc(s["k"], s["v"])
        if case["op"] == "decode":
            n = P.pkv_decode_scaled_workspace_bytes(s["desc"], S, H, s["max_ctx"])
            s["workspace"] = torch.empty(max(n, 1), dtype=torch.uint8, device=dev)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        P = s["P"]
        if op == "rope_append":
            q = P.pkv_rope_append(s["desc"], s["q"], s["new_k"], s["new_v"], s["inv_freq"], s["cu"],
                                  s["max_new"], s["tables"], s["ctx"], s["max_ctx"],
                                  interleaved=s["case"]["layout"] == "interleaved",
                                  mscale=s["mscale"], scales=s["scales"])
            return _cache_out(q, s)
        if op == "decode":
            return P.pkv_paged_attention_decode_scaled(s["desc"], s["scales"], s["q"], s["tables"],
                                                       s["ctx"], s["max_ctx"], s["scale"],
                                                       workspace=s["workspace"])
        if op == "prefill":
            return P.pkv_paged_attention_prefill_scaled(s["desc"], s["scales"], s["q"], s["cu"],
                                                        s["max_new"], s["tables"], s["ctx"],
                                                        s["max_ctx"], s["scale"])
        P.pkv_copy_blocks_scaled(s["descs"], s["layer_scales"], s["pairs"])
        return s["k"], s["v"], s["scales"]
    if op == "rope_append":
        return _plain_rope_append(s)
    if op == "decode":
        return _plain_decode(s)
    if op == "prefill":
        return _plain_prefill(s)
    src, dst = s["pairs"].unbind(1)
    for t in (_bytes(s["k"]), _bytes(s["v"]), s["scales"]):
        t[:, dst] = t[:, src]
    return s["k"], s["v"], s["scales"]


def _bytes(t):
    return t.view(torch.uint8)


def _cache_out(q, s):
    """The rotated q and the updated cache (its buffers)."""
    return (q, s["k"], s["v"]) if s["scales"] is None else (q, s["k"], s["v"], s["scales"])


def _row_positions(s):
    """Sequence and position of every new token's row."""
    row = torch.arange(s["q"].shape[0], device="cuda")
    cu = s["cu"].long()
    seq = torch.bucketize(row, cu[1:], right=True)
    return seq, s["ctx"].long()[seq] - cu[seq + 1] + row


def _rotate(x, cos, sin, r, interleaved):
    """Rotated copy of x [rows, heads, D] in 32 bits."""
    y = x.float().clone()
    a, b = (y[..., 0:r:2], y[..., 1:r:2]) if interleaved else (y[..., :r // 2], y[..., r // 2:r])
    na, nb = a * cos - b * sin, b * cos + a * sin
    a.copy_(na)
    b.copy_(nb)
    return y


def _to_codes(x, s):
    return (x / s).clamp(-F8_MAX, F8_MAX).to(F8)


def _plain_rope_append(s):
    case = s["case"]
    r, dt, bs = case["rot"], DTYPES[case["dtype"]], case["block"]
    seq, pos = _row_positions(s)
    # angles in 64 bits: a float's product is off by whole radians far out
    ang = pos.double()[:, None] * s["inv_freq"]
    cos = (torch.cos(ang) * s["mscale"]).float()[:, None]
    sin = (torch.sin(ang) * s["mscale"]).float()[:, None]
    inter = case["layout"] == "interleaved"
    q = _rotate(s["q"], cos, sin, r, inter).to(dt)
    k = _rotate(s["new_k"], cos, sin, r, inter)
    phys, off = s["tables"][seq, pos // bs].long(), pos % bs
    if s["scales"] is None:
        s["k"][phys, :, off] = k.to(dt)
        s["v"][phys, :, off] = s["new_v"]
        return _cache_out(q, s)
    # the blocks that the call writes, and their scales
    old = s["scales"]
    c = max(1.0, SQRT2_32 * abs(s["mscale"]))
    bound = torch.stack([s["new_k"].float().abs().amax(-1) * c, s["new_v"].float().abs().amax(-1)], -1)
    need = torch.zeros_like(old).index_reduce_(0, phys, bound, "amax")
    begun = torch.zeros(old.shape[0], device="cuda").index_add_(0, phys, (off == 0).float()) > 0
    touched = torch.zeros(old.shape[0], device="cuda").index_fill_(0, phys, 1.0) > 0
    need = _power_of_two(need)
    new = torch.where(begun[:, None, None], need, torch.maximum(old, need))
    new = torch.where(touched[:, None, None], new, old)
    # blocks that held tokens before: their codes follow the scale
    grow = torch.nonzero(touched & ~begun)[:, 0]
    for i, t in enumerate((s["k"], s["v"])):
        f = (old[grow, :, i] / new[grow, :, i])[..., None, None]
        _bytes(t)[grow] = _bytes((_bytes(t)[grow].view(F8).float() * f).to(F8))
    ks, vs = new[phys].unbind(-1)
    _bytes(s["k"])[phys, :, off] = _bytes(_to_codes(k, ks[..., None]))
    _bytes(s["v"])[phys, :, off] = _bytes(_to_codes(s["new_v"].float(), vs[..., None]))
    old.copy_(new)
    return _cache_out(q, s)


def _gather(s):
    """K and V of every sequence, [S, kv_heads, T, D] in 32 bits."""
    ids = s["tables"].long().clamp(min=0)
    out = []
    for i, t in enumerate((s["k"], s["v"])):
        x = _bytes(t)[ids].view(F8).float() * s["scales"][ids][..., i, None, None]
        out.append(x.transpose(1, 2).flatten(2, 3))          # [S, K, blocks * bs, D]
    return out


def _softmax_times(x, live, v):
    """softmax over the last axis of x where live, times v."""
    x = x.masked_fill(~live, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    return (p @ v) / torch.where(total > 0, total, torch.ones_like(total))


def _plain_decode(s):
    k, v = _gather(s)
    S, K, T, D = k.shape
    H = s["q"].shape[1]
    q = s["q"].float().view(S, K, H // K, D)
    x = (q @ k.transpose(2, 3)) * s["scale"]
    live = torch.arange(T, device="cuda") < s["ctx"].long()[:, None, None, None]
    return _softmax_times(x, live, v).view(S, H, D).to(s["q"].dtype)


def _plain_prefill(s):
    k, v = _gather(s)
    S, K, T, D = k.shape
    H, N = s["q"].shape[1], s["max_new"]
    seq, pos = _row_positions(s)
    j = torch.arange(s["q"].shape[0], device="cuda") - s["cu"].long()[seq]
    q = torch.zeros(S, N, H, D, device="cuda")
    q[seq, j] = s["q"].float()
    q = q.view(S, N, K, H // K, D).permute(0, 2, 3, 1, 4).reshape(S, K, -1, D)
    x = ((q @ k.transpose(2, 3)) * s["scale"]).view(S, K, H // K, N, T)
    last = torch.full((S, N), -1, device="cuda", dtype=torch.int64)
    last[seq, j] = pos
    live = torch.arange(T, device="cuda") <= last[:, None, None, :, None]
    o = _softmax_times(x, live, v[:, :, None])                # [S, K, G, N, D]
    return o.permute(0, 3, 1, 2, 4).reshape(S, N, H, D)[seq, j].to(s["q"].dtype)


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """The definition in 64 bits, one sequence at a time; codes of new tokens
    are given as the unrounded value over the scale."""
    s = prepare(case, seed)
    if case["op"] == "copy":
        src, dst = s["pairs"][:, 0], s["pairs"][:, 1]
        out = []
        for t in (s["k"], s["v"], s["scales"]):
            x = t.to(torch.float32)
            y = x.clone()
            for i in range(len(src)):
                y[:, dst[i]] = x[:, src[i]]
            out.append(y if t.dtype == F8 else y.double())
        return tuple(out)
    if case["op"] == "rope_append":
        return _exact_rope_append(case, s)
    cu, ctx = s["cu"].tolist(), s["ctx"].tolist()
    H, K, D, bs = case["heads"], case["kv_heads"], case["dim"], case["block"]
    out = torch.zeros(cu[-1], H, D, dtype=torch.float64, device="cuda")
    for i, c in enumerate(ctx):
        n = cu[i + 1] - cu[i]
        ids = s["tables"][i, :-(-c // bs)].long()
        for h in range(K):
            kv = []
            for w, t in enumerate((s["k"], s["v"])):
                x = t[:, h].view(torch.uint8)[ids].view(F8).double()
                kv.append((x * s["scales"][ids, h, w].double()[:, None, None]).reshape(-1, D)[:c])
            rows = s["q"][cu[i]:cu[i + 1], h * (H // K):(h + 1) * (H // K)].double()
            x = torch.einsum("ngd,td->ngt", rows, kv[0]) * s["scale"]
            t = torch.arange(c, device="cuda")
            hidden = t[None, :] > (c - n + torch.arange(n, device="cuda"))[:, None]
            x.masked_fill_(hidden[:, None, :], -math.inf)
            w = torch.exp(x - x.max(-1, keepdim=True).values)
            out[cu[i]:cu[i + 1], h * (H // K):(h + 1) * (H // K)] = torch.einsum(
                "ngt,td->ngd", w / w.sum(-1, keepdim=True), kv[1])
    return out


def _exact_rope_append(case, s):
    r, bs, K = case["rot"], case["block"], case["kv_heads"]
    cu, ctx = s["cu"].tolist(), s["ctx"].tolist()
    q, k, v = s["q"].double().clone(), s["new_k"].double().clone(), s["new_v"].double()
    m = s["mscale"]
    for i, c in enumerate(ctx):
        n = cu[i + 1] - cu[i]
        pos = torch.arange(c - n, c, device="cuda", dtype=torch.float64)
        z = torch.polar(torch.full((n, r // 2), m, dtype=torch.float64, device="cuda"),
                        pos[:, None] * s["inv_freq"][None])
        for t in (q, k):
            x = t[cu[i]:cu[i + 1], :, :r]
            pairs = x.reshape(n, -1, r // 2, 2) if case["layout"] == "interleaved" else \
                x.reshape(n, -1, 2, r // 2).transpose(2, 3)
            y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z[:, None])
            x.copy_((y if case["layout"] == "interleaved" else y.transpose(2, 3)).reshape(x.shape))
    ck = s["k"].to(torch.float64)
    cv = s["v"].to(torch.float64)
    scaled = s["scales"] is not None
    sc = s["scales"].double() if scaled else None
    c = max(1.0, math.sqrt(2.0) * abs(m))
    for i, n_ctx in enumerate(ctx):
        first = n_ctx - (cu[i + 1] - cu[i])
        ids = s["tables"][i].tolist()
        for b in range(first // bs, (n_ctx - 1) // bs + 1):
            lo, hi = max(first, b * bs), min(n_ctx, (b + 1) * bs)
            rows = slice(cu[i] + lo - first, cu[i] + hi - first)
            at = slice(lo - b * bs, hi - b * bs)
            for w, (t, x, raw, f) in enumerate(((ck, k, s["new_k"], c), (cv, v, s["new_v"], 1.0))):
                x = x[rows].transpose(0, 1)                    # [K, tokens, D]
                if not scaled:
                    t[ids[b], :, at] = x
                    continue
                amax = raw[rows].double().abs().amax((0, 2)) * f
                need = torch.exp2((torch.floor(torch.log2(amax)) - 8).clamp(min=-126))
                need = torch.where(448 * need < amax, 2 * need, need)
                new = need if lo == b * bs else torch.maximum(sc[ids[b], :, w], need)
                if lo > b * bs:
                    t[ids[b]] *= (sc[ids[b], :, w] / new)[:, None, None]
                sc[ids[b], :, w] = new
                t[ids[b], :, at] = x / new[:, None, None]
    q = q.contiguous()
    return (q, ck, cv) if not scaled else (q, ck, cv, sc)
