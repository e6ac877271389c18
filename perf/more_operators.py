"""The operators that share and shrink long contexts, as a program of plain torch
operations and as calls of the library.

Four operators of a serving engine's layer:

* ``shared``: one query token per sequence attends over the scaled 8-bit cache,
  where groups of sequences share their leading blocks (forked samples, a common
  system prompt);
* ``weights``: the attention weights of each sequence's last rows, summed over
  rows and the query heads of a KV head, added to a running total per token;
* ``decode``: a decode step over the scaled cache that adds its own weights;
* ``evict``: every KV head keeps the tokens of largest total (and the first and
  the last ones), moved to blocks of their own.

A scaled cache holds ``torch.float8_e4m3fn`` codes [num_blocks, kv_heads,
block_size, head_dim] and float32 scales [num_blocks, kv_heads, 2] (K, V); a
value is its code times its scale.  Totals are float32 [num_seqs, kv_heads,
width], entry t for token t of the sequence's context.
"""
import math
import random

import torch

own = False

F8 = torch.float8_e4m3fn
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases

def _shared(name, **kw):
    c = dict(name=name, op="shared", groups=1, members=1, prefix_lo=1, prefix_hi=1, own_lo=1,
             own_hi=1, heads=8, kv_heads=8, dim=128, block=16, dtype="bf16", lens=1)
    c.update(kw)
    return c


def _weights(name, **kw):
    c = dict(name=name, op="weights", num_seqs=1, window=1, new_lo=1, new_hi=1, cached_lo=0,
             cached_hi=0, heads=8, kv_heads=8, dim=128, block=16, dtype="bf16", cache="scaled",
             lens=1)
    c.update(kw)
    return c


def _decode(name, **kw):
    c = dict(name=name, op="decode", num_seqs=1, ctx_lo=1, ctx_hi=1, heads=8, kv_heads=8, dim=128,
             block=16, dtype="bf16", lens=1)
    c.update(kw)
    return c


def _evict(name, **kw):
    c = dict(name=name, op="evict", num_seqs=1, ctx_lo=1, ctx_hi=1, keep=1, first=0, last=0,
             kv_heads=8, dim=128, block=16, cache="scaled", dtype="bf16", lens=1)
    c.update(kw)
    return c


def listed():
    return [
        # two prompts of a small model with three samples each: latency
        _shared("shared_tiny", groups=2, members=3, prefix_lo=32, prefix_hi=40, own_lo=1, own_hi=70,
                heads=8, kv_heads=8, dim=64, dtype="f16"),
        # parallel sampling: 16 prompts of 504 tokens, six samples each
        _shared("shared_parallel_sampling", groups=16, members=6, prefix_lo=504, prefix_hi=504,
                own_lo=16, own_hi=512, heads=32, kv_heads=32, dtype="f16"),
        # 64 requests behind one long system prompt, a Llama-2-70B layer
        _shared("shared_system_prompt", groups=1, members=64, prefix_lo=8192, prefix_hi=8192,
                own_lo=64, own_hi=1024, heads=64, kv_heads=8),
        # the last rows of a short prompt, cache kept in fp16: latency
        _weights("weights_tiny", window=16, new_lo=37, new_hi=37, cached_lo=300, cached_hi=300,
                 heads=32, kv_heads=8, dtype="f16", cache="same"),
        # the last 32 rows of long prompts of a Llama-2-70B layer
        _weights("weights_long_prompts", num_seqs=4, window=32, new_lo=512, new_hi=512,
                 cached_lo=16384, cached_hi=32768, heads=64, kv_heads=8),
        # the last 64 rows of whole prompts of a Llama-2-7B layer, cache kept in bf16
        _weights("weights_prompts_16bit", num_seqs=8, window=64, new_lo=512, new_hi=2048, heads=32,
                 kv_heads=32, cache="same"),
        # one decode step of a small model: latency
        _decode("decode_tiny", num_seqs=4, ctx_lo=5, ctx_hi=64, dim=64, dtype="f16"),
        # a Llama-2-70B layer's decode step
        _decode("decode_gqa", num_seqs=64, ctx_lo=1024, ctx_hi=4096, heads=64, kv_heads=8),
        # a Llama-2-7B layer over long contexts, block size 32
        _decode("decode_long", num_seqs=16, ctx_lo=8192, ctx_hi=32768, heads=32, kv_heads=32,
                block=32),
        # two short contexts of a small model, cache kept in fp16: latency
        _evict("evict_small_16bit", num_seqs=2, ctx_lo=300, ctx_hi=700, keep=256, first=4, last=64,
               kv_heads=8, dim=64, cache="same", dtype="f16"),
        # a batch whose contexts grew past their budget sheds what weighed least
        _evict("evict_budget", num_seqs=64, ctx_lo=1500, ctx_hi=2600, keep=2048, first=4, last=256),
        # long prompts shrink to an eighth or less once they have been read
        _evict("evict_long_prompts", num_seqs=4, ctx_lo=16384, ctx_hi=32768, keep=2048, first=4,
               last=32),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["shared", "weights", "decode", "evict"])
    dim, block = rng.choice([64, 128, 128]), rng.choice([8, 16, 16, 32])
    dtype, lens = rng.choice(["f16", "bf16"]), rng.randrange(1, 1 << 20)
    kv = rng.choice([1, 2, 4, 5, 8, 16, 32])
    group = rng.choice([1, 1, 2, 3, 4, 7, 8, 16])
    if kv * group > 64:
        group = max(1, 64 // kv)
    heads = kv * group
    common = dict(heads=heads, kv_heads=kv, dim=dim, block=block, dtype=dtype, lens=lens)
    if op == "shared":
        groups = _log_int(rng, 1, 24)
        members = _log_int(rng, 1, 96 // groups)
        hi = _log_int(rng, 1, 1024)
        budget = 96 * 1024 * 32 // (kv * groups)          # tokens a group reads, all heads alike
        prefix = _log_int(rng, 1, max(1, min(8192, budget - members * hi)))
        c = _shared("", groups=groups, members=members, prefix_lo=max(1, prefix // 2),
                    prefix_hi=prefix, own_lo=max(1, hi // rng.randint(1, 8)), own_hi=hi, **common)
    elif op == "weights":
        seqs = _log_int(rng, 1, 8)
        window = _log_int(rng, 1, 64)
        new = _log_int(rng, 1, 2048)
        room = 4 * 33000 * 64 * 32 // (seqs * heads * window)
        cached = rng.choice([0, _log_int(rng, 1, max(1, min(32000, room)))])
        c = _weights("", num_seqs=seqs, window=window, new_lo=max(1, new // rng.randint(1, 4)),
                     new_hi=new, cached_lo=cached // 2, cached_hi=cached,
                     cache=rng.choice(["scaled", "same"]), **common)
    elif op == "decode":
        seqs = _log_int(rng, 1, 64)
        total = _log_int(rng, seqs, 300000 * 32 * 128 // (kv * dim))
        hi = max(1, min(40000, total // seqs))
        c = _decode("", num_seqs=seqs, ctx_lo=max(1, hi // rng.randint(1, 8)), ctx_hi=hi, **common)
    else:
        seqs = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, max(1, min(33000, 160000 * 8 // (seqs * kv))))
        keep = max(1, int(hi * rng.uniform(0.05, 1.1)))
        del common["heads"]
        c = _evict("", num_seqs=seqs, ctx_lo=max(1, hi // rng.randint(1, 4)), ctx_hi=hi, keep=keep,
                   first=rng.choice([0, 1, 4, 16]), last=rng.choice([0, 1, _log_int(rng, 1, keep + 1)]),
                   cache=rng.choice(["scaled", "scaled", "same"]), **common)
    del c["name"]
    return c


def _lengths(case):
    """(prefix, new tokens, tokens after the step) of every sequence."""
    r = random.Random(case["lens"])
    if case["op"] == "shared":
        pre, ctx = [], []
        for _ in range(case["groups"]):
            p = r.randint(case["prefix_lo"], case["prefix_hi"]) // case["block"] * case["block"]
            for _ in range(case["members"]):
                pre.append(p)
                ctx.append(p + r.randint(case["own_lo"], case["own_hi"]))
        return pre, [1] * len(ctx), ctx
    S = case["num_seqs"]
    if case["op"] == "weights":
        new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(S)]
        return [0] * S, new, [n + r.randint(case["cached_lo"], case["cached_hi"]) for n in new]
    return [0] * S, [1] * S, [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(S)]


def _element(case):
    return 1 if case.get("cache", "scaled") == "scaled" else 2


def work(case):
    pre, new, ctx = _lengths(case)
    K, D, bs, e = case["kv_heads"], case["dim"], case["block"], _element(case)
    per_block = 4 + (8 * K if e == 1 else 0)                  # its id and its scales
    if case["op"] == "evict":
        kept = [min(c, case["keep"]) for c in ctx]
        blocks = sum(-(-c // bs) for c in ctx) + sum(-(-n // bs) for n in kept)
        return {"bytes": sum(ctx) * K * 4 + len(ctx) * K * max(ctx) * 4 + 4 * sum(kept) * K * D * e +
                blocks * per_block, "flops": 0}
    H = case["heads"]
    if case["op"] == "shared":
        once = pre[::case["members"]]
        tokens = sum(once) + sum(c - p for c, p in zip(ctx, pre))
        return {"bytes": tokens * K * D * 2 + -(-tokens // bs) * per_block + len(ctx) * H * D * 4,
                "flops": 4 * sum(ctx) * H * D}
    blocks = sum(-(-c // bs) for c in ctx)
    if case["op"] == "decode":
        return {"bytes": sum(ctx) * K * (D * 2 + 8) + blocks * per_block + len(ctx) * H * D * 4,
                "flops": 4 * sum(ctx) * H * D}
    rows = [min(n, case["window"]) for n in new]
    pairs = sum(m * (c - m) + m * (m + 1) // 2 for m, c in zip(rows, ctx))
    return {"bytes": sum(ctx) * K * (D * e + 8) + blocks * per_block + sum(rows) * H * D * 2,
            "flops": 2 * pairs * H * D}


# ------------------------------------------------------------------ inputs

def _power_of_two(bound):
    """The smallest power of two s >= 2^-126 with bound <= 448 s (bound finite, >= 0)."""
    m, e = torch.frexp(bound)                     # bound = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-126)
    return torch.ldexp(torch.ones_like(bound), torch.where(bound > 0, e, torch.full_like(e, -126)))


def _random_cache(g, nb, K, bs, D, dtype):
    """A cache of normal values whose size varies by KV head and channel (keys
    have a few channels far larger than the rest): of `dtype`, or (None) codes
    and scales."""
    dev = "cuda"
    scales = torch.empty(nb, K, 2, device=dev) if dtype is None else None
    out = []
    for i in range(2):
        t = torch.empty(nb, K, bs, D, device=dev, dtype=F8 if dtype is None else dtype)
        mag = torch.exp(0.5 * torch.randn(1, K, 1, 1, generator=g, device=dev))
        if i == 0:
            mag = mag * (1 + 3 * (torch.rand(1, K, 1, D, generator=g, device=dev) < 0.03))
        step = max(1, (1 << 27) // (K * bs * D))
        for j in range(0, nb, step):
            x = torch.randn(min(step, nb - j), K, bs, D, generator=g, device=dev) * mag
            if dtype is None:
                s = _power_of_two(x.abs().amax((2, 3)))
                scales[j:j + step, :, i] = s
                t[j:j + step] = (x / s[:, :, None, None]).to(F8)
            else:
                t[j:j + step] = x.to(dtype)
        out.append(t)
    return out[0], out[1], scales


def _totals(g, S, K, width, ctx):
    """Totals of earlier steps: heavy tails, many tokens that never weighed
    anything, equal ones among the rest; zeros behind each context."""
    w = torch.exp(2.5 * torch.randn(S, K, width, generator=g, device="cuda") - 4)
    w = torch.where(torch.rand(S, K, width, generator=g, device="cuda") < 0.1,
                    torch.round(w * 8) / 8, w)
    return w * (torch.arange(width, device="cuda") < ctx[:, None, None])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = "cuda"
    pre, new, ctx = _lengths(case)
    S, K, D, bs = len(ctx), case["kv_heads"], case["dim"], case["block"]
    dt = DTYPES[case["dtype"]]
    shared_blocks = sum(p // bs for p in pre[::case.get("members", 1)])
    own_blocks = sum(-(-(c - p) // bs) for c, p in zip(ctx, pre))
    kept = [min(c, case["keep"]) for c in ctx] if case["op"] == "evict" else []
    nb = shared_blocks + own_blocks + sum(-(-n // bs) for n in kept) + 8
    order = torch.randperm(nb, generator=g, device=dev).to(torch.int32)
    tables = torch.full((S, max(-(-c // bs) for c in ctx)), -1, dtype=torch.int32, device=dev)
    at = 0
    for i in range(S):
        p, n = pre[i] // bs, -(-ctx[i] // bs)
        if p and i % case["members"]:
            tables[i, :p] = tables[i - 1, :p]
        else:
            tables[i, :p] = order[at:at + p]
            at += p
        tables[i, p:n] = order[at:at + n - p]
        at += n - p
    s = dict(case=case, tables=tables, ctx=torch.tensor(ctx, dtype=torch.int32, device=dev),
             max_ctx=max(ctx), scale=1 / math.sqrt(D))
    s["k"], s["v"], s["scales"] = _random_cache(g, nb, K, bs, D, None if _element(case) == 1 else dt)
    if case["op"] != "shared":
        s["totals"] = _totals(g, S, K, s["max_ctx"], s["ctx"])
    if case["op"] == "evict":
        s["keep"] = torch.full((S,), case["keep"], dtype=torch.int32, device=dev)
        s["dst"] = torch.full((S, -(-max(kept) // bs)), -1, dtype=torch.int32, device=dev)
        for i, m in enumerate(kept):
            n = -(-m // bs)
            s["dst"][i, :n] = order[at:at + n]
            at += n
    else:
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        s["q"] = torch.randn(cu[-1], case["heads"], D, generator=g, device=dev).to(dt)
    if case["op"] == "shared":
        m = case["members"]
        s["begin"] = torch.arange(0, S + 1, m, dtype=torch.int32, device=dev)
        s["prefix"] = torch.tensor([p // bs for p in pre[::m]], dtype=torch.int32, device=dev)
        s["max_prefix"] = max(pre) // bs
    if own:  # the descriptor and the workspace, which an engine keeps
        import paged_kv_cache_130_gb300 as P
        s["P"] = P
        s["desc"] = P.cache_desc(s["k"], s["v"])
        if case["op"] == "shared":
            n = P.pkv_decode_scaled_shared_prefix_workspace_bytes(
                s["desc"], S, case["heads"], case["groups"], case["members"], s["max_ctx"])
        elif case["op"] == "weights":
            n = P.pkv_attention_weights_workspace_bytes(s["desc"], S, case["heads"], case["window"],
                                                        s["max_ctx"])
        elif case["op"] == "decode":
            n = P.pkv_decode_scaled_weights_workspace_bytes(s["desc"], S, case["heads"], s["max_ctx"])
        else:
            n = P.pkv_evict_workspace_bytes(s["desc"], S, case["keep"], s["max_ctx"])
        s["workspace"] = torch.empty(max(n, 1), dtype=torch.uint8, device=dev)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    if own:
        P = s["P"]
        if case["op"] == "shared":
            return P.pkv_paged_attention_decode_scaled_shared_prefix(
                s["desc"], s["scales"], s["q"], s["tables"], s["ctx"], s["max_ctx"], s["begin"],
                s["prefix"], case["members"], s["max_prefix"], s["scale"], workspace=s["workspace"])
        if case["op"] == "weights":
            return P.pkv_attention_weights(
                s["desc"], s["q"], s["cu"], case["window"], s["tables"], s["ctx"], s["max_ctx"],
                s["scale"], s["totals"], scales=s["scales"], workspace=s["workspace"])
        if case["op"] == "decode":
            out = P.pkv_paged_attention_decode_scaled_weights(
                s["desc"], s["scales"], s["q"], s["tables"], s["ctx"], s["max_ctx"], s["scale"],
                s["totals"], workspace=s["workspace"])
            return out, s["totals"]
        lens, totals = P.pkv_evict(
            s["desc"], s["tables"], s["ctx"], s["max_ctx"], s["totals"], s["keep"], case["keep"],
            case["first"], case["last"], s["dst"], scales=s["scales"], workspace=s["workspace"])
        return _evict_out(s, lens, totals)
    if case["op"] == "shared":
        return _plain_decode(s)[0]
    if case["op"] == "weights":
        return _plain_weights(s)
    if case["op"] == "decode":
        out, w = _plain_decode(s)
        s["totals"] += w
        return out, s["totals"]
    return _plain_evict(s)


def _evict_out(s, lens, totals):
    """The cache (its buffers), lengths and totals after an eviction."""
    out = (s["k"], s["v"], lens, totals)
    return out if s["scales"] is None else out + (s["scales"],)


def _gather(s, i):
    """K (i = 0) or V of every sequence, [S, kv_heads, T, D] in 32 bits."""
    ids = s["tables"].long().clamp(min=0)
    t = (s["k"], s["v"])[i]
    if s["scales"] is None:
        x = t[ids].float()
    else:
        x = t.view(torch.uint8)[ids].view(F8).float() * s["scales"][ids][..., i, None, None]
    return x.transpose(1, 2).flatten(2, 3)                   # [S, K, blocks * bs, D]


def _softmax(x, live):
    """softmax over the last axis of x where live, 0 elsewhere."""
    x = x.masked_fill(~live, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total > 0, total, torch.ones_like(total))


def _plain_decode(s):
    """Attention and the weights of every token, summed over query heads."""
    k, v = _gather(s, 0), _gather(s, 1)
    S, K, T, D = k.shape
    H = s["q"].shape[1]
    q = s["q"].float().view(S, K, H // K, D)
    live = torch.arange(T, device="cuda") < s["ctx"].long()[:, None, None, None]
    p = _softmax((q @ k.transpose(2, 3)) * s["scale"], live)
    return (p @ v).view(S, H, D).to(s["q"].dtype), p.sum(2)[..., :s["max_ctx"]]


def _plain_weights(s):
    k = _gather(s, 0)
    S, K, T, D = k.shape
    H = s["q"].shape[1]
    cu, ctx = s["cu"].long(), s["ctx"].long()
    # the last rows of every sequence, in front of which some are empty
    j = torch.arange(-s["case"]["window"], 0, device="cuda")
    row = cu[1:, None] + j
    real = row >= cu[:-1, None]
    q = s["q"][row.clamp(min=0)].float() * real[..., None, None]
    q = q.view(S, -1, K, H // K, D).permute(0, 2, 3, 1, 4).reshape(S, K, -1, D)
    x = ((q @ k.transpose(2, 3)) * s["scale"]).view(S, K, H // K, -1, T)
    last = torch.where(real, ctx[:, None] + j, torch.full_like(row, -1))
    live = torch.arange(T, device="cuda") <= last[:, None, None, :, None]
    s["totals"] += _softmax(x, live).sum((2, 3))[..., :s["max_ctx"]]
    return s["totals"]


def _plain_evict(s):
    case, w, ctx = s["case"], s["totals"], s["ctx"].long()
    S, K, W = w.shape
    bs = case["block"]
    n = torch.minimum(ctx, s["keep"].long())
    last = n.clamp(max=case["last"])
    first = (n - last).clamp(max=case["first"])
    t = torch.arange(W, device="cuda")
    inside = t < ctx[:, None]
    always = inside & ((t < first[:, None]) | (t >= (ctx - last)[:, None]))
    # candidates in order of weight, the lower index first where they are equal
    key = torch.where(w.isnan(), torch.full_like(w, -math.inf), w)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    rank = inside[:, None].expand_as(w).gather(2, order).long()
    rank = rank * 2 + always[:, None].expand_as(w).gather(2, order).long()     # 3, 2 or 0
    order = order.gather(2, torch.sort(rank, dim=-1, descending=True, stable=True).indices)
    m = min(case["keep"], W)
    live = torch.arange(m, device="cuda") < n[:, None]
    idx = torch.where(live[:, None], order[..., :m], torch.full_like(order[..., :m], W))
    idx = torch.sort(idx, dim=-1).values                                       # [S, K, m]
    totals = torch.zeros_like(w)
    totals[..., :m] = torch.where(live[:, None], w.gather(2, idx.clamp(max=W - 1)), totals[..., :m])
    # every kept token of every head: where it comes from, where it goes
    si, ki, ri = torch.nonzero(live[:, None].expand(S, K, m), as_tuple=True)
    at = idx[si, ki, ri]
    src, dst = s["tables"][si, at // bs].long(), s["dst"][si, ri // bs].long()
    for i, c in enumerate((s["k"], s["v"])):
        if s["scales"] is None:
            c[dst, ki, ri % bs] = c[src, ki, at % bs]
            continue
        old = s["scales"][src, ki, i]
        flat = dst * K + ki
        new = torch.zeros(s["scales"].shape[0] * K, device="cuda").index_reduce_(0, flat, old, "amax")
        x = c.view(torch.uint8)[src, ki, at % bs].view(F8).float() * (old / new[flat])[:, None]
        c.view(torch.uint8)[dst, ki, ri % bs] = x.to(F8).view(torch.uint8)
        s["scales"][dst, ki, i] = new[flat]
    return _evict_out(s, n.to(torch.int32), totals)


# ------------------------------------------------------------------ 64 bits

def _values(case, s, i, h, w, c):
    """Tokens 0..c-1 of sequence i, KV head h, of K (w = 0) or V in 64 bits."""
    ids = s["tables"][i, :-(-c // case["block"])].long()
    t = (s["k"], s["v"])[w][:, h]
    if s["scales"] is None:
        return t[ids].double().reshape(-1, case["dim"])[:c]
    x = t.view(torch.uint8)[ids].view(F8).double() * s["scales"][ids, h, w].double()[:, None, None]
    return x.reshape(-1, case["dim"])[:c]


def exact(case, seed):
    """The definition in 64 bits, one sequence and KV head at a time; moved codes
    are given as the unrounded value over the scale."""
    s = prepare(case, seed)
    if case["op"] == "evict":
        return _exact_evict(case, s)
    K = case["kv_heads"]
    G = case["heads"] // K
    cu, ctx = s["cu"].tolist(), s["ctx"].tolist()
    out = torch.zeros(cu[-1], case["heads"], case["dim"], dtype=torch.float64, device="cuda")
    totals = s["totals"].double() if "totals" in s else None
    for i, c in enumerate(ctx):
        n = min(cu[i + 1] - cu[i], case.get("window", 1))
        rows = slice(cu[i + 1] - n, cu[i + 1])
        t = torch.arange(c, device="cuda")
        hidden = t[None, :] > (c - n + torch.arange(n, device="cuda"))[:, None]
        for h in range(K):
            q = s["q"][rows, h * G:(h + 1) * G].double()
            x = torch.einsum("ngd,td->ngt", q, _values(case, s, i, h, 0, c)) * s["scale"]
            x.masked_fill_(hidden[:, None, :], -math.inf)
            w = torch.exp(x - x.max(-1, keepdim=True).values)
            w = w / w.sum(-1, keepdim=True)
            if totals is not None:
                totals[i, h, :c] += w.sum((0, 1))
            if case["op"] != "weights":
                out[rows, h * G:(h + 1) * G] = torch.einsum("ngt,td->ngd", w,
                                                            _values(case, s, i, h, 1, c))
    return {"shared": out, "weights": totals, "decode": (out, totals)}[case["op"]]


def _exact_evict(case, s):
    bs, K, W = case["block"], case["kv_heads"], s["totals"].shape[2]
    ck, cv = s["k"].to(torch.float64), s["v"].to(torch.float64)
    sc = s["scales"].double() if s["scales"] is not None else None
    totals = torch.zeros_like(s["totals"], dtype=torch.float64)
    lens = []
    for i, c in enumerate(s["ctx"].tolist()):
        n = min(c, case["keep"])
        lens.append(n)
        last = min(case["last"], n)
        first = min(case["first"], n - last)
        for h in range(K):
            w = s["totals"][i, h, :c].double()
            # whoever beats a token: a larger total, or an equal one before it
            middle = w[first:c - last]
            by = torch.argsort(-middle, stable=True)[:n - first - last] + first
            kept = torch.cat([torch.arange(first, device="cuda"), by.sort().values,
                              torch.arange(c - last, c, device="cuda")])
            totals[i, h, :n] = w[kept]
            block = torch.arange(n, device="cuda") // bs
            to, src = s["dst"][i].long()[block], s["tables"][i].long()[kept // bs]
            for j, t in enumerate((ck, cv)):
                x = t[src, h, kept % bs]
                if sc is not None:
                    old = sc[src, h, j]
                    most = torch.stack([old[b:b + bs].max() for b in range(0, n, bs)])[block]
                    x = x * (old / most)[:, None]
                    sc[to, h, j] = most
                t[to, h, torch.arange(n, device="cuda") % bs] = x
    lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    return (ck, cv, lens, totals) if sc is None else (ck, cv, lens, totals, sc)
