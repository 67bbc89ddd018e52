"""What is measured of the rotate-and-append, page-summary and block-sparse decode operators.

``own`` false: the operators in their plain form, elementary torch operations
in 32 bits (64 for the angles).  ``own`` true: the calls a user makes of
``paged_kv_cache_193_gb300.api``.  Both take what ``prepare`` gives.

Three kinds of case:

* ``append``: the position rotation of q and k over one or several position
  axes, and the write of k and v into the paged cache;
* ``summary``: the int8 bounds of every page that a batch of new tokens
  completes;
* ``sparse``: for every sequence and KV head, the choice of ``top_k`` pages by
  the bound of q . k over each page, and the attention of the new token over
  the chosen pages.
"""
import math

import torch

own = False

DEVICE = "cuda"


def listed():
    return [
        # one new token of one sequence: the latency of a single decode step
        _append("append-1", tokens=1, q_heads=32, kv_heads=8),
        # a decode batch whose q, k and v rows are slices of one projection's output, E4M3 cache with a scale per head
        _append("append-256-e4m3", tokens=256, q_heads=64, kv_heads=8, cache="e4m3", per_head=True, fused=True),
        # a chunk of prompt tokens, bf16 cache
        _append("append-8192", tokens=8192, q_heads=32, kv_heads=8, fused=True),
        # prompt tokens of images: three axes, adjacent pairs, part of the head dim turned, an odd count, padded rows
        _append("append-axes-4109", tokens=4109, q_heads=16, kv_heads=16, head_dim=64, block=32, rotary=48, axes=3,
                adjacent=True, padded=13),
        # a decode batch: one token in `block` completes a page
        _summary("summary-256", tokens=256, kv_heads=8),
        # a long chunk of prompt tokens: every page of it is completed, E4M3 cache
        _summary("summary-16384-e4m3", tokens=16384, kv_heads=8, cache="e4m3"),
        # one sequence of a few thousand tokens: latency
        _sparse("sparse-1", seqs=1, low=5003, high=5003, q_heads=32, kv_heads=8, top_k=64),
        # a decode batch of short contexts: half the pages or fewer are read
        _sparse("sparse-256", seqs=256, low=512, high=2048, q_heads=32, kv_heads=8, top_k=32),
        # long contexts, eight query heads to a KV head
        _sparse("sparse-64-long", seqs=64, low=4096, high=32768, q_heads=64, kv_heads=8, top_k=128),
        # ragged contexts down to one token, E4M3 cache of 32-token pages with a scale per head
        _sparse("sparse-64-e4m3", seqs=64, low=1, high=32768, q_heads=32, kv_heads=8, top_k=64, block=32, cache="e4m3",
                per_head=True),
        # head dim 64, one query head to a KV head, an odd number of pages
        _sparse("sparse-17-d64", seqs=17, low=1, high=9001, q_heads=16, kv_heads=16, top_k=25, head_dim=64),
        # a few very long contexts, sixteen query heads to a KV head
        _sparse("sparse-8-128k", seqs=8, low=131072, high=131072, q_heads=128, kv_heads=8, top_k=256),
    ]


def _append(name, tokens, q_heads, kv_heads, head_dim=128, block=16, cache="bf16", per_head=False, fused=False, rotary=0,
            axes=1, adjacent=False, padded=0):
    return {"name": name, "kind": "append", "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim,
            "block": block, "cache": cache, "per_head": per_head, "fused": fused, "rotary": rotary or head_dim, "axes": axes,
            "adjacent": adjacent, "padded": padded}


def _summary(name, tokens, kv_heads, head_dim=128, block=16, cache="bf16"):
    return {"name": name, "kind": "summary", "tokens": tokens, "kv_heads": kv_heads, "head_dim": head_dim, "block": block,
            "cache": cache}


def _sparse(name, seqs, low, high, q_heads, kv_heads, top_k, head_dim=128, block=16, cache="bf16", per_head=False, sink=1,
            recent=2):
    return {"name": name, "kind": "sparse", "seqs": seqs, "low": low, "high": high, "q_heads": q_heads, "kv_heads": kv_heads,
            "top_k": top_k, "head_dim": head_dim, "block": block, "cache": cache, "per_head": per_head, "sink": sink,
            "recent": recent}


def _spread(rng, low, high):
    """A whole number, its logarithm spread evenly over [low, high]."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    head_dim, block = rng.choice([64, 128]), rng.choice([16, 32])
    cache = rng.choice(["bf16", "e4m3"])
    per_head = cache == "e4m3" and rng.random() < 0.5
    kv_heads, group = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8, 16])
    kind = rng.choice(["append", "append", "summary", "sparse", "sparse", "sparse"])
    if kind == "append":
        group = min(group, 8)
        case = _append("", _spread(rng, 1, 8192), kv_heads * group, kv_heads, head_dim, block, cache, per_head,
                       rng.random() < 0.5, rng.choice([head_dim, head_dim, head_dim // 2, head_dim - 16]), rng.choice([1, 1, 2, 3, 4]),
                       rng.random() < 0.5, rng.choice([0, 0, 0, 5]))
    elif kind == "summary":
        case = _summary("", _spread(rng, 32, 16384), kv_heads, head_dim, block, cache)
    else:
        high = _spread(rng, 100, 65536)
        most = max(1, min(256, 64 * 16384 * 8 // (high * kv_heads)))
        seqs = _spread(rng, 1, most)
        low = rng.choice([1, high, max(1, high // 2), max(1, high // 8)])
        sink, recent = rng.choice([0, 1, 2]), rng.choice([1, 2, 3])
        case = _sparse("", seqs, low, high, kv_heads * group, kv_heads, _spread(rng, 8, 256), head_dim, block, cache, per_head,
                       sink, recent)
        while work(case)["bytes"] > 6e8:
            case["seqs"] = max(1, case["seqs"] // 2)
    del case["name"]
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _lengths(case):
    """The context lengths of a sparse case, spread evenly from low to high."""
    n, low, high = case["seqs"], case["low"], case["high"]
    return [high] if n == 1 else [low + (high - low) * i // (n - 1) for i in range(n)]


def _normal(gen, shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.float32) * scale).to(dtype)


def _pool(gen, blocks, heads, block, head_dim, cache, offset=None):
    """A cache [blocks, heads, block, head_dim] of normal values, in bf16 or as E4M3 codes, made a slice at a time."""
    dtype = torch.bfloat16 if cache == "bf16" else torch.float8_e4m3fn
    out = torch.empty(blocks, heads, block, head_dim, dtype=dtype, device=DEVICE)
    step = max(1, (1 << 27) // (heads * block * head_dim))
    for b in range(0, blocks, step):
        x = torch.randn(out[b:b + step].shape, generator=gen, device=DEVICE)
        if offset is not None:
            x += offset
        out[b:b + step] = (x if cache == "bf16" else x * 32.0).to(dtype)
    return out if cache == "bf16" else out.view(torch.uint8)


def _scales(gen, heads, per_head):
    """(kv_scale, k_scales, v_scales): E4M3 scales that put normal values well inside the format's range."""
    if not per_head:
        return 1.0 / 32, None, None
    k, v = (0.02 + 0.02 * torch.rand(heads, generator=gen, device=DEVICE) for _ in range(2))
    return 1.0, k, v


def _fused_or_not(gen, case, t, hq, hkv, d):
    if case["fused"]:  # one projection's rows, [q | k | v]
        rows = _normal(gen, (t, (hq + 2 * hkv) * d))
        q, k, v = rows.split([hq * d, hkv * d, hkv * d], dim=1)
        return q.view(t, hq, d), k.view(t, hkv, d), v.view(t, hkv, d)
    return _normal(gen, (t, hq, d)), _normal(gen, (t, hkv, d)), _normal(gen, (t, hkv, d))


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(int(seed))
    return {"append": _prepare_append, "summary": _prepare_summary, "sparse": _prepare_sparse}[case["kind"]](case, gen)


def _prepare_append(case, gen):
    t, hq, hkv, d, block = case["tokens"], case["q_heads"], case["kv_heads"], case["head_dim"], case["block"]
    pairs, axes = case["rotary"] // 2, case["axes"]
    q, k, v = _fused_or_not(gen, case, t, hq, hkv, d)
    blocks = (t + block - 1) // block + 4
    slots = torch.randperm(blocks * block, generator=gen, device=DEVICE)[:t].to(torch.int32)
    live = t - min(case["padded"], t - 1)
    slots[live:] = -1  # a padded batch's last rows
    first = torch.randint(0, 100000, (axes, 1), generator=gen, device=DEVICE)
    if axes == 1:  # positions of a prompt
        positions = (first + torch.arange(t, device=DEVICE)).to(torch.int32)
    else:  # time stands still while height and width walk over the image
        at = torch.arange(t, device=DEVICE)
        walk = [at // 4096, (at // 64) % 64, at % 64, at]
        positions = (first + torch.stack(walk[:axes])).to(torch.int32)
    inv_freq = 500000.0 ** (-torch.arange(pairs, dtype=torch.float64, device=DEVICE) / pairs)
    pair_axis = None if axes == 1 else (torch.arange(pairs, device=DEVICE) * axes // pairs).to(torch.int32)
    kv_scale, k_scales, v_scales = _scales(gen, hkv, case["per_head"])
    return {"kind": "append", "q": q, "k": k, "v": v, "positions": positions if axes > 1 else positions[0].contiguous(),
            "inv_freq": inv_freq, "pair_axis": pair_axis, "adjacent": case["adjacent"], "slots": slots,
            "k_cache": _pool(gen, blocks, hkv, block, d, case["cache"]),
            "v_cache": _pool(gen, blocks, hkv, block, d, case["cache"]),
            "kv_scale": kv_scale, "k_scales": k_scales, "v_scales": v_scales,
            "out": torch.empty(t, hq, d, dtype=torch.bfloat16, device=DEVICE)}


def _prepare_summary(case, gen):
    t, heads, block = case["tokens"], case["kv_heads"], case["block"]
    d = case["head_dim"]
    if t <= 512:  # decode: token i is row i % block of a page of its own
        blocks = t + 3
        page = torch.randperm(blocks, generator=gen, device=DEVICE)[:t]
        slots = page * block + torch.arange(t, device=DEVICE) % block
    else:  # a chunk: the pages one after the other
        blocks = (t + block - 1) // block + 3
        page = torch.randperm(blocks, generator=gen, device=DEVICE)
        at = torch.arange(t, device=DEVICE)
        slots = page[at // block] * block + at % block
    offset = torch.randn(heads, 1, d, generator=gen, device=DEVICE)
    k_cache = _pool(gen, blocks, heads, block, d, case["cache"], offset)
    return {"kind": "summary", "k_cache": k_cache, "slots": slots.to(torch.int32),
            "summary": torch.zeros(blocks, heads, 2, d, dtype=torch.int8, device=DEVICE),
            "exponents": torch.zeros(blocks, heads, dtype=torch.int8, device=DEVICE)}


def _prepare_sparse(case, gen):
    s, hq, hkv, d, block = case["seqs"], case["q_heads"], case["kv_heads"], case["head_dim"], case["block"]
    lengths = torch.tensor(_lengths(case), device=DEVICE)
    lengths = lengths[torch.randperm(s, generator=gen, device=DEVICE)]
    need = (lengths + block - 1) // block
    total, width = int(need.sum()), int(need.max())
    page = torch.randperm(total, generator=gen, device=DEVICE)
    start = torch.cumsum(need, 0) - need
    at = torch.arange(width, device=DEVICE)
    tables = torch.where(at < need[:, None], page[(start[:, None] + at).clamp(max=total - 1)], -1)
    # keys: a mean of its own for each channel, as rotated keys have
    k_cache = _pool(gen, total, hkv, block, d, case["cache"], torch.randn(hkv, 1, d, generator=gen, device=DEVICE))
    v_cache = _pool(gen, total, hkv, block, d, case["cache"])
    kv_scale, k_scales, v_scales = _scales(gen, hkv, case["per_head"])
    summary = torch.empty(total, hkv, 2, d, dtype=torch.int8, device=DEVICE)
    exponents = torch.empty(total, hkv, dtype=torch.int8, device=DEVICE)
    step = max(1, (1 << 27) // (hkv * block * d))
    for b in range(0, total, step):  # a user's program has these from the appends before
        summary[b:b + step], exponents[b:b + step] = _bounds(_values(k_cache[b:b + step]))
    return {"kind": "sparse", "q": _normal(gen, (s, hq, d)), "k_cache": k_cache, "v_cache": v_cache,
            "tables": tables.to(torch.int32), "lengths": lengths.to(torch.int32), "summary": summary, "exponents": exponents,
            "top_k": case["top_k"], "sink": case["sink"], "recent": case["recent"], "kv_scale": kv_scale,
            "k_scales": k_scales, "v_scales": v_scales, "softmax_scale": 1.0 / math.sqrt(d),
            "selected": torch.empty(s, hkv, case["top_k"], dtype=torch.int32, device=DEVICE),
            "counts": torch.empty(s, hkv, dtype=torch.int32, device=DEVICE),
            "out": torch.empty(s, hq, d, dtype=torch.bfloat16, device=DEVICE)}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    kind = state["kind"]
    if own:
        return {"append": _own_append, "summary": _own_summary, "sparse": _own_sparse}[kind](state)
    return {"append": _plain_append, "summary": _plain_summary, "sparse": _plain_sparse}[kind](state)


def _as_values(cache):
    """A cache as the values its bytes stand for (before the scale)."""
    return cache if cache.dtype == torch.bfloat16 else cache.view(torch.float8_e4m3fn)


def _own_append(st):
    from paged_kv_cache_193_gb300 import api
    out = api.rope_append(st["q"], st["k"], st["v"], st["positions"], st["inv_freq"], st["slots"], st["k_cache"], st["v_cache"],
                          pair_axis=st["pair_axis"], adjacent=st["adjacent"], kv_scale=st["kv_scale"], k_scales=st["k_scales"],
                          v_scales=st["v_scales"], out=st["out"])
    return {"q": out, "k_cache": _as_values(st["k_cache"]), "v_cache": _as_values(st["v_cache"])}


def _own_summary(st):
    from paged_kv_cache_193_gb300 import api
    api.block_summary(st["k_cache"], st["slots"], st["summary"], st["exponents"])
    return {"summary": st["summary"], "exponents": st["exponents"]}


def _own_sparse(st):
    from paged_kv_cache_193_gb300 import api
    api.sparse_attend(st["q"], st["k_cache"], st["v_cache"], st["summary"], st["exponents"], st["tables"], st["lengths"],
                      st["top_k"], sink_blocks=st["sink"], recent_blocks=st["recent"], softmax_scale=st["softmax_scale"],
                      kv_scale=st["kv_scale"], k_scales=st["k_scales"], v_scales=st["v_scales"], selected=st["selected"],
                      counts=st["counts"], out=st["out"])
    return {"selected": st["selected"], "counts": st["counts"], "out": st["out"]}


def _values(cache):
    return _as_values(cache).float()


def _plain_append(st):
    q, k, v, freq = st["q"], st["k"], st["v"], st["inv_freq"]
    pairs = freq.numel()
    positions = st["positions"].view(-1, q.shape[0])
    axis = torch.zeros(pairs, dtype=torch.int64, device=q.device) if st["pair_axis"] is None else st["pair_axis"].long()
    angle = positions[axis].T.double() * freq  # [tokens, pairs]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turn(x):
        x = x.float()
        y = x.clone()
        first, second = (slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)) if st["adjacent"] else (slice(0, pairs), slice(pairs, 2 * pairs))
        a, b = x[..., first], x[..., second]
        y[..., first] = a * cos - b * sin
        y[..., second] = a * sin + b * cos
        return y

    k_cache, v_cache = _as_values(st["k_cache"]), _as_values(st["v_cache"])
    block = k_cache.shape[2]
    new_k, new_v = turn(k), v.float()
    if k_cache.dtype != torch.bfloat16:
        k_scale, v_scale = (st["kv_scale"] if x is None else x[:, None] for x in (st["k_scales"], st["v_scales"]))
        new_k, new_v = (new_k / k_scale).clamp(-448, 448), (new_v / v_scale).clamp(-448, 448)
    kept = (st["slots"] >= 0).nonzero()[:, 0]
    slot = st["slots"][kept].long()
    bits = torch.int16 if k_cache.dtype == torch.bfloat16 else torch.uint8
    for cache, new in ((k_cache, new_k), (v_cache, new_v)):
        cache.view(bits)[slot // block, :, slot % block] = new.to(cache.dtype)[kept].view(bits)
    st["out"].copy_(turn(q))
    return {"q": st["out"], "k_cache": k_cache, "v_cache": v_cache}


def _power(e):
    """Two to the whole number e (-126 .. 127), from its bits."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _to_int8(x, amax):
    """x as whole numbers of at most 127 times two to a shared exponent, the least one that holds amax (in [-60, 40])."""
    part, exponent = torch.frexp(amax)
    e = exponent - 7 + (part * 128 > 127).to(exponent.dtype)
    e = torch.where(amax > 0, e, -60).clamp(-60, 40)
    return (x * _power(-e)[..., None]).round().clamp(-127, 127), e


def _bounds(x):
    """Of pages [..., block, d] in 32 bits: the int8 bounds [..., 2, d] (largest, least) and the exponents [...]."""
    fine = x.isfinite().flatten(-2).all(-1)
    x = torch.where(fine[..., None, None], x, 0.0)
    high, low = x.amax(-2), x.amin(-2)
    amax = torch.maximum(high.abs(), low.abs()).amax(-1)
    both, e = _to_int8(torch.cat([high, low], -1), amax)
    return both.to(torch.int8).unflatten(-1, (2, -1)), torch.where(fine, e, 127).to(torch.int8)


def _plain_summary(st):
    block = st["k_cache"].shape[2]
    ends = st["slots"][(st["slots"] >= 0) & (st["slots"] % block == block - 1)].long() // block
    st["summary"][ends], st["exponents"][ends] = _bounds(_values(st["k_cache"][ends]))
    return {"summary": st["summary"], "exponents": st["exponents"]}


def _plain_sparse(st):
    q, tables, n = st["q"], st["tables"].long(), st["lengths"].long()
    seqs, hq, d = q.shape
    _, hkv, block, _ = st["k_cache"].shape
    width, top_k = tables.shape[1], st["top_k"]
    # the score of every page: whole numbers throughout, so 32 bits hold them exactly
    x = q.float().view(seqs, hkv, hq // hkv, d)
    fine = x.isfinite().all(-1, keepdim=True)
    r, eq = _to_int8(torch.where(fine, x, 0.0), torch.where(fine, x, 0.0).abs().amax(-1))
    pages = tables.clamp(min=0)
    bounds = st["summary"][pages].permute(0, 2, 1, 3, 4).flatten(-2).float()  # [seqs, hkv, width, 2 d]
    dots = torch.cat([r.clamp(min=0), r.clamp(max=0)], -1) @ bounds.transpose(-1, -2)
    ej = st["exponents"][pages].permute(0, 2, 1).int()
    score = (dots * _power(eq)[..., None]).amax(2) * _power(ej)
    score = torch.where(ej == 127, torch.inf, score)
    # sink and recent pages come first, pages past the end never; ties go to the lower index
    at = torch.arange(width, device=q.device)
    have = ((n + block - 1) // block)[:, None]
    rank = torch.where(at < have, torch.where((at < st["sink"]) | (at >= have - st["recent"]), 2, 1), 0)[:, None].expand_as(score)
    order = torch.sort(torch.where(rank == 1, score, 0.0), dim=-1, descending=True, stable=True).indices
    order = order.gather(-1, torch.sort(rank.gather(-1, order), dim=-1, descending=True, stable=True).indices)
    chosen = order[..., :top_k]
    count = have.clamp(max=top_k).expand(seqs, hkv)
    chosen = torch.where(torch.arange(chosen.shape[-1], device=q.device) < count[..., None], chosen, width).sort(-1).values
    chosen = torch.nn.functional.pad(chosen, (0, top_k - chosen.shape[-1]), value=width)
    selected = torch.where(chosen < width, chosen, -1)
    # attention over the chosen pages
    page = tables.gather(1, selected.clamp(min=0).flatten(1)).view_as(selected).clamp(min=0)
    head = torch.arange(hkv, device=q.device)[:, None]
    k, v = (_as_values(c)[page, head] if c.dtype == torch.bfloat16 else c[page, head].view(torch.float8_e4m3fn)
            for c in (st["k_cache"], st["v_cache"]))  # [seqs, hkv, top_k, block, d]
    k_scale, v_scale = (1.0 if k.dtype == torch.bfloat16 else st["kv_scale"] if s is None else s[:, None, None]
                        for s in (st["k_scales"], st["v_scales"]))
    k, v = k.float().flatten(2, 3), v.float().flatten(2, 3)
    position = selected[..., None] * block + torch.arange(block, device=q.device)
    live = ((selected >= 0)[..., None] & (position < n[:, None, None, None])).flatten(2)[:, :, None]
    logit = (x @ k.transpose(-1, -2)) * (st["softmax_scale"] * k_scale)
    logit = torch.where(live, logit, -torch.inf)
    p = torch.exp(logit - logit.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min))
    p = torch.where(live, p, 0.0)
    total = p.sum(-1, keepdim=True)
    out = torch.where(total > 0, (p @ v) / torch.where(total > 0, total, 1.0) * v_scale, 0.0)
    st["selected"].copy_(selected)
    st["counts"].copy_(count)
    st["out"].copy_(out.view(seqs, hq, d))
    return {"selected": st["selected"], "counts": st["counts"], "out": st["out"]}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    d, block, elem = case["head_dim"], case["block"], 2 if case["cache"] == "bf16" else 1
    hkv = case["kv_heads"]
    if case["kind"] == "append":
        t, hq = case["tokens"], case["q_heads"]
        live = t - min(case["padded"], t - 1)
        moved = t * hq * d * 4 + live * hkv * d * 2 * (2 + elem)
        return {"bytes": moved + t * 4 * (1 + case["axes"]), "flops": 3 * case["rotary"] * (t * hq + live * hkv)}
    if case["kind"] == "summary":
        ends = case["tokens"] // block
        return {"bytes": ends * hkv * (block * d * elem + 2 * d + 1) + 4 * case["tokens"], "flops": 2 * ends * hkv * block * d}
    hq, top_k = case["q_heads"], case["top_k"]
    moved, flops = case["seqs"] * hq * d * 4, 0
    for n in _lengths(case):
        pages = -(-n // block)
        scored = max(0, pages - case["sink"] - case["recent"]) if pages > top_k else 0
        read = n if pages <= top_k else (top_k - 1) * block + (n - 1) % block + 1
        moved += hkv * (scored * (2 * d + 1) + read * 2 * d * elem + 4 * top_k) + 4 * pages
        flops += hq * (scored * 2 * d + read * 4 * d)
    return {"bytes": moved, "flops": flops}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, written apart from the plain forms
# ---------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "summary": _exact_summary, "sparse": _exact_sparse}[case["kind"]](st)


def _exact_append(st):
    t = st["q"].shape[0]
    freq = st["inv_freq"]
    pairs = freq.numel()
    positions = st["positions"].reshape(-1, t).double()
    axis = [0] * pairs if st["pair_axis"] is None else st["pair_axis"].tolist()
    angle = torch.stack([positions[a] * f for a, f in zip(axis, freq)], 1)
    unit = torch.polar(torch.ones_like(angle), angle)[:, None]  # a pair as a complex number, turned by a product

    def turned(x):
        x = x.double()
        part = x[..., :2 * pairs]
        pair = part.unflatten(-1, (pairs, 2)) if st["adjacent"] else part.unflatten(-1, (2, pairs)).transpose(-1, -2)
        y = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * unit)
        y = y.flatten(-2) if st["adjacent"] else y.transpose(-1, -2).flatten(-2)
        return torch.cat([y, x[..., 2 * pairs:]], -1)

    caches = []
    for name, new in (("k", turned(st["k"])), ("v", st["v"].double())):
        cache = _as_values(st[name + "_cache"])
        if cache.dtype != torch.bfloat16:
            s = st[name + "_scales"]
            new = (new / (st["kv_scale"] if s is None else s.double()[:, None])).clamp(-448.0, 448.0)
        block = cache.shape[2]
        rows = cache.double().transpose(1, 2).flatten(0, 1)  # by slot
        live = st["slots"] >= 0
        rows[st["slots"][live].long()] = new[live]
        caches.append(rows.unflatten(0, (-1, block)).transpose(1, 2).contiguous())
    return {"q": turned(st["q"]), "k_cache": caches[0], "v_cache": caches[1]}


def _exact_whole(x, dims):
    """Whole numbers of x [..., dims] and their unit, by doubling the least unit until it holds the largest."""
    top = x.abs().amax(dims, keepdim=True)
    unit = torch.full_like(top, 2.0 ** -60)
    for _ in range(100):
        unit = torch.where((top > 127 * unit) & (unit < 2.0 ** 40), unit * 2, unit)
    return (x / unit).round().clamp(-127, 127), unit


def _exact_summary(st):
    k = _as_values(st["k_cache"])
    block = k.shape[2]
    summary, exponents = st["summary"].clone(), st["exponents"].clone()
    done = sorted({s // block for s in st["slots"].tolist() if s >= 0 and s % block == block - 1})
    for i in range(0, len(done), 256):
        page = torch.tensor(done[i:i + 256], device=k.device)
        x = st["k_cache"][page]
        x = _as_values(x).double()
        both, unit = _exact_whole(torch.stack([x.max(2).values, x.min(2).values], 2), (2, 3))
        summary[page], exponents[page] = both.to(torch.int8), unit[..., 0, 0].log2().round().to(torch.int8)
    return {"summary": summary, "exponents": exponents}


def _exact_sparse(st):
    q = st["q"].double()
    seqs, hq, d = q.shape
    _, hkv, block, _ = st["k_cache"].shape
    top_k, group = st["top_k"], hq // hkv
    selected = torch.full((seqs, hkv, top_k), -1, dtype=torch.int32)
    counts = torch.zeros(seqs, hkv, dtype=torch.int32)
    out = torch.zeros(seqs, hq, d, dtype=torch.float64, device=q.device)
    ones = torch.ones(hkv, dtype=torch.float64, device=q.device)
    bf16 = st["k_cache"].dtype == torch.bfloat16
    k_scale, v_scale = (ones if bf16 else ones * st["kv_scale"] if s is None else s.double() for s in (st["k_scales"], st["v_scales"]))
    for s, n in enumerate(st["lengths"].tolist()):
        pages = -(-n // block)
        table = st["tables"][s, :pages].long()
        qs = q[s].view(hkv, group, 1, d)
        picks = [list(range(pages))] * hkv
        if pages > top_k:
            low, high = st["sink"], pages - st["recent"]
            bound = st["summary"][table[low:high]].double().permute(1, 0, 2, 3)[:, None]  # [hkv, 1, pages, 2, d]
            whole, unit = _exact_whole(qs, (3,))
            dot = torch.zeros(hkv, group, high - low, dtype=torch.float64, device=q.device)
            for g in range(group):
                dot[:, g] = torch.maximum(whole[:, g] * bound[:, 0, :, 0], whole[:, g] * bound[:, 0, :, 1]).sum(-1)
            size = torch.tensor([[2.0 ** int(e) for e in row] for row in st["exponents"][table[low:high]].T.tolist()],
                                dtype=torch.float64, device=q.device)
            score = (dot * unit[..., 0]).amax(1) * size
            best = torch.argsort(score, dim=-1, descending=True, stable=True)[:, :top_k - st["sink"] - st["recent"]].tolist()
            picks = [sorted(list(range(low)) + [low + j for j in b] + list(range(high, pages))) for b in best]
        pick = torch.tensor(picks, dtype=torch.int64)
        counts[s] = pick.shape[1]
        selected[s, :, :pick.shape[1]] = pick.to(torch.int32)
        if not n:
            continue
        pick = pick.to(q.device)
        head = torch.arange(hkv, device=q.device)[:, None]
        k, v = (_as_values(c[table[pick], head]).double().flatten(1, 2) for c in (st["k_cache"], st["v_cache"]))
        dead = (pick[..., None] * block + torch.arange(block, device=q.device)).flatten(1) >= n
        logit = torch.einsum("hgd,htd->hgt", qs[:, :, 0], k) * (st["softmax_scale"] * k_scale)[:, None, None]
        p = torch.softmax(logit.masked_fill(dead[:, None], -torch.inf), -1)
        out[s] = (torch.einsum("hgt,htd->hgd", p, v) * v_scale[:, None, None]).reshape(hq, d)
    return {"selected": selected.to(q.device), "counts": counts.to(q.device), "out": out}
