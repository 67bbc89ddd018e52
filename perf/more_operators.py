"""What is measured of the normalised rotate-and-append, shared-prefix decode and cross-attention operators.

``own`` false: the operators in their plain form, elementary torch operations
in 32 bits (64 for the angles).  ``own`` true: the calls a user makes of
``paged_kv_cache_193_gb300.api``.  Both take what ``prepare`` gives.

Three kinds of case:

* ``norm``: the root-mean-square norm of every head's q and k row with its
  weights, the position rotation, and the write of k and v into the paged
  cache;
* ``shared``: decode attention of a batch whose sequences, in groups, have the
  first pages of their contexts in common;
* ``cross``: attention of each sequence's rows (one decoded token, the rows of
  several beams, or a chunk) to all of an encoder's states in the paged cache.
"""
import math

import torch

own = False

DEVICE = "cuda"


def listed():
    return [
        # one new token of one sequence: the latency of a single decode step
        _norm("norm-1", tokens=1, q_heads=32, kv_heads=8),
        # a decode batch whose q, k and v rows are slices of one projection's output, E4M3 cache with a scale per head
        _norm("norm-256-e4m3", tokens=256, q_heads=64, kv_heads=8, cache="e4m3", per_head=True, fused=True),
        # a chunk of prompt tokens, bf16 cache
        _norm("norm-8192", tokens=8192, q_heads=32, kv_heads=8, fused=True),
        # prompt tokens of images: three axes, adjacent pairs, part of the head dim turned, weights of each head's own
        # around 1, an odd count, padded rows
        _norm("norm-axes-4109", tokens=4109, q_heads=16, kv_heads=16, head_dim=64, block=32, rotary=48, axes=3, adjacent=True,
              padded=13, weights="heads", offset=1.0),
        # four answers to one prompt: latency
        _shared("shared-4", seqs=4, groups=1, prefix_low=1008, prefix_high=1008, suffix_low=1, suffix_high=90, q_heads=32, kv_heads=8),
        # one system prompt for a batch of 256, E4M3 cache
        _shared("shared-256-e4m3", seqs=256, groups=1, prefix_low=2048, prefix_high=2048, suffix_low=64, suffix_high=512, q_heads=32,
                kv_heads=8, cache="e4m3"),
        # questions about one long document, eight query heads to a KV head
        _shared("shared-64-long", seqs=64, groups=1, prefix_low=32768, prefix_high=32768, suffix_low=1, suffix_high=2048, q_heads=64,
                kv_heads=8),
        # several prompts of different lengths (the shortest of none), head dim 64, one query head to a KV head, padded rows
        _shared("shared-groups-90", seqs=90, groups=7, prefix_low=0, prefix_high=9001, suffix_low=1, suffix_high=1500, q_heads=16,
                kv_heads=16, head_dim=64, block=32, padded=3),
        # one decoded token against one encoder's states: latency
        _cross("cross-1", seqs=1, rows_low=1, rows_high=1, states_low=1500, states_high=1500, q_heads=16, kv_heads=16, head_dim=64),
        # five beams of 32 sequences
        _cross("cross-32-beams", seqs=32, rows_low=5, rows_high=5, states_low=1, states_high=4000, q_heads=32, kv_heads=8),
        # a training-sized batch of decoder rows
        _cross("cross-16-512", seqs=16, rows_low=512, rows_high=512, states_low=2048, states_high=2048, q_heads=32, kv_heads=8),
        # ragged rows and states, none among them, E4M3 cache of 32-token pages with a scale per head
        _cross("cross-40-e4m3", seqs=40, rows_low=0, rows_high=301, states_low=0, states_high=2999, q_heads=24, kv_heads=8, block=32,
               cache="e4m3", per_head=True),
    ]


def _norm(name, tokens, q_heads, kv_heads, head_dim=128, block=16, cache="bf16", per_head=False, fused=False, rotary=0, axes=1,
          adjacent=False, padded=0, weights="shared", offset=0.0):
    return {"name": name, "kind": "norm", "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim,
            "block": block, "cache": cache, "per_head": per_head, "fused": fused, "rotary": rotary or head_dim, "axes": axes,
            "adjacent": adjacent, "padded": padded, "weights": weights, "offset": offset}


def _shared(name, seqs, groups, prefix_low, prefix_high, suffix_low, suffix_high, q_heads, kv_heads, head_dim=128, block=16,
            cache="bf16", per_head=False, padded=0):
    return {"name": name, "kind": "shared", "seqs": seqs, "groups": groups, "prefix_low": prefix_low, "prefix_high": prefix_high,
            "suffix_low": suffix_low, "suffix_high": suffix_high, "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim,
            "block": block, "cache": cache, "per_head": per_head, "padded": padded}


def _cross(name, seqs, rows_low, rows_high, states_low, states_high, q_heads, kv_heads, head_dim=128, block=16, cache="bf16",
           per_head=False):
    return {"name": name, "kind": "cross", "seqs": seqs, "rows_low": rows_low, "rows_high": rows_high, "states_low": states_low,
            "states_high": states_high, "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "block": block,
            "cache": cache, "per_head": per_head}


def _spread(rng, low, high):
    """A whole number, its logarithm spread evenly over [low, high]."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    head_dim, block = rng.choice([64, 128]), rng.choice([16, 32])
    cache = rng.choice(["bf16", "e4m3"])
    per_head = cache == "e4m3" and rng.random() < 0.5
    kv_heads, group = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8, 16])
    kind = rng.choice(["norm", "shared", "shared", "cross", "cross"])
    if kind == "norm":
        case = _norm("", _spread(rng, 1, 8192), kv_heads * min(group, 8), kv_heads, head_dim, block, cache, per_head,
                     rng.random() < 0.5, rng.choice([head_dim, head_dim, head_dim // 2, head_dim - 16]), rng.choice([1, 1, 2, 3, 4]),
                     rng.random() < 0.5, rng.choice([0, 0, 0, 5]), rng.choice(["shared", "shared", "heads", "none"]),
                     rng.choice([0.0, 1.0]))
    elif kind == "shared":
        seqs = _spread(rng, 1, 256)
        high = _spread(rng, 32, 32768)
        case = _shared("", seqs, _spread(rng, 1, min(seqs, 12)), rng.choice([high, high // 2, 0]), high, 1, _spread(rng, 1, 2048),
                       kv_heads * group, kv_heads, head_dim, block, cache, per_head, rng.choice([0, 0, 2]))
        while _elements(case) > 64 * 8 * 34816 * 128 or work(case)["flops"] > 6.5e10:
            case["seqs"] = max(1, case["seqs"] // 2)
            case["groups"] = min(case["groups"], case["seqs"])
    else:
        rows, states = _spread(rng, 1, 1024), _spread(rng, 1, 16384)
        case = _cross("", _spread(rng, 1, 64), rng.choice([rows, rows // 2, 0]), rows, rng.choice([states, states // 3, 0]), states,
                      kv_heads * group, kv_heads, head_dim, block, cache, per_head)
        while _scores(case) > 6e8 or work(case)["flops"] > 2.5e11:
            case["seqs"], case["rows_high"] = max(1, case["seqs"] // 2), max(1, case["rows_high"] * 3 // 4)
            case["rows_low"] = min(case["rows_low"], case["rows_high"])
    del case["name"]
    return case


def _elements(case):
    """Elements of the keys that the plain form of a shared case brings together."""
    return case["seqs"] * case["kv_heads"] * case["head_dim"] * (case["prefix_high"] + case["suffix_high"])


def _scores(case):
    """Scores that the plain form of a cross case makes."""
    return case["seqs"] * case["q_heads"] * case["rows_high"] * case["states_high"]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _even(n, low, high):
    """n whole numbers spread evenly from low to high."""
    return [high] if n == 1 else [low + (high - low) * i // (n - 1) for i in range(n)]


def _groups(case):
    """(first sequence of each group and behind the last, shared pages of each): later groups are larger, prefixes in no order."""
    n, g = case["seqs"], case["groups"]
    start = [n * i * (i + 1) // (g * (g + 1)) for i in range(g + 1)]
    pages = [p // case["block"] for p in _even(g, case["prefix_low"], case["prefix_high"])]
    return start, [pages[(5 * i + 2) % g] if g % 5 else pages[i] for i in range(g)]


def _suffixes(case):
    """How many tokens each sequence of a shared case has of its own; the last ones of a padded batch have none, and no prefix."""
    n = case["seqs"]
    each = _even(n, case["suffix_low"], case["suffix_high"])
    step = next(p for p in (7, 11, 13, 17, 19, 23) if n % p)
    return [each[i * step % n] for i in range(n)]


def _padded(case):
    return min(case["padded"], case["seqs"] - 1)


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


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(int(seed))
    return {"norm": _prepare_norm, "shared": _prepare_shared, "cross": _prepare_cross}[case["kind"]](case, gen)


def _prepare_norm(case, gen):
    t, hq, hkv, d, block = case["tokens"], case["q_heads"], case["kv_heads"], case["head_dim"], case["block"]
    pairs, axes = case["rotary"] // 2, case["axes"]
    # rows as a projection gives them: some dims larger than others, the tokens' sizes apart
    size = torch.exp(0.7 * torch.randn(1, hq + 2 * hkv, d, generator=gen, device=DEVICE))
    size = size * torch.exp(torch.randn(t, 1, 1, generator=gen, device=DEVICE))
    rows = _normal(gen, (t, hq + 2 * hkv, d), scale=size)
    q, k, v = rows.split([hq, hkv, hkv], dim=1)  # slices of one projection's output
    if not case["fused"]:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
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
    weights = [None, None]
    if case["weights"] != "none":
        shapes = [(d,), (d,)] if case["weights"] == "shared" else [(hq, d), (hkv, d)]
        weights = [(1.0 - case["offset"] + 0.3 * torch.randn(s, generator=gen, device=DEVICE)).to(torch.bfloat16) for s in shapes]
    return {"kind": "norm", "q": q, "k": k, "v": v, "positions": positions if axes > 1 else positions[0].contiguous(),
            "inv_freq": inv_freq, "pair_axis": pair_axis, "adjacent": case["adjacent"], "slots": slots,
            "q_weight": weights[0], "k_weight": weights[1], "offset": case["offset"], "eps": 1e-6,
            "k_cache": _pool(gen, blocks, hkv, block, d, case["cache"]),
            "v_cache": _pool(gen, blocks, hkv, block, d, case["cache"]),
            "kv_scale": kv_scale, "k_scales": k_scales, "v_scales": v_scales,
            "out": torch.empty(t, hq, d, dtype=torch.bfloat16, device=DEVICE)}


def _caches(case, gen, blocks):
    """Keys with a mean of its own for each channel, as rotated keys have, values, and their scales."""
    hkv, block, d = case["kv_heads"], case["block"], case["head_dim"]
    k = _pool(gen, blocks, hkv, block, d, case["cache"], 0.5 * torch.randn(hkv, 1, d, generator=gen, device=DEVICE))
    v = _pool(gen, blocks, hkv, block, d, case["cache"])
    kv_scale, k_scales, v_scales = _scales(gen, hkv, case["per_head"])
    return {"k_cache": k, "v_cache": v, "kv_scale": kv_scale, "k_scales": k_scales, "v_scales": v_scales,
            "softmax_scale": 1.0 / math.sqrt(d)}


def _prepare_shared(case, gen):
    s, block = case["seqs"], case["block"]
    start, pages = _groups(case)
    of = torch.tensor([g for g in range(case["groups"]) for _ in range(start[g + 1] - start[g])], device=DEVICE)
    shared = torch.tensor(pages, device=DEVICE)
    live = torch.arange(s, device=DEVICE) < s - _padded(case)
    suffix = torch.tensor(_suffixes(case), device=DEVICE)
    lengths = torch.where(live, shared[of] * block + suffix, 0)
    mine = torch.where(live, (suffix + block - 1) // block, 0)
    need = shared[of] * live + mine
    # physical pages: the groups' first, then each sequence's own, all shuffled
    first, base = torch.cumsum(shared, 0) - shared, int(shared.sum())
    own_first = base + torch.cumsum(mine, 0) - mine
    total, width = base + int(mine.sum()), max(1, int(need.max()))
    page = torch.randperm(total, generator=gen, device=DEVICE)
    at = torch.arange(width, device=DEVICE)
    which = torch.where(at < shared[of][:, None], first[of][:, None] + at, own_first[:, None] + at - shared[of][:, None])
    tables = torch.where(at < need[:, None], page[which.clamp(0, total - 1)], -1)
    return {"kind": "shared", "q": _normal(gen, (s, case["q_heads"], case["head_dim"])), "tables": tables.to(torch.int32),
            "lengths": lengths.to(torch.int32), "group_start": torch.tensor(start, dtype=torch.int32, device=DEVICE),
            "prefix_blocks": shared.to(torch.int32), "max_prefix_blocks": max(pages),
            "out": torch.empty(s, case["q_heads"], case["head_dim"], dtype=torch.bfloat16, device=DEVICE), **_caches(case, gen, total)}


def _rows_and_states(case):
    """How many rows and how many states each sequence of a cross case has, the two in different orders."""
    n = case["seqs"]
    step = next(p for p in (7, 11, 13, 17, 19, 23) if n % p)
    states = _even(n, case["states_low"], case["states_high"])
    return _even(n, case["rows_low"], case["rows_high"]), [states[(i * step + 3) % n] for i in range(n)]


def _prepare_cross(case, gen):
    n, block = case["seqs"], case["block"]
    rows, states = _rows_and_states(case)
    start = [0]
    for r in rows:
        start.append(start[-1] + r)
    lengths = torch.tensor(states, device=DEVICE)
    need = (lengths + block - 1) // block
    total, width = max(1, int(need.sum())), max(1, int(need.max()))
    page = torch.randperm(total, generator=gen, device=DEVICE)
    first = torch.cumsum(need, 0) - need
    at = torch.arange(width, device=DEVICE)
    tables = torch.where(at < need[:, None], page[(first[:, None] + at).clamp(max=total - 1)], -1)
    seq = torch.tensor([i for i, r in enumerate(rows) for _ in range(r)], dtype=torch.int64, device=DEVICE)
    return {"kind": "cross", "q": _normal(gen, (start[-1], case["q_heads"], case["head_dim"])), "tables": tables.to(torch.int32),
            "lengths": lengths.to(torch.int32), "query_start": torch.tensor(start, dtype=torch.int32, device=DEVICE), "seq": seq,
            "max_rows": max(rows), "out": torch.empty(start[-1], case["q_heads"], case["head_dim"], dtype=torch.bfloat16, device=DEVICE),
            **_caches(case, gen, total)}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    kind = state["kind"]
    if own:
        return {"norm": _own_norm, "shared": _own_shared, "cross": _own_cross}[kind](state)
    return {"norm": _plain_norm, "shared": _plain_shared, "cross": _plain_cross}[kind](state)


def _as_values(cache):
    """A cache as the values its bytes stand for (before the scale)."""
    return cache if cache.dtype == torch.bfloat16 else cache.view(torch.float8_e4m3fn)


def _own_norm(st):
    from paged_kv_cache_193_gb300 import api
    out = api.norm_rope_append(st["q"], st["k"], st["v"], st["positions"], st["inv_freq"], st["slots"], st["k_cache"], st["v_cache"],
                               q_weight=st["q_weight"], k_weight=st["k_weight"], eps=st["eps"], weight_offset=st["offset"],
                               pair_axis=st["pair_axis"], adjacent=st["adjacent"], kv_scale=st["kv_scale"], k_scales=st["k_scales"],
                               v_scales=st["v_scales"], out=st["out"])
    return {"q": out, "k_cache": _as_values(st["k_cache"]), "v_cache": _as_values(st["v_cache"])}


def _own_shared(st):
    from paged_kv_cache_193_gb300 import api
    if "workspace" not in st:  # a serving program keeps one
        st["workspace"] = api.alloc_shared_prefix_workspace(st["q"], st["k_cache"], st["group_start"], st["max_prefix_blocks"])
    return api.shared_prefix_decode(st["q"], st["k_cache"], st["v_cache"], st["tables"], st["lengths"], st["group_start"],
                                    st["prefix_blocks"], st["max_prefix_blocks"], softmax_scale=st["softmax_scale"],
                                    kv_scale=st["kv_scale"], k_scales=st["k_scales"], v_scales=st["v_scales"],
                                    workspace=st["workspace"], out=st["out"])


def _own_cross(st):
    from paged_kv_cache_193_gb300 import api
    if "workspace" not in st:
        st["workspace"] = api.alloc_cross_workspace(st["q"], st["k_cache"], st["tables"], st["max_rows"])
    return api.cross_attention(st["q"], st["k_cache"], st["v_cache"], st["tables"], st["lengths"], st["query_start"], st["max_rows"],
                               softmax_scale=st["softmax_scale"], kv_scale=st["kv_scale"], k_scales=st["k_scales"],
                               v_scales=st["v_scales"], workspace=st["workspace"], out=st["out"])


def _plain_norm(st):
    q, k, v, freq = st["q"], st["k"], st["v"], st["inv_freq"]
    pairs = freq.numel()
    positions = st["positions"].view(-1, q.shape[0])
    axis = torch.zeros(pairs, dtype=torch.int64, device=q.device) if st["pair_axis"] is None else st["pair_axis"].long()
    angle = positions[axis].T.double() * freq  # [tokens, pairs]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def normed(x, weight):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + st["eps"])
        return x if weight is None else x * (weight.float() + st["offset"])

    def turn(x):
        y = x.clone()
        first, second = (slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)) if st["adjacent"] else (slice(0, pairs), slice(pairs, 2 * pairs))
        a, b = x[..., first], x[..., second]
        y[..., first] = a * cos - b * sin
        y[..., second] = a * sin + b * cos
        return y

    k_cache, v_cache = _as_values(st["k_cache"]), _as_values(st["v_cache"])
    block = k_cache.shape[2]
    new_k, new_v = turn(normed(k, st["k_weight"])), v.float()
    if k_cache.dtype != torch.bfloat16:
        k_scale, v_scale = (st["kv_scale"] if x is None else x[:, None] for x in (st["k_scales"], st["v_scales"]))
        new_k, new_v = (new_k / k_scale).clamp(-448, 448), (new_v / v_scale).clamp(-448, 448)
    kept = (st["slots"] >= 0).nonzero()[:, 0]
    slot = st["slots"][kept].long()
    bits = torch.int16 if k_cache.dtype == torch.bfloat16 else torch.uint8
    k_cache.view(bits)[slot // block, :, slot % block] = new_k.to(k_cache.dtype)[kept].view(bits)
    v_cache.view(bits)[slot // block, :, slot % block] = new_v.to(v_cache.dtype)[kept].view(bits)
    st["out"].copy_(turn(normed(q, st["q_weight"])))
    return {"q": st["out"], "k_cache": k_cache, "v_cache": v_cache}


def _gathered(cache, tables):
    """The cached rows of each table row in 32 bits, [sequences, heads, tokens, head_dim] (rows of no page: any)."""
    rows = _as_values(cache[tables.long().clamp(min=0)]).float()
    return rows.transpose(1, 2).flatten(2, 3)


def _softmax_of(x, keys, values, lengths, st):
    """The attention of x [sequences, heads, rows, head_dim] to the first `lengths` keys, zeros where there are none."""
    bf16 = st["k_cache"].dtype == torch.bfloat16
    k_scale, v_scale = (1.0 if bf16 else st["kv_scale"] if s is None else s[:, None, None] for s in (st["k_scales"], st["v_scales"]))
    live = (torch.arange(keys.shape[2], device=x.device) < lengths[:, None])[:, None, None]
    logit = (x @ keys.transpose(-1, -2)) * (st["softmax_scale"] * k_scale)
    logit = torch.where(live, logit, -torch.inf)
    p = torch.exp(logit - logit.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min))
    total = p.sum(-1, keepdim=True)
    values = torch.where(live.transpose(-1, -2), values, 0.0)
    return torch.where(total > 0, (p @ values) / torch.where(total > 0, total, 1.0) * v_scale, 0.0)


def _plain_shared(st):
    q = st["q"]
    s, hq, d = q.shape
    hkv = st["k_cache"].shape[1]
    keys, values = _gathered(st["k_cache"], st["tables"]), _gathered(st["v_cache"], st["tables"])
    out = _softmax_of(q.float().view(s, hkv, hq // hkv, d), keys, values, st["lengths"], st)
    return st["out"].copy_(out.view(s, hq, d))


def _plain_cross(st):
    q, seq, n = st["q"], st["seq"], st["lengths"].shape[0]
    t, hq, d = q.shape
    hkv = st["k_cache"].shape[1]
    keys, values = _gathered(st["k_cache"], st["tables"]), _gathered(st["v_cache"], st["tables"])
    at = torch.arange(t, device=q.device) - st["query_start"].long()[seq]
    x = q.new_zeros(n, st["max_rows"], hq, d, dtype=torch.float32)
    x[seq, at] = q.float()
    x = x.unflatten(2, (hkv, hq // hkv)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [n, hkv, rows * group, d]
    out = _softmax_of(x, keys, values, st["lengths"], st)
    out = out.unflatten(2, (st["max_rows"], hq // hkv)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    return st["out"].copy_(out[seq, at])


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    d, block, elem = case["head_dim"], case["block"], 2 if case["cache"] == "bf16" else 1
    hq, hkv = case["q_heads"], case["kv_heads"]
    if case["kind"] == "norm":
        t = case["tokens"]
        live = t - min(case["padded"], t - 1)
        moved = t * hq * d * 4 + live * hkv * d * 2 * (2 + elem)
        weights = {"none": 0, "shared": 4 * d, "heads": 2 * d * (hq + hkv)}[case["weights"]]
        return {"bytes": moved + weights + t * 4 * (1 + case["axes"]),
                "flops": (4 * d + 3 * case["rotary"]) * (t * hq + live * hkv)}
    if case["kind"] == "shared":
        start, pages = _groups(case)
        live = case["seqs"] - _padded(case)
        moved, flops = case["seqs"] * (hq * d * 4 + 4), 0
        suffix = _suffixes(case)
        for g, n in enumerate(pages):
            seqs = range(start[g], min(start[g + 1], live))
            tokens = sum(suffix[s] for s in seqs)
            moved += ((n * block if len(seqs) else 0) + tokens) * hkv * d * 2 * elem
            moved += 4 * (n + sum(-(-suffix[s] // block) for s in seqs))
            flops += 4 * hq * d * (len(seqs) * n * block + tokens)
        return {"bytes": moved, "flops": flops}
    moved, flops = 0, 0
    for r, n in zip(*_rows_and_states(case)):
        moved += r * hq * d * 4 + (n * hkv * d * 2 * elem + 4 * -(-n // block) if r else 0)
        flops += 4 * hq * d * r * n
    return {"bytes": moved, "flops": flops}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, written apart from the plain forms
# ---------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "shared": _exact_shared, "cross": _exact_cross}[case["kind"]](st)


def _exact_norm(st):
    t = st["q"].shape[0]
    freq = st["inv_freq"]
    pairs = freq.numel()
    positions = st["positions"].reshape(-1, t).double()
    axis = [0] * pairs if st["pair_axis"] is None else st["pair_axis"].tolist()
    angle = torch.stack([positions[a] * f for a, f in zip(axis, freq)], 1)
    unit = torch.polar(torch.ones_like(angle), angle)[:, None]  # a pair as a complex number, turned by a product

    def made(x, weight):
        x = x.double()
        x = x / (torch.linalg.vector_norm(x, dim=-1, keepdim=True).square() / x.shape[-1] + st["eps"]).sqrt()
        if weight is not None:
            x = x * (weight.double() + st["offset"])
        part = x[..., :2 * pairs]
        pair = part.unflatten(-1, (pairs, 2)) if st["adjacent"] else part.unflatten(-1, (2, pairs)).transpose(-1, -2)
        y = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * unit)
        y = y.flatten(-2) if st["adjacent"] else y.transpose(-1, -2).flatten(-2)
        return torch.cat([y, x[..., 2 * pairs:]], -1)

    caches = []
    for name, new in (("k", made(st["k"], st["k_weight"])), ("v", st["v"].double())):
        cache = _as_values(st[name + "_cache"])
        if cache.dtype != torch.bfloat16:
            s = st[name + "_scales"]
            new = (new / (st["kv_scale"] if s is None else s.double()[:, None])).clamp(-448.0, 448.0)
        block = cache.shape[2]
        rows = cache.double().transpose(1, 2).flatten(0, 1)  # by slot
        live = st["slots"] >= 0
        rows[st["slots"][live].long()] = new[live]
        caches.append(rows.unflatten(0, (-1, block)).transpose(1, 2).contiguous())
    return {"q": made(st["q"], st["q_weight"]), "k_cache": caches[0], "v_cache": caches[1]}


def _exact_attention(st, q, table, n):
    """q [rows, q_heads, head_dim] over the n tokens of one table row."""
    r, hq, d = q.shape
    hkv, block = st["k_cache"].shape[1:3]
    out = torch.zeros(r, hq, d, dtype=torch.float64, device=q.device)
    if not n or not r:
        return out
    page = table[:-(-n // block)].long()
    ones = torch.ones(hkv, dtype=torch.float64, device=q.device)
    bf16 = st["k_cache"].dtype == torch.bfloat16
    k_scale, v_scale = (ones if bf16 else ones * st["kv_scale"] if s is None else s.double() for s in (st["k_scales"], st["v_scales"]))
    for h in range(hkv):
        k, v = (_as_values(c[page, h]).double().reshape(-1, d)[:n] for c in (st["k_cache"], st["v_cache"]))
        group = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
        logit = torch.einsum("rgd,td->rgt", q[:, group].double(), k) * (st["softmax_scale"] * k_scale[h])
        out[:, group] = torch.einsum("rgt,td->rgd", torch.softmax(logit, -1), v) * v_scale[h]
    return out


def _exact_shared(st):
    return torch.cat([_exact_attention(st, st["q"][s:s + 1], st["tables"][s], n) for s, n in enumerate(st["lengths"].tolist())])


def _exact_cross(st):
    start = st["query_start"].tolist()
    return torch.cat([_exact_attention(st, st["q"][start[s]:start[s + 1]], st["tables"][s], n)
                      for s, n in enumerate(st["lengths"].tolist())])
