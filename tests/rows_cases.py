"""Batches for the shared-prefix and cross-attention tests: caches whose unused
blocks and slots hold NaN, tables, and what the definition gives in 64 bits."""
import numpy as np
import torch

import ops_reference as R

bf = torch.bfloat16


def _round(x, fp8):
    """x as a cache of that type holds it."""
    return (x * 16).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else x.to(bf)


class Pool:
    """A paged cache that is filled sequence by sequence."""

    def __init__(self, blocks, Hkv, B, D, fp8, per_head, g):
        self.B, self.Hkv, self.D, self.fp8, self.g = B, Hkv, D, fp8, g
        self.free = torch.randperm(blocks, generator=g).tolist()
        fill = torch.full((blocks, Hkv, B, D), 0x7f, dtype=torch.uint8) if fp8 else torch.full((blocks, Hkv, B, D), float("nan"), dtype=bf)
        self.k, self.v = fill, fill.clone()
        self.kv_scale = 1 / 16
        self.scales = (0.03 + 0.05 * torch.rand(2, Hkv, generator=g)) if per_head else None

    def add(self, tokens, spread=1.0):
        """Blocks with `tokens` new tokens (those behind them in the last block stay NaN)."""
        out = []
        for t0 in range(0, tokens, self.B):
            b, n = self.free.pop(), min(self.B, tokens - t0)
            self.k[b, :, :n] = _round(spread * torch.randn(self.Hkv, n, self.D, generator=self.g), self.fp8)
            self.v[b, :, :n] = _round(torch.randn(self.Hkv, n, self.D, generator=self.g), self.fp8)
            out.append(b)
        return out

    def to(self, device):
        self.kd, self.vd = self.k.to(device), self.v.to(device)
        self.sd = (None, None) if self.scales is None else tuple(s.contiguous().to(device) for s in self.scales)
        return self

    def head_scales(self):
        if not self.fp8:
            return np.ones(self.Hkv), np.ones(self.Hkv)
        if self.scales is None:
            return np.full(self.Hkv, self.kv_scale), np.full(self.Hkv, self.kv_scale)
        return tuple(s.numpy().astype(np.float64) for s in self.scales)

    def kwargs(self):
        return dict(kv_scale=self.kv_scale, k_scales=self.sd[0], v_scales=self.sd[1])


def table_of(rows, width=None):
    width = width or max(1, max(len(r) for r in rows))
    t = torch.full((len(rows), width), -1, dtype=torch.int32)
    for i, r in enumerate(rows):
        t[i, :len(r)] = torch.tensor(r, dtype=torch.int32)
    return t


def expected(pool, q, tables, lens, scale, raised=True):
    """(out, bound) of ops_reference.attend over whole contexts, a row of `tables` and `lens` to each row of q."""
    width = tables.shape[1]
    lens = np.asarray(lens)
    nb = [-(-int(n) // pool.B) for n in lens]
    sel = np.tile(np.arange(width, dtype=np.int32), (len(nb), pool.Hkv, 1))
    cnt = np.tile(np.asarray(nb, np.int32)[:, None], (1, pool.Hkv))
    ks, vs = pool.head_scales()
    return R.attend(q.float().cpu().numpy(), R.values(pool.k), R.values(pool.v), tables.numpy(), lens, sel, cnt, scale, ks, vs,
                    probability="fp16" if pool.fp8 else "bf16")


def within(out, want, what=""):
    ref, bound = want
    got = out.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all(), f"{what}: not finite"
    off = np.abs(got - ref) - bound
    assert off.size == 0 or off.max() <= 0, f"{what}: {off.max()} beyond the bound at {np.unravel_index(off.argmax(), off.shape)}"


class Shared:
    """groups: (pages of the prefix, tokens behind it of each sequence); a negative number is that many tokens less than
    the prefix holds, None no token at all.  `alone`: tokens of sequences behind the last group."""

    def __init__(self, device, groups, Hq, Hkv, D=128, B=16, fp8=False, per_head=False, alone=(), seed=0, extra=0, spread=1.0):
        g = torch.Generator().manual_seed(seed + 17)
        blocks = sum(p + sum(2 + abs(n or 0) // B for n in own) for p, own in groups) + sum(1 + n // B for n in alone) + 3
        self.pool = Pool(blocks, Hkv, B, D, fp8, per_head, g)
        rows, lens, start, pages = [], [], [0], []
        for p, own in groups:
            prefix = self.pool.add(p * B, spread)
            for n in own:
                if n is None:
                    rows.append([])
                    lens.append(0)
                elif n < 0:  # shares the first pages all the same
                    lens.append(p * B + n)
                    rows.append(prefix[:-(-lens[-1] // B)])
                else:
                    rows.append(prefix + self.pool.add(n, spread))
                    lens.append(p * B + n)
            start.append(len(rows))
            pages.append(p)
        for n in alone:
            rows.append(self.pool.add(n, spread))
            lens.append(n)
        self.pool.to(device)
        S = len(rows)
        self.tables = table_of(rows, max(1, max(len(r) for r in rows)) + extra)
        self.lens = lens
        self.q = torch.randn(S, Hq, D, generator=g).to(bf).to(device)
        self.bt, self.cl = self.tables.to(device), torch.tensor(lens, dtype=torch.int32, device=device)
        self.gs = torch.tensor(start, dtype=torch.int32, device=device)
        self.pb = torch.tensor(pages, dtype=torch.int32, device=device)
        self.most = max(pages, default=0)
        self.scale = 0.11 if D == 64 else 0.08

    def call(self, api, **kw):
        args = dict(max_prefix_blocks=self.most, softmax_scale=self.scale, **self.pool.kwargs())
        args.update(kw)
        q = args.pop("q", self.q)
        return api.shared_prefix_decode(q, self.pool.kd, self.pool.vd, self.bt, self.cl, self.gs, self.pb, **args)

    def expected(self):
        return expected(self.pool, self.q, self.tables, self.lens, self.scale)


class Cross:
    """rows and states of each sequence; `gap` rows of no sequence behind the last."""

    def __init__(self, device, rows, states, Hq, Hkv, D=128, B=16, fp8=False, per_head=False, seed=0, gap=0, extra=0, spread=1.0):
        g = torch.Generator().manual_seed(seed + 29)
        self.pool = Pool(sum(1 + n // B for n in states) + 3, Hkv, B, D, fp8, per_head, g)
        self.tables = table_of([self.pool.add(n, spread) for n in states], max(1, max(-(-n // B) for n in states)) + extra)
        self.pool.to(device)
        start = np.concatenate([[0], np.cumsum(rows)])
        self.rows, self.states, self.gap = rows, states, gap
        self.q = torch.randn(int(start[-1]) + gap, Hq, D, generator=g).to(bf).to(device)
        self.bt, self.sl = self.tables.to(device), torch.tensor(states, dtype=torch.int32, device=device)
        self.qs = torch.tensor(start, dtype=torch.int32, device=device)
        self.seq = np.repeat(np.arange(len(rows)), rows)
        self.most = max(rows)
        self.scale = 0.11 if D == 64 else 0.08

    def call(self, api, **kw):
        args = dict(softmax_scale=self.scale, **self.pool.kwargs())
        args.update(kw)
        q, most = args.pop("q", self.q), args.pop("most", self.most)
        return api.cross_attention(q, self.pool.kd, self.pool.vd, self.bt, self.sl, self.qs, most, **args)

    def expected(self, only=None):
        at = np.arange(len(self.seq)) if only is None else only
        seq = self.seq[at]
        return expected(self.pool, self.q[torch.from_numpy(at).to(self.q.device)], self.tables[torch.from_numpy(seq)],
                        np.asarray(self.states)[seq], self.scale)
