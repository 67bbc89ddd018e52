"""Plain 64-bit implementations of the rotate-and-append, block-summary,
block-choice and block-sparse decode operators (numpy, one loop per thing
defined), for the tests.  They share no code with the library, its plain
torch forms or the C oracle; tests/test_ops_reference.py ties them to torch
and to the oracle."""
from __future__ import annotations

import numpy as np
import torch

HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24, "e4m3": 2.0 ** -4}


def values(cache) -> np.ndarray:
    """A cache's stored values in 64 bits (E4M3: what the codes stand for,
    before the scale)."""
    t = cache.detach().cpu()
    if t.dtype == torch.uint8:
        t = t.view(torch.float8_e4m3fn)
    return t.float().numpy().astype(np.float64)


def rotate(x, positions, inv_freq, pair_axis, adjacent, magnitude=1.0):
    """x [T, H, D] turned: pair i by positions[pair_axis[i]][t] * inv_freq[i]."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    pos = np.atleast_2d(np.asarray(positions, np.float64))
    R = 2 * len(inv_freq)
    for i, f in enumerate(np.asarray(inv_freq, np.float64)):
        theta = pos[0 if pair_axis is None else int(pair_axis[i])] * f
        c, s = np.cos(theta)[:, None], np.sin(theta)[:, None]
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + R // 2)
        y[:, :, a] = magnitude * (x[:, :, a] * c - x[:, :, b] * s)
        y[:, :, b] = magnitude * (x[:, :, a] * s + x[:, :, b] * c)
    return y


def rotate_slack(x, positions, inv_freq, pair_axis, adjacent, magnitude=1.0):
    """How far fp32 arithmetic on the same inputs may be from ``rotate``:
    cos and sin each within 2^-22 (a 2^-24 fraction of a half turn, pi * 2^-25
    radians, and two units in the last place of the function), three fp32
    roundings of products and sums (2^-24 each, relative to at most
    |x_a| + |x_b|): 2^-21 (|x_a| + |x_b|) magnitude in all.  The angle itself
    is good to 2^-51 of its size (four 64-bit roundings of the frequency and
    product, on both sides)."""
    x = np.abs(np.asarray(x, np.float64))
    out = np.zeros_like(x)
    pos = np.abs(np.atleast_2d(np.asarray(positions, np.float64)))
    R = 2 * len(inv_freq)
    for i, f in enumerate(np.abs(np.asarray(inv_freq, np.float64))):
        theta = pos[0 if pair_axis is None else int(pair_axis[i])] * f
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + R // 2)
        w = magnitude * (x[:, :, a] + x[:, :, b]) * (2.0 ** -21 + 2.0 ** -51 * theta)[:, None]
        out[:, :, a] = out[:, :, b] = w
    return out


def int8_form(x):
    """(whole numbers, exponent) of x: the least exponent in [-60, 40] with
    max |x| <= 127 * 2^e, by trying them in turn."""
    top = float(np.abs(x).max()) if x.size else 0.0
    e = -60
    while e < 40 and top > 127 * 2.0 ** e:
        e += 1
    return np.clip(np.rint(x * 2.0 ** -e), -127, 127).astype(np.int64), e


def block_summary(k_values, slots, summary, exponents):
    """In place, summary [NB, Hkv, 2, D] and exponents [NB, Hkv]."""
    NB, Hkv, B, D = k_values.shape
    for slot in np.asarray(slots):
        if slot < 0 or slot >= NB * B or slot % B != B - 1:
            continue
        for h in range(Hkv):
            x = k_values[slot // B, h]
            if not np.isfinite(x).all():
                summary[slot // B, h] = 0
                exponents[slot // B, h] = 127
                continue
            w, e = int8_form(np.stack([x.max(0), x.min(0)]))
            summary[slot // B, h] = w
            exponents[slot // B, h] = e


def select(q, summary, exponents, tables, lens, B, top_k, sink, recent):
    """(selected [S, Hkv, top_k], counts [S, Hkv]) by sorting (score, index)."""
    q = np.asarray(q, np.float64)
    S, Hq, D = q.shape
    NB, Hkv = summary.shape[:2]
    G = Hq // Hkv
    sel = np.full((S, Hkv, top_k), -1, np.int32)
    cnt = np.zeros((S, Hkv), np.int32)
    for s in range(S):
        n = min(int(lens[s]), tables.shape[1] * B)
        nb = max(0, -(-n // B))
        for h in range(Hkv):
            if nb <= top_k:
                pick = list(range(nb))
            else:
                qs = []
                for g in range(G):
                    x = q[s, h * G + g]
                    qs.append(int8_form(x) if np.isfinite(x).all() else (np.zeros(D, np.int64), -60))
                scored = []
                for j in range(sink, nb - recent):
                    b = int(tables[s, j])
                    if b < 0 or b >= NB:
                        scored.append((np.inf, j))
                        continue
                    if exponents[b, h] == 127:
                        scored.append((-np.inf, j))
                        continue
                    hi, lo = summary[b, h].astype(np.int64)
                    best = max(2.0 ** e * float(np.maximum(r * hi, r * lo).sum()) for r, e in qs)
                    scored.append((-best * 2.0 ** int(exponents[b, h]), j))
                take = [j for _, j in sorted(scored)[: top_k - sink - recent]]
                pick = sorted(list(range(sink)) + take + list(range(nb - recent, nb)))
            sel[s, h, : len(pick)] = pick
            cnt[s, h] = len(pick)
    return sel, cnt


def attend(q, k_values, v_values, tables, lens, selected, counts, scale, k_scales, v_scales, probability="bf16"):
    """(out [S, Hq, D], bound [S, Hq, D]): the softmax over the listed blocks'
    tokens, and how far a kernel may be off: one rounding of each probability
    (bf16 or fp16) on the way into P V, fp32 sums in the scores (D products
    of at most sum |q k|, in numerator and denominator) and in the outputs,
    one bf16 rounding of the output.  fp16 probabilities have a floor: below
    2^-14 they are off by 2^-25 of the largest, and the query (rounded to
    fp16) by 2^-25 an element."""
    q = np.asarray(q, np.float64)
    S, Hq, D = q.shape
    _, Hkv, B, _ = k_values.shape
    G = Hq // Hkv
    out, bound = np.zeros((S, Hq, D)), np.zeros((S, Hq, D))
    for s in range(S):
        n = min(int(lens[s]), tables.shape[1] * B)
        for h in range(Hkv):
            ks, vs = [], []
            for j in selected[s, h, : counts[s, h]]:
                if j < 0 or j * B >= n:
                    continue
                b = int(tables[s, j])
                rows = min(B, n - int(j) * B)
                ks.append(k_values[b, h, :rows])
                vs.append(v_values[b, h, :rows])
            if not ks:
                continue
            k = np.concatenate(ks) * k_scales[h]
            v = np.concatenate(vs) * v_scales[h]
            for g in range(G):
                x = q[s, h * G + g]
                z = scale * (k @ x)
                p = np.exp(z - z.max())
                p /= p.sum()
                o = h * G + g
                out[s, o] = p @ v
                size = np.abs(scale) * (np.abs(k) @ np.abs(x)).max()
                off = 2 * (D + 4) * HALF["fp32"] * size + 2.0 ** -18
                mass = p @ np.abs(v)
                extra = 0.0
                if probability == "fp16":
                    off += 2 * abs(scale) * D * 2.0 ** -25 * np.abs(k).max()
                    extra = len(p) * 2.0 ** -25 * np.abs(v).max(0)
                bound[s, o] = HALF["bf16"] * np.abs(out[s, o]) + (HALF[probability] + off) * mass * (1 + HALF["bf16"]) + extra
    return out, bound
