"""The angle of the rotation: how exactly it is reduced to a fraction of a
turn, and what that leaves of far positions and small frequencies."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import ops_reference as R

PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
MASK = 2 ** 64 - 1


def turn_fraction(f):
    """The integer arithmetic of the kernel's function of that name."""
    bits = int(np.float64(f).view(np.uint64))
    shift = (bits >> 52 & 0x7FF) - 1023 - 1
    significand = (bits | 1 << 52) << 11 & MASK
    part = significand * 0xA2F9836E4E44152A >> 64
    turn = 0 if shift <= -64 or shift >= 64 else part << shift & MASK if shift >= 0 else part >> -shift
    return -turn & MASK if bits >> 63 else turn


def test_the_constant_is_two_over_pi():
    assert 0xA2F9836E4E44152A == round(2 / PI * 2 ** 64)


@pytest.mark.parametrize("position", [1, -1, 3, 4096, 131071, 10 ** 6, 2 ** 31 - 1, -2 ** 31])
def test_the_angle_is_off_by_its_stated_bound(position):
    """position * f / 2 pi modulo a turn: within |position| (2^-64 turns + 2^-61 f), and at position 2^31 far below the
    2^-25 of a turn that the step of fp32 sine and cosine arguments is."""
    rng = np.random.default_rng(position & 0xFFFF)
    freqs = [1.0, 2.46e-6, 1e-7, 1e-8, 1e-12, 1e-19, 1e-30, 5e-324, 0.0, 3.7e4, 1e15, 2.0 ** 64]
    freqs += list(10.0 ** rng.uniform(-12, 6, 300))
    for f in [x * s for x in freqs for s in (1, -1)]:
        exact = Fraction(float(f)) * position / (2 * PI)
        got = Fraction(turn_fraction(f) * position & MASK, 2 ** 64)
        off = (got - exact + Fraction(1, 2)) % 1 - Fraction(1, 2)
        bound = abs(position) * (Fraction(1, 2 ** 64) + abs(Fraction(float(f))) / 2 ** 61)
        assert abs(off) <= bound, (f, float(off), float(bound))
        if abs(f) <= 1:
            assert abs(off) < Fraction(1, 2 ** 29)


def angle_slack(x, positions, inv_freq, adjacent):
    """How far the rotated elements may be from ``R.rotate``'s: fp32 arithmetic as in ``R.rotate_slack`` (2^-21 of |x_a| +
    |x_b|), the reduction's |position| (2^-64 2 pi + 2^-61 f) radians (f turns are f / 2 pi, times 2 pi), and 2^-51 of the
    angle for the 64-bit roundings of the reference's own product, sine and cosine."""
    x, pos = np.abs(np.asarray(x, np.float64)), np.abs(np.asarray(positions, np.float64))
    out = np.zeros_like(x)
    half = len(inv_freq)
    for i, f in enumerate(np.abs(np.asarray(inv_freq, np.float64))):
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
        radians = pos * (2.0 ** -64 * 2 * np.pi + 2.0 ** -61 * 2 * np.pi * f + 2.0 ** -51 * f)
        out[:, :, a] = out[:, :, b] = (x[:, :, a] + x[:, :, b]) * (2.0 ** -21 + radians)[:, None]
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("adjacent", [False, True])
def test_small_frequencies_at_far_positions(cuda_device, adjacent):
    from paged_kv_cache_193_gb300 import api
    g = torch.Generator().manual_seed(9)
    D, Hq = 128, 3
    freq = torch.cat([10.0 ** (-12 * torch.rand(40, dtype=torch.float64, generator=g)),
                      torch.tensor([2.46e-6, 1e-7, 1e-8, 1e-9, 1e-10, 3e-10, 1e-12, 1e-19, 1e-300, 0.0], dtype=torch.float64),
                      500000.0 ** (-torch.arange(50, 64, dtype=torch.float64) / 64)])
    pos = torch.tensor([0, 1, -1, 131071, 10 ** 6, 2 ** 30 + 12345, 2 ** 31 - 1, -2 ** 31, -(2 ** 31) + 7, 1999999973], dtype=torch.int32)
    T = len(pos)
    q, k = (torch.randn(T, h, D, generator=g).to(torch.bfloat16) for h in (Hq, 1))
    kc = torch.zeros(1, 1, 16, D, dtype=torch.bfloat16, device=cuda_device)
    kd = k.to(cuda_device)
    out = api.rope_append(q.to(cuda_device), kd, kd, pos.to(cuda_device), freq.to(cuda_device),
                          torch.arange(T, dtype=torch.int32, device=cuda_device), kc, torch.zeros_like(kc), adjacent=adjacent)
    for x, got in ((q, out), (k, kc[0, 0, :T, None])):
        x = x.double().numpy()
        want = R.rotate(x, pos.numpy(), freq.numpy(), None, adjacent)
        slack = angle_slack(x, pos.numpy(), freq.numpy(), adjacent)
        off = np.abs(got.double().cpu().numpy() - want) - (R.HALF["bf16"] * (np.abs(want) + slack) + slack)
        assert off.max() <= 0, np.unravel_index(off.argmax(), off.shape)


def by_differences(q, k, v, freq, apart, scale):
    """(out [H, D], bound [H, D]): attention of one query to T tokens ``apart`` positions away, in 64 bits, each score
    from the difference of positions alone, and how far a decode over rows rotated by the positions themselves may be.

    An element of a rotated row is off by 2^-21 of its pair in fp32 and by at most 2^-8 of itself in bf16, so score t by
    e_t = scale sum_d ((2^-8 + 2^-20) (|q'_d| |k'_d|) 2 + 2^-16 |q'_d| |k'_d|), with |x'_d| at most its pair's length, and by
    2^-17 (128 fp32 products of at most that, 2^-24 each).  The probabilities p then become p_t exp(d_t) / sum, |d_t| <= e_t, and
    are off by at most p_t (exp(e_t + e) - 1) with exp(e) = sum_t p_t exp(e_t); one more 2^-8 for their rounding to bf16
    and one for the output's."""
    H, D = q.shape
    half = D // 2
    group = H // k.shape[1]
    out, bound = np.zeros((H, D)), np.zeros((H, D))
    turn = np.exp(1j * np.outer(apart, freq))
    for h in range(H):
        qc = q[h, :half] + 1j * q[h, half:]
        kc = k[:, h // group, :half] + 1j * k[:, h // group, half:]
        z = scale * ((qc * kc.conj()) * turn).real.sum(1)
        p = np.exp(z - z.max())
        p /= p.sum()
        out[h] = p @ v[:, h // group]
        # |q_a k_a| + |q_b k_b| of two rotated pairs is at most the product of their lengths
        size = scale * (np.abs(qc) * np.abs(kc)).sum(1)
        e = (2 * (2.0 ** -8 + 2.0 ** -20) + 2.0 ** -16) * size + 2.0 ** -17 * size
        moved = p * (np.exp(e + np.log(p @ np.exp(e))) - 1)
        bound[h] = moved @ np.abs(v[:, h // group] - out[h])
        bound[h] += 2.0 ** -8 * (p + moved) @ np.abs(v[:, h // group]) + 2.0 ** -8 * (np.abs(out[h]) + bound[h])
    return out, bound


def _sequence():
    T, Hq, Hkv, D = 48, 4, 2, 128
    g = torch.Generator().manual_seed(4)
    # every key is much like every query, so a score is a sum of cosines that falls off with the distance
    alike = torch.randn(D, generator=g)
    q, k = (1.5 * alike + 0.2 * torch.randn(T, h, D, generator=g) for h in (Hq, Hkv))
    v = torch.randn(T, Hkv, D, generator=g)
    q, k, v = (x.to(torch.bfloat16) for x in (q, k, v))
    freq = 30.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))
    apart = (T // 2 - np.arange(T)).astype(np.float64)  # the query stands in the middle
    return q, k, v, freq, apart


def _exact(moved=0):
    q, k, v, freq, apart = _sequence()
    return by_differences(q[-1].double().numpy(), k.double().numpy(), v.double().numpy(), freq.numpy(), apart + moved, 128 ** -0.5)


def test_a_shift_of_one_position_is_past_the_bound():
    """The test below can fail: with the query one position off, three quarters of the outputs are past its bound, half
    past twice the bound."""
    (want, bound), (a, _), (b, _) = _exact(), _exact(1), _exact(-1)
    for wrong in (a, b):
        assert (np.abs(wrong - want) > bound).mean() > 0.7 and (np.abs(wrong - want) > 2 * bound).mean() > 0.5


@pytest.mark.gpu
@pytest.mark.parametrize("first", [0, 4096, -70000, 2 ** 31 - 48])
def test_rotated_attention_is_that_of_the_differences(cuda_device, first):
    """Through the cache, at near and far positions: the attention that the differences of positions alone define."""
    from paged_kv_cache_193_gb300 import api
    q, k, v, freq, apart = _sequence()
    (T, Hkv, D), B = k.shape, 16
    kc = torch.zeros(T // B, Hkv, B, D, dtype=torch.bfloat16, device=cuda_device)
    vc = torch.zeros_like(kc)
    pos = torch.arange(first, first + T, dtype=torch.int64).to(torch.int32).to(cuda_device)
    slots = torch.arange(T, dtype=torch.int32, device=cuda_device)
    f = freq.to(cuda_device)
    api.rope_append(None, k.to(cuda_device), v.to(cuda_device), pos, f, slots, kc, vc)
    one = k[:1].to(cuda_device)
    rq = api.rope_append(q[-1:].to(cuda_device), one, one, pos[T // 2:T // 2 + 1].contiguous(), f, slots[:1] - 1, kc, vc)
    out = api.decode(rq, kc, vc, torch.arange(T // B, dtype=torch.int32, device=cuda_device)[None],
                     torch.tensor([T], dtype=torch.int32, device=cuda_device))
    want, bound = _exact()
    off = np.abs(out[0].double().cpu().numpy() - want) - bound
    assert off.max() <= 0, off.max()
