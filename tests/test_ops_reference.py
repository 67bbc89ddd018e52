"""The 64-bit references of the rotate-and-append and block-sparse operators,
tied to torch and to the C oracle (no GPU)."""
import numpy as np
import pytest
import torch

import ops_reference as R
from paged_cases import LogicalCase, bits_to_f64


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("axes", [1, 3])
def test_rotation_is_a_complex_product(adjacent, axes):
    rng = np.random.default_rng(axes)
    T, H, D, rot = 7, 3, 64, 48
    x = rng.standard_normal((T, H, D))
    freq = 10000.0 ** (-np.arange(rot // 2) / (rot // 2))
    pos = rng.integers(-50, 100000, (axes, T))
    axis = rng.integers(0, axes, rot // 2)
    y = R.rotate(x, pos, freq, axis, adjacent, 1.5)
    angle = torch.from_numpy(pos[axis].T * freq)
    part = torch.from_numpy(x[..., :rot])
    pair = part.unflatten(-1, (rot // 2, 2)) if adjacent else part.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    z = torch.view_as_complex(pair.contiguous()) * torch.polar(torch.full_like(angle, 1.5), angle)[:, None]
    back = torch.view_as_real(z)
    back = back.flatten(-2) if adjacent else back.transpose(-1, -2).flatten(-2)
    assert np.abs(y[..., :rot] - back.numpy()).max() < 1e-12
    assert np.array_equal(y[..., rot:], x[..., rot:])


def test_rotation_depends_on_the_difference_of_positions():
    rng = np.random.default_rng(5)
    q, k = rng.standard_normal((1, 1, 64)), rng.standard_normal((1, 1, 64))
    freq = 500000.0 ** (-np.arange(32) / 32)
    dots = [float((R.rotate(q, [p], freq, None, False) * R.rotate(k, [p - 17], freq, None, False)).sum())
            for p in (17, 1000, 65536)]
    assert np.ptp(dots) < 1e-9


def test_int8_form_is_least_and_a_bound():
    rng = np.random.default_rng(6)
    for scale in (1e-30, 3e-5, 1.0, 127.0, 127.5, 128.0, 1e9, 1e30):
        x = rng.standard_normal(64)
        x *= scale / np.abs(x).max()
        w, e = R.int8_form(x)
        if -60 < e < 40:
            assert np.abs(x).max() <= 127 * 2.0 ** e and np.abs(x).max() > 127 * 2.0 ** (e - 1)
            assert np.abs(w * 2.0 ** e - x).max() <= 2.0 ** (e - 1)
    assert R.int8_form(np.zeros(4)) [1] == -60


def test_score_bounds_every_key():
    rng = np.random.default_rng(7)
    B, D = 16, 64
    k = rng.standard_normal((3, 1, B, D))
    summary, ex = np.zeros((3, 1, 2, D), np.int8), np.zeros((3, 1), np.int8)
    R.block_summary(k, np.arange(3 * B), summary, ex)
    q = rng.standard_normal(D)
    for b in range(3):
        hi, lo = summary[b, 0] * 2.0 ** int(ex[b, 0])
        step = 2.0 ** (int(ex[b, 0]) - 1)  # of each rounding
        assert np.maximum(q * hi, q * lo).sum() + step * np.abs(q).sum() >= (k[b, 0] @ q).max()


def test_summary_of_a_page_that_is_not_complete_is_left_alone():
    k = np.ones((2, 1, 16, 64))
    summary, ex = np.full((2, 1, 2, 64), 7, np.int8), np.full((2, 1), 9, np.int8)
    R.block_summary(k, [0, 14, -1, 16], summary, ex)
    assert (summary == 7).all() and (ex == 9).all()
    R.block_summary(k, [31], summary, ex)
    assert (summary[0] == 7).all() and (summary[1] == 64).all() and ex[1, 0] == -6


def test_choice_of_everything_when_it_fits_and_of_the_best_otherwise():
    rng = np.random.default_rng(8)
    B, D, Hkv = 16, 64, 2
    k = rng.standard_normal((12, Hkv, B, D))
    k[5, 1] *= 8.0  # by far the largest bound for head 1
    summary, ex = np.zeros((12, Hkv, 2, D), np.int8), np.zeros((12, Hkv), np.int8)
    R.block_summary(k, np.arange(12 * B), summary, ex)
    q = rng.standard_normal((1, 4, D))
    tables = np.arange(12, dtype=np.int32)[None]
    sel, cnt = R.select(q, summary, ex, tables, [12 * B - 3], B, 12, 1, 1)
    assert (cnt == 12).all() and np.array_equal(sel[0, 0], np.arange(12))
    sel, cnt = R.select(q, summary, ex, tables, [12 * B - 3], B, 4, 1, 2)
    assert (cnt == 4).all() and sel[0, 1].tolist() == [0, 5, 10, 11]
    summary[:], ex[:] = 1, 0  # every score the same: the lowest indexes
    sel, _ = R.select(q, summary, ex, tables, [12 * B], B, 6, 0, 1)
    assert sel[0, 0].tolist() == [0, 1, 2, 3, 4, 11]


@pytest.mark.parametrize("Hq,Hkv,D,B", [(8, 2, 64, 16), (4, 4, 128, 32)])
def test_all_pages_chosen_is_the_oracles_decode(oracle, Hq, Hkv, D, B):
    case = LogicalCase([1, B, 3 * B + 5, 0], Hq, Hkv, D, 11)
    tables, kc, vc = case.paged(B, 12, np.random.default_rng(1))
    ref = oracle.decode(case.q, kc, vc, tables, np.array(case.ctx, np.int32), Hkv, B, 0.125)
    cnt = np.array([[-(-c // B)] * Hkv for c in case.ctx], np.int32)
    sel = np.tile(np.arange(tables.shape[1], dtype=np.int32), (4, Hkv, 1))
    one = np.ones(Hkv)
    out, bound = R.attend(bits_to_f64(case.q), bits_to_f64(kc), bits_to_f64(vc), tables, case.ctx, sel, cnt, 0.125, one, one)
    assert np.abs(out - ref).max() < 1e-12
    assert (bound[:3] > 0).all() and (out[3] == 0).all()
