"""Rotate-and-append against its definition in 64 bits: both pairings, one
and several axes, partly rotated heads, strided rows, both cache types, skipped
tokens, far positions, one token to many, captured and on another stream."""
import numpy as np
import pytest
import torch

import ops_reference as R
from gpu_helpers import Guarded
from paged_kv_cache_193_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api(cuda_device):
    from paged_kv_cache_193_gb300 import api as a
    a._lib_handle()
    return a


class Case:
    def __init__(self, device, T, Hq, Hkv, D=128, B=16, fp8=False, rot=0, axes=1, adjacent=False, per_head=False,
                 fused=False, skip=0, magnitude=1.0, far=100000, seed=0, base=500000.0):
        g = torch.Generator().manual_seed(seed + 1000 * T)
        self.rot, self.adjacent, self.magnitude, self.fp8, self.B = rot or D, adjacent, magnitude, fp8, B
        self.Hq, self.Hkv = Hq, Hkv
        if fused:
            rows = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g).to(torch.bfloat16).to(device)
            q, k, v = rows.split([Hq * D, Hkv * D, Hkv * D], dim=1)
            self.q, self.k, self.v = q.view(T, Hq, D), k.view(T, Hkv, D), v.view(T, Hkv, D)
        else:
            self.q, self.k, self.v = (torch.randn(T, h, D, generator=g).to(torch.bfloat16).to(device) for h in (Hq, Hkv, Hkv))
        self.pos = torch.randint(-100 if far > 0 else far, max(far, 1), (axes, T), generator=g, dtype=torch.int32)
        self.freq = base ** (-torch.arange(self.rot // 2, dtype=torch.float64) / (self.rot // 2))
        self.axis = None if axes == 1 else torch.randint(0, axes, (self.rot // 2,), generator=g, dtype=torch.int32)
        NB = (T + B - 1) // B + 2
        self.slots = torch.randperm(NB * B, generator=g)[:T].to(torch.int32)
        if skip:
            self.slots[::skip] = -1
        dtype = torch.uint8 if fp8 else torch.bfloat16
        self.k0 = torch.randint(0, 120, (NB, Hkv, B, D), generator=g).to(dtype).to(device)
        self.v0 = torch.randint(0, 120, (NB, Hkv, B, D), generator=g).to(dtype).to(device)
        self.kv_scale = 0.03
        self.scales = (0.02 + 0.02 * torch.rand(2, Hkv, generator=g)) if per_head else None
        self.device = device

    def call(self, api, out=None, stream=None, kc=None, vc=None):
        dev = self.device
        kc = self.k0.clone() if kc is None else kc
        vc = self.v0.clone() if vc is None else vc
        ks, vs = (None, None) if self.scales is None else (self.scales[0].to(dev), self.scales[1].to(dev))
        pos = (self.pos if self.pos.shape[0] > 1 else self.pos[0]).to(dev)
        out = api.rope_append(self.q, self.k, self.v, pos, self.freq.to(dev), self.slots.to(dev), kc, vc,
                              pair_axis=None if self.axis is None else self.axis.to(dev), adjacent=self.adjacent,
                              magnitude=self.magnitude, kv_scale=self.kv_scale, k_scales=ks, v_scales=vs, out=out, stream=stream)
        return out, kc, vc

    def check(self, oracle, out, kc, vc):
        f64 = lambda t: t.float().cpu().numpy().astype(np.float64)  # noqa: E731
        how = (self.pos.numpy(), self.freq.numpy(), None if self.axis is None else self.axis.numpy(), self.adjacent, self.magnitude)
        # q: one bf16 rounding of the fp32 result
        ref, slack = R.rotate(f64(self.q), *how), R.rotate_slack(f64(self.q), *how)
        off = np.abs(f64(out) - ref) - (R.HALF["bf16"] * np.abs(ref) + 1.01 * slack)
        assert off.max() <= 0, f"q: {off.max()}"
        # k: one rounding to the cache's type; v: the append's own bits
        live = (self.slots >= 0).numpy()
        slot = self.slots.numpy()[live]
        ref, slack = R.rotate(f64(self.k), *how)[live], R.rotate_slack(f64(self.k), *how)[live]
        got = R.values(kc).transpose(0, 2, 1, 3).reshape(-1, self.Hkv, ref.shape[-1])
        if not self.fp8:
            bound = R.HALF["bf16"] * np.abs(ref) + 1.01 * slack
        else:
            s = np.full(self.Hkv, np.float64(np.float32(self.kv_scale))) if self.scales is None else self.scales[0].numpy().astype(np.float64)
            ref, slack = np.clip(ref / s[:, None], -448, 448), slack / s[:, None]
            # half a step of e4m3: 2^-4 of the value, 2^-10 below its normals; the division adds 2^-24
            bound = np.maximum(R.HALF["e4m3"] * np.abs(ref), 2.0 ** -10) + 1.1 * slack + 2.0 ** -23 * np.abs(ref)
        off = np.abs(got[slot] - ref) - bound
        assert off.size == 0 or off.max() <= 0, f"k: {off.max()}"
        want_v, same_k = W.bits(self.v0).copy(), W.bits(self.k0).copy()
        if self.scales is None:
            oracle.cache_append(W.bits(self.v.contiguous()), W.bits(self.v.contiguous()), self.slots.numpy(), same_k, want_v, self.B,
                                int(self.fp8), np.float32(self.kv_scale))
        else:
            s = self.scales[1].numpy().copy()
            oracle.cache_append_scaled(W.bits(self.v.contiguous()), W.bits(self.v.contiguous()), self.slots.numpy(), same_k, want_v,
                                       self.B, s, s)
        assert np.array_equal(W.bits(vc), want_v)
        # rows that no slot names are left as they were
        untouched = np.ones(got.shape[0], bool)
        untouched[slot] = False
        rows = lambda t: W.bits(t).transpose(0, 2, 1, 3).reshape(got.shape)  # noqa: E731
        assert np.array_equal(rows(kc)[untouched], rows(self.k0)[untouched])


CASES = [
    dict(T=1, Hq=8, Hkv=2),
    dict(T=1, Hq=1, Hkv=1, D=64, fused=True, adjacent=True),
    dict(T=5, Hq=4, Hkv=4, rot=16),
    dict(T=37, Hq=16, Hkv=2, fused=True, skip=3),
    dict(T=37, Hq=6, Hkv=3, D=64, B=32, adjacent=True, rot=48, axes=3, fused=True),
    dict(T=64, Hq=32, Hkv=2, fp8=True, per_head=True, fused=True),
    dict(T=64, Hq=5, Hkv=1, fp8=True, adjacent=True, magnitude=1.3, skip=7),
    dict(T=33, Hq=3, Hkv=3, D=64, fp8=True, rot=32, axes=2, B=32),
    dict(T=153, Hq=7, Hkv=1, rot=112, axes=4, magnitude=0.7),
    dict(T=1217, Hq=2, Hkv=2, fused=True),
    dict(T=2435, Hq=2, Hkv=1, D=64, adjacent=True, rot=64, axes=3),
    dict(T=4867, Hq=1, Hkv=1, fp8=True, per_head=True, skip=5),
    dict(T=200, Hq=70, Hkv=70, D=64),
    dict(T=9, Hq=2, Hkv=2, far=2 ** 31 - 1),
    dict(T=9, Hq=2, Hkv=2, far=-2 ** 31, adjacent=True),
    dict(T=9, Hq=2, Hkv=2, base=1e-3),     # frequencies above one turn per position
]


@pytest.mark.parametrize("kw", CASES, ids=[",".join(f"{k}={v}" for k, v in c.items()) for c in CASES])
def test_matches_the_definition(api, oracle, cuda_device, kw):
    case = Case(cuda_device, **kw)
    guards = [Guarded(t.shape, t.dtype, cuda_device) for t in (case.q, case.k0, case.v0)]
    guards[1].tensor.copy_(case.k0)
    guards[2].tensor.copy_(case.v0)
    out, kc, vc = case.call(api, guards[0].tensor, None, guards[1].tensor, guards[2].tensor)
    torch.cuda.synchronize()
    case.check(oracle, out, kc, vc)
    for g in guards:
        g.check()
    assert api.device_errors() == 0


def test_in_place_equals_out_of_place(api, cuda_device):
    case = Case(cuda_device, T=300, Hq=8, Hkv=2, rot=96)
    out, kc, vc = case.call(api)
    q0 = case.q.clone()
    again, kc2, vc2 = case.call(api, out=case.q)
    assert again.data_ptr() == case.q.data_ptr()
    assert torch.equal(out, again) and torch.equal(kc, kc2) and torch.equal(vc, vc2)
    assert not torch.equal(q0, again)


def test_keys_alone(api, cuda_device):
    case = Case(cuda_device, T=20, Hq=4, Hkv=2)
    _, kc, vc = case.call(api)
    k2, v2 = case.k0.clone(), case.v0.clone()
    dev = cuda_device
    assert api.rope_append(None, case.k, case.v, case.pos[0].to(dev), case.freq.to(dev), case.slots.to(dev), k2, v2) is None
    assert torch.equal(kc, k2) and torch.equal(vc, v2)


def test_no_tokens(api, cuda_device):
    case = Case(cuda_device, T=4, Hq=2, Hkv=1)
    z = lambda t: t[:0].to(cuda_device)  # noqa: E731
    out = api.rope_append(z(case.q), z(case.k), z(case.v), case.pos[0, :0].to(cuda_device), case.freq.to(cuda_device), z(case.slots),
                          case.k0, case.v0)
    assert out.shape == (0, 2, 128) and api.device_errors() == 0


def test_infinities_and_nans_stay_in_their_pair(api, cuda_device):
    case = Case(cuda_device, T=3, Hq=2, Hkv=1, rot=64)
    base, _, _ = case.call(api)
    case.q[1, 0, 5] = float("nan")
    case.q[2, 1, 100] = float("inf")  # behind the rotated part
    out, _, _ = case.call(api)
    assert out[1, 0, 5].isnan() and out[1, 0, 37].isnan() and out[2, 1, 100] == float("inf")
    changed = (out != base).nonzero().tolist()
    assert sorted(changed) == [[1, 0, 5], [1, 0, 37], [2, 1, 100]]


def test_bad_slot_and_axis_are_flagged_and_skipped(api, cuda_device):
    from paged_kv_cache_193_gb300 import _lib
    case = Case(cuda_device, T=6, Hq=2, Hkv=1, axes=2)
    case.axis[3] = 2
    case.slots[4] = case.k0.shape[0] * case.B
    out, kc, vc = case.call(api)
    assert api.device_errors() == _lib.PA_DEVERR_BAD_SLOT | _lib.PA_DEVERR_BAD_AXIS
    case.axis[3] = 0
    case.slots[4] = -1
    out2, kc2, vc2 = case.call(api)
    assert torch.equal(out, out2) and torch.equal(kc, kc2) and torch.equal(vc, vc2) and api.device_errors() == 0


def test_captured_and_on_another_stream(api, oracle, cuda_device):
    case = Case(cuda_device, T=65, Hq=8, Hkv=2, fused=True, seed=3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, kc, vc = case.call(api, stream=side)
    side.synchronize()
    case.check(oracle, out, kc, vc)
    dev = cuda_device
    pos, freq, slots = case.pos[0].to(dev), case.freq.to(dev), case.slots.to(dev)
    k1, v1, o1 = case.k0.clone(), case.v0.clone(), torch.zeros_like(out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.rope_append(case.q, case.k, case.v, pos, freq, slots, k1, v1, kv_scale=case.kv_scale, out=o1)
    pos += 11
    case.pos += 11
    graph.replay()
    torch.cuda.synchronize()
    case.check(oracle, o1, k1, v1)


def test_rotated_attention_depends_on_differences_of_positions(api, cuda_device):
    """Through the cache: the same tokens moved 4096 positions on give the same attention up to roundings."""
    T, Hq, Hkv, D, B = 48, 4, 2, 128, 16
    g = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn(T, h, D, generator=g).to(torch.bfloat16).to(cuda_device) for h in (Hq, Hkv, Hkv))
    freq = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).to(cuda_device)
    tables = torch.arange(T // B, dtype=torch.int32, device=cuda_device)[None]
    outs = []
    for first in (0, 4096):
        kc = torch.zeros(T // B, Hkv, B, D, dtype=torch.bfloat16, device=cuda_device)
        vc = torch.zeros_like(kc)
        pos = torch.arange(first, first + T, dtype=torch.int32, device=cuda_device)
        rq = api.rope_append(q, k, v, pos, freq, torch.arange(T, dtype=torch.int32, device=cuda_device), kc, vc)
        outs.append(api.decode(rq[-1:].contiguous(), kc, vc, tables, torch.tensor([T], dtype=torch.int32, device=cuda_device)).float())
    # scores move by the bf16 roundings of q and k: 2 * 2^-8 |q||k| / sqrt(D) in the worst direction, |q||k| about D
    assert (outs[0] - outs[1]).abs().max() <= 2 * 2 * 2.0 ** -8 * D ** 0.5 * v.float().abs().max()


@pytest.mark.parametrize("scale", [1.0, 0.03, 1 / 448, 0.6250001, 1.9999999, 3.0, 1e-3, 7e-18, 9e17, 1e-20, 1e25, 1e-40, 3e38])
def test_every_value_into_an_e4m3_cache(api, oracle, cuda_device, scale):
    """All 65,536 bf16 values as V and as unrotated K (position 0 turns nothing): the codes of the plain append, which
    divides.  NaN only has to stay NaN."""
    D, Hkv = 128, 2
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(-1, Hkv, D)
    T = bits.shape[0]
    x = bits.to(cuda_device)
    kc, vc = (torch.zeros(T // 16, Hkv, 16, D, dtype=torch.uint8, device=cuda_device) for _ in range(2))
    k2, v2 = torch.zeros_like(kc), torch.zeros_like(vc)
    slots = torch.arange(T, dtype=torch.int32, device=cuda_device)
    zero = torch.zeros(T, dtype=torch.int32, device=cuda_device)
    freq = torch.ones(16, dtype=torch.float64, device=cuda_device)
    # elements from 32 on are not rotated at all
    api.rope_append(None, x, x, zero, freq, slots, kc, vc, kv_scale=scale)
    api.cache_append(x, x, slots, k2, v2, scale)
    nan = lambda c: (c & 0x7F) == 0x7F  # noqa: E731
    assert torch.equal(nan(vc), nan(v2)) and torch.equal(vc[~nan(v2)], v2[~nan(v2)])
    kr, kw = kc[..., 32:], k2[..., 32:]
    assert torch.equal(nan(kr), nan(kw)) and torch.equal(kr[~nan(kw)], kw[~nan(kw)])
    per_head = torch.full((Hkv,), scale, device=cuda_device)
    v3 = torch.zeros_like(vc)
    api.rope_append(None, x, x, zero, freq, slots, torch.zeros_like(kc), v3, k_scales=per_head, v_scales=per_head)
    assert torch.equal(v3, vc)
