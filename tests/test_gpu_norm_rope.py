"""Normalised rotate-and-append against its definition in 64 bits."""
import numpy as np
import pytest
import torch

import ops_reference as R
import test_gpu_rope
from gpu_helpers import Guarded
from paged_kv_cache_193_gb300 import workloads as W
from test_gpu_rope import Case, api  # noqa: F401  (api: a fixture)

pytestmark = pytest.mark.gpu
bf = torch.bfloat16


def normed(x, weight, offset, eps):
    """x [T, H, D] over its root mean square, times its head's weights, in 64 bits."""
    x = np.asarray(x, np.float64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return y if weight is None else y * (np.float64(offset) + weight)


# How far fp32 may be from `normed`, relative to it: the sum of squares 8 fused steps in a thread, one sum and three
# exchanges, all of positive terms, its mean and eps two more, 14 roundings of 2^-24, which the root halves; the root's own
# two units in the last place, 2^-22; x times it, offset + w and their product three.  14 / 2 + 4 + 3 = 14 times 2^-24.
# A sum offset + w rounds relative to itself, so cancellation in it costs nothing more.
SLACK = 14 * 2.0 ** -24


class NormCase(Case):
    def __init__(self, device, T, Hq, Hkv, weights="shared", offset=0.0, eps=1e-6, size=1.0, **kw):
        super().__init__(device, T, Hq, Hkv, **kw)
        D = self.q.shape[2]
        g = torch.Generator().manual_seed(77 + T)
        # rows of very different sizes, in place so that slices of one projection stay that
        for x in (self.q, self.k):
            x.mul_((size * torch.exp(torch.randn(T, x.shape[1], 1, generator=g) * 1.5)).to(bf).to(device))
        shape = {"shared": lambda h: (D,), "heads": lambda h: (h, D), "none": lambda h: None}[weights]
        self.w = [None if shape(h) is None else (1 - offset + 0.3 * torch.randn(shape(h), generator=g)).to(bf).to(device) for h in (Hq, Hkv)]
        self.offset, self.eps = offset, eps

    def call(self, api, out=None, stream=None, kc=None, vc=None, **kw):  # noqa: F811
        dev = self.device
        kc = self.k0.clone() if kc is None else kc
        vc = self.v0.clone() if vc is None else vc
        ks, vs = (None, None) if self.scales is None else (self.scales[0].to(dev), self.scales[1].to(dev))
        pos = (self.pos if self.pos.shape[0] > 1 else self.pos[0]).to(dev)
        args = dict(q_weight=self.w[0], k_weight=self.w[1], eps=self.eps, weight_offset=self.offset,
                    pair_axis=None if self.axis is None else self.axis.to(dev), adjacent=self.adjacent,
                    magnitude=self.magnitude, kv_scale=self.kv_scale, k_scales=ks, v_scales=vs, out=out, stream=stream)
        args.update(kw)
        out = api.norm_rope_append(self.q, self.k, self.v, pos, self.freq.to(dev), self.slots.to(dev), kc, vc, **args)
        return out, kc, vc

    def check(self, oracle, out, kc, vc):
        f64 = lambda t: t.float().cpu().numpy().astype(np.float64)  # noqa: E731
        how = (self.pos.numpy(), self.freq.numpy(), None if self.axis is None else self.axis.numpy(), self.adjacent, self.magnitude)

        def made(x, w):
            y = normed(f64(x), None if w is None else f64(w), self.offset, self.eps)
            # a turn moves an error of a pair's two elements into both
            part = np.abs(y)
            a, b = (slice(0, self.rot, 2), slice(1, self.rot, 2)) if self.adjacent else (slice(0, self.rot // 2), slice(self.rot // 2, self.rot))
            both = self.magnitude * (part[..., a] + part[..., b])
            part[..., a] = part[..., b] = both
            return R.rotate(y, *how), 1.01 * (R.rotate_slack(y, *how) + SLACK * part)

        ref, slack = made(self.q, self.w[0])
        off = np.abs(f64(out) - ref) - (R.HALF["bf16"] * np.abs(ref) + 1.01 * slack)
        assert off.max() <= 0, f"q: {off.max()}"
        live = (self.slots >= 0).numpy()
        slot = self.slots.numpy()[live]
        ref, slack = (x[live] for x in made(self.k, self.w[1]))
        got = R.values(kc).transpose(0, 2, 1, 3).reshape(-1, self.Hkv, ref.shape[-1])
        if not self.fp8:
            bound = R.HALF["bf16"] * np.abs(ref) + 1.01 * slack
        else:
            s = np.full(self.Hkv, np.float64(np.float32(self.kv_scale))) if self.scales is None else self.scales[0].numpy().astype(np.float64)
            ref, slack = np.clip(ref / s[:, None], -448, 448), slack / s[:, None]
            bound = np.maximum(R.HALF["e4m3"] * np.abs(ref), 2.0 ** -10) + 1.1 * slack + 2.0 ** -23 * np.abs(ref)
        off = np.abs(got[slot] - ref) - bound
        assert off.size == 0 or off.max() <= 0, f"k: {off.max()}"
        # v is the plain append's, whatever the norm
        plain, _, want_v = test_gpu_rope.Case.call(self, _api())
        assert np.array_equal(W.bits(vc), W.bits(want_v))
        untouched = np.ones(got.shape[0], bool)
        untouched[slot] = False
        rows = lambda t: W.bits(t).transpose(0, 2, 1, 3).reshape(got.shape)  # noqa: E731
        assert np.array_equal(rows(kc)[untouched], rows(self.k0)[untouched])


def _api():
    from paged_kv_cache_193_gb300 import api as a
    return a


CASES = [
    dict(T=1, Hq=8, Hkv=2),
    dict(T=1, Hq=1, Hkv=1, D=64, fused=True, adjacent=True, weights="none"),
    dict(T=5, Hq=4, Hkv=4, rot=16, weights="heads"),
    dict(T=37, Hq=16, Hkv=2, fused=True, skip=3, offset=1.0),
    dict(T=37, Hq=6, Hkv=3, D=64, B=32, adjacent=True, rot=48, axes=3, fused=True, weights="heads", offset=1.0),
    dict(T=64, Hq=32, Hkv=2, fp8=True, per_head=True, fused=True),
    dict(T=64, Hq=5, Hkv=1, fp8=True, adjacent=True, magnitude=1.3, skip=7, weights="heads"),
    dict(T=33, Hq=3, Hkv=3, D=64, fp8=True, rot=32, axes=2, B=32, weights="none"),
    dict(T=153, Hq=7, Hkv=1, rot=112, axes=4, magnitude=0.7, offset=-0.5),
    dict(T=1217, Hq=2, Hkv=2, fused=True),
    dict(T=2435, Hq=2, Hkv=1, D=64, adjacent=True, rot=64, axes=3, weights="heads"),
    dict(T=4867, Hq=1, Hkv=1, fp8=True, per_head=True, skip=5),
    dict(T=200, Hq=70, Hkv=70, D=64, weights="heads", offset=1.0),
    dict(T=9, Hq=2, Hkv=2, size=1e-4, eps=1e-6),        # rows near sqrt(eps)
    dict(T=9, Hq=2, Hkv=2, size=1e-9, eps=1e-12),       # and far below
    dict(T=9, Hq=2, Hkv=2, size=1e15, eps=1e-5),
    dict(T=9, Hq=2, Hkv=2, eps=2.0),
]


@pytest.mark.parametrize("kw", CASES, ids=[",".join(f"{k}={v}" for k, v in c.items()) for c in CASES])
def test_matches_the_definition(api, oracle, cuda_device, kw):  # noqa: F811
    case = NormCase(cuda_device, **kw)
    guards = [Guarded(t.shape, t.dtype, cuda_device) for t in (case.q, case.k0, case.v0)]
    guards[1].tensor.copy_(case.k0)
    guards[2].tensor.copy_(case.v0)
    out, kc, vc = case.call(api, guards[0].tensor, None, guards[1].tensor, guards[2].tensor)
    torch.cuda.synchronize()
    case.check(oracle, out, kc, vc)
    for g in guards:
        g.check()
    assert api.device_errors() == 0


def test_in_place_and_keys_alone(api, cuda_device):  # noqa: F811
    case = NormCase(cuda_device, T=300, Hq=8, Hkv=2, rot=96, weights="heads")
    out, kc, vc = case.call(api)
    dev = cuda_device
    k2, v2 = case.k0.clone(), case.v0.clone()
    assert api.norm_rope_append(None, case.k, case.v, case.pos[0].to(dev), case.freq.to(dev), case.slots.to(dev), k2, v2,
                                k_weight=case.w[1], eps=case.eps, kv_scale=case.kv_scale) is None
    assert torch.equal(kc, k2) and torch.equal(vc, v2)
    again, k3, _ = case.call(api, out=case.q)
    assert again.data_ptr() == case.q.data_ptr() and torch.equal(out, again) and torch.equal(kc, k3)


def test_a_row_of_zeros_and_odd_values_stay_in_their_row(api, cuda_device):  # noqa: F811
    case = NormCase(cuda_device, T=4, Hq=2, Hkv=1, rot=64)
    base, kc, _ = case.call(api)
    case.q[0, 1] = 0
    case.q[1, 0, 5] = float("nan")
    case.q[2, 1, 100] = float("inf")
    out, k2, _ = case.call(api)
    assert (out[0, 1] == 0).all() and out[1, 0].isnan().all() and torch.equal(kc, k2)
    # over an infinite root the others are 0, and infinity times 0 is NaN
    assert out[2, 1, 100].isnan() and (out[2, 1, :64] == 0).all()
    same = torch.ones(4, 2, dtype=torch.bool)
    same[0, 1] = same[1, 0] = same[2, 1] = False
    assert torch.equal(out[same], base[same])


def test_captured_and_on_another_stream(api, oracle, cuda_device):  # noqa: F811
    case = NormCase(cuda_device, T=65, Hq=8, Hkv=2, fused=True, seed=3)
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
        api.norm_rope_append(case.q, case.k, case.v, pos, freq, slots, k1, v1, q_weight=case.w[0], k_weight=case.w[1], eps=case.eps,
                             kv_scale=case.kv_scale, out=o1)
    pos += 11
    case.pos += 11
    case.w[0].mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    case.check(oracle, o1, k1, v1)


def test_the_same_as_the_rotation_of_rows_that_need_no_norm(api, cuda_device):  # noqa: F811
    """Rows of plus and minus one have a mean square of 1: what rope_append gives, but for the norm's own roundings, which
    bf16 hides except at a border."""
    case = NormCase(cuda_device, T=50, Hq=4, Hkv=2, weights="none", eps=1e-12)
    for x in (case.q, case.k):
        x.copy_(torch.where(x > 0, 1.0, -1.0))
    out, kc, vc = case.call(api)
    want, k2, v2 = test_gpu_rope.Case.call(case, api)
    assert torch.equal(vc, v2) and (out.float() - want.float()).abs().max() <= 2.0 ** -7
    assert (out != want).float().mean() < 0.01 and (kc.float() - k2.float()).abs().max() <= 2.0 ** -7


def test_a_sparse_step_of_normalised_rows(api, cuda_device):  # noqa: F811
    """SparseDecodeStep with a norm: the same as its parts called one after the other."""
    dev = cuda_device
    g = torch.Generator().manual_seed(8)
    S, Hq, Hkv, D, B, MB = 3, 8, 2, 128, 16, 10
    kv = torch.randn(2, S * MB, Hkv, B, D, generator=g).to(bf).to(dev)
    tables = torch.randperm(S * MB, generator=g).view(S, MB).to(torch.int32).to(dev)
    lens = torch.tensor([150, 33, 80], dtype=torch.int32, device=dev)
    freq = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).to(dev)
    w = (1 + 0.2 * torch.randn(2, D, generator=g)).to(bf).to(dev)
    q, k, v = (torch.randn(S, h, D, generator=g).to(bf).to(dev) for h in (Hq, Hkv, Hkv))
    s, e = api.alloc_block_summary(kv[0])
    api.block_summary(kv[0], torch.arange(B - 1, S * MB * B, B, dtype=torch.int32, device=dev), s, e)
    k1, v1, k2, v2 = kv[0].clone(), kv[1].clone(), kv[0].clone(), kv[1].clone()
    step = api.SparseDecodeStep(k1, v1, tables, lens, lens - 1, freq, Hq, 4, q_weight=w[0], k_weight=w[1], eps=1e-5,
                                summary=s.clone(), exponents=e.clone())
    out = step(q, k, v)
    slots = api.slot_mapping(tables, lens, B)
    rq = api.norm_rope_append(q, k, v, lens - 1, freq, slots, k2, v2, q_weight=w[0], k_weight=w[1], eps=1e-5)
    api.block_summary(k2, slots, s, e)
    assert torch.equal(out, api.sparse_attend(rq, k2, v2, s, e, tables, lens, 4)) and torch.equal(k1, k2) and torch.equal(v1, v2)
    plain = api.SparseDecodeStep(kv[0].clone(), kv[1].clone(), tables, lens, lens - 1, freq, Hq, 4, summary=s.clone(), exponents=e.clone())
    assert not plain.norm and not torch.equal(plain(q, k, v), out)


@pytest.mark.parametrize("heads", [False, True])
def test_weights_that_the_call_before_writes(api, cuda_device, heads):  # noqa: F811
    """Each call's weights are the query rows that the one before has written, without a wait between: the same as with one."""
    dev = cuda_device
    g = torch.Generator().manual_seed(3)
    T, H, D = 40, 24, 64
    kc, vc = (torch.zeros(H, H, 16, D, dtype=bf, device=dev) for _ in range(2))
    freq = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).to(dev)
    pos = torch.arange(T, dtype=torch.int32, device=dev)
    q, k, v = (torch.randn(T, H, D, generator=g).to(bf).to(dev) for _ in range(3))
    bufs = [torch.ones(T, H, D, dtype=bf, device=dev) for _ in range(2)]

    def chain(wait):
        bufs[0].fill_(1)
        for i in range(30):
            w = bufs[i % 2][i] if heads else bufs[i % 2][i, i % H]
            api.norm_rope_append(q, k, v, pos, freq, pos, kc, vc, q_weight=w, k_weight=w, out=bufs[1 - i % 2])
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return bufs[0].clone(), kc.clone()

    want = chain(True)
    for _ in range(5):
        for a, b in zip(chain(False), want):
            assert torch.equal(a, b)
    assert want[0].float().abs().max() < 2.0 ** 20 and api.device_errors() == 0
