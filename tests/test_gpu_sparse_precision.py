"""What the block-sparse attention rounds: its output once, and on the way no
more than the plain form in 32 bits does."""
import numpy as np
import pytest
import torch

import ops_reference as R
from paged_kv_cache_193_gb300 import _lib  # noqa: F401
from test_gpu_sparse import Case, api, f64  # noqa: F401  (api: a fixture)

pytestmark = pytest.mark.gpu

# A probability p goes into P V as two bf16 numbers, hi = p (1 - 2^-9) cut off to bf16 and the rest: below
# (2^-9 + 2^-7) p, rounded by at most 2^-8 of itself.  (2^-9 + 2^-7) 2^-8 < 2^-14.
TWO_BF16 = 2.0 ** -14

CASES = [
    dict(lens=[700, 64, 333], Hq=16, Hkv=1, top_k=9),
    dict(lens=[500, 501, 512, 3], Hq=5, Hkv=5, D=64, top_k=8),
    dict(lens=[900, 31, 32, 33], Hq=6, Hkv=2, B=32, top_k=7),
    dict(lens=[900, 31, 32, 33], Hq=24, Hkv=2, D=64, B=32, top_k=5),
    dict(lens=[5000], Hq=8, Hkv=2, top_k=40),
    dict(lens=[2000] * 90, Hq=16, Hkv=8, D=64, top_k=64),
]


@pytest.mark.parametrize("kw", CASES, ids=[str(i) for i in range(len(CASES))])
def test_probabilities_keep_their_bits(api, cuda_device, kw, monkeypatch):  # noqa: F811
    kw = dict(kw)
    top_k = kw.pop("top_k")
    case = Case(cuda_device, **kw)
    s, e = case.summaries(api)
    sel, cnt, out = case.attend(api, s, e, top_k)
    monkeypatch.setitem(R.HALF, "bf16x2", TWO_BF16)
    ref, bound = R.attend(f64(case.q), R.values(case.kc), R.values(case.vc), case.tables, case.lens, sel, cnt, case.scale,
                          *case.ref_scales, probability="bf16x2")
    off = np.abs(f64(out) - ref) - bound
    assert off.max() <= 0, f"{off.max()}: {(off > 0).mean():.3f} of the outputs are further off"


@pytest.mark.parametrize("D,B,Hq", [(128, 16, 4), (64, 32, 9)])
def test_one_token_gives_its_value(api, cuda_device, D, B, Hq):  # noqa: F811
    """Its probability is 1: the output is v, bit for bit, infinities and the largest numbers too."""
    case = Case(cuda_device, [1, 1, 1], Hq, 1, D, B)
    row = torch.randn(D, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    row[:4] = torch.tensor([float("inf"), float("-inf"), 3.38e38, -3.38e38]).to(torch.bfloat16)
    for i in range(3):
        case.vc[case.tables[i, 0], 0, 0] = (row * (1 + i)).to(cuda_device)
    s, e = case.summaries(api)
    _, _, out = case.attend(api, s, e, 4)
    for i in range(3):
        want = (row * (1 + i)).to(cuda_device)
        assert torch.equal(out[i], want[None].expand(Hq, D))


@pytest.mark.parametrize("fp8", [False, True])
def test_infinite_and_nan_values_reach_the_outputs_that_hold_them(api, cuda_device, fp8):  # noqa: F811
    case = Case(cuda_device, [777, 60], 8, 2, fp8=fp8)
    s, e = case.summaries(api)
    _, _, base = case.attend(api, s, e, 12)
    page = int(case.tables[0, 0])  # the first page is always read
    v = case.vc.view(torch.float8_e4m3fn) if fp8 else case.vc
    wrong = {3: float("nan")} if fp8 else {3: float("inf"), 70: float("-inf"), 99: float("nan")}
    for d, x in wrong.items():
        v[page, 1, 5, d] = torch.tensor(x).to(v.dtype)
    _, _, out = case.attend(api, s, e, 12)
    for d, x in wrong.items():
        got = out[0, 4:, d].float()
        assert got.isnan().all() if x != x else (got == x).all()
    rest = torch.ones_like(out, dtype=torch.bool)
    for d in wrong:
        rest[0, 4:, d] = False
    assert torch.equal(out[rest], base[rest]) and api.device_errors() == 0


@pytest.mark.parametrize("D,B,Hq", [(128, 16, 4), (64, 32, 9), (128, 32, 16), (64, 16, 1)])
def test_many_small_probabilities_count_in_full(api, cuda_device, D, B, Hq):  # noqa: F811
    """A token in each of the first 32 pages takes nearly all of the softmax and has value 0, thousands have some 2^-23 of
    it each and the same value.  The probabilities are fp16 times 2^7: each is off by at most 2^-25 2^-7 of the largest,
    and by 2^-16 of itself through its fp32 score."""
    n, few, value = 6000, 32, 384.0
    case = Case(cuda_device, [n], Hq, 1, D, B, fp8=True)
    case.kc.zero_()
    case.vc.zero_()
    k, v = case.kc.view(torch.float8_e4m3fn), case.vc.view(torch.float8_e4m3fn)
    live = torch.from_numpy(case.tables[0].astype(np.int64)).to(cuda_device)
    v[live] = torch.tensor(value).to(v.dtype)
    for page in live[:few].tolist():
        v[page, 0, 2] = torch.tensor(0.0).to(v.dtype)
        k[page, 0, 2, 0] = torch.tensor(16.0).to(k.dtype)
    case.q.zero_()
    # score of those: scale kv_scale 16 q0 = ln(2^23 / 1.5) and a little less from head to head
    q0 = torch.linspace(1.0, 0.98, Hq) * float(np.log(2.0 ** 23 / 1.5)) / (case.scale * case.kv_scale * 16)
    case.q[0, :, 0] = q0.to(torch.bfloat16).to(cuda_device)
    top_k = -(-n // B)
    sel = torch.arange(top_k, dtype=torch.int32, device=cuda_device)[None, None].contiguous()
    cnt = torch.full((1, 1), top_k, dtype=torch.int32, device=cuda_device)
    p = (n - few) * np.exp(-f64(case.q)[0, :, 0] * case.scale * case.kv_scale * 16)
    want = p / (few + p) * value * case.kv_scale
    bound = (2.0 ** -8 + 2.0 ** -16) * want + n * 2.0 ** -32 / few * value * case.kv_scale
    for splits in (1, 4):
        out = api.sparse_decode(case.q, case.kc, case.vc, case.bt, case.cl, sel, cnt, case.scale, case.kv_scale, splits=splits)
        off = np.abs(f64(out)[0] - want[:, None])
        assert (off <= bound[:, None]).all(), (off / want[:, None]).max()


@pytest.mark.parametrize("step", [8, 16])
@pytest.mark.parametrize("fp8", [False, True])
def test_scores_past_the_whole_numbers_of_fp32(api, cuda_device, fp8, step):  # noqa: F811
    """A score of 3 * 2^23 and one 8 above, or of 2^27 + 16 and one 16 above, in powers of two: fp32 steps by 2 and by 16
    there.  The second token, in a later page of the same warp, weighs 2^step against the first, all others nothing."""
    D, n = 128, 400
    case = Case(cuda_device, [n], 4, 1, D, 16, fp8=fp8)
    case.kc.zero_()
    case.vc.zero_()
    scale = float(np.float32(2) / np.float32(1.4426950408889634))
    assert np.float32(scale) * np.float32(1.4426950408889634) == 2  # a product q . k counts twice
    k, v = (c.view(torch.float8_e4m3fn) if fp8 else c for c in (case.kc, case.vc))
    put = lambda t, at, x: t.__setitem__(at, torch.tensor(x).to(t.dtype))  # noqa: E731
    dims, size, unit, extras = (1, 49152.0, 4.0, (0.0, 1.0)) if step == 8 else (8, 32768.0, 8.0, (1.0, 2.0))
    case.q.zero_()
    case.q[0, :, :dims], case.q[0, :, 64] = size, unit
    for page, extra, value in ((int(case.tables[0, 0]), extras[0], 3.0), (int(case.tables[0, 16]), extras[1], 5.0)):
        for d in range(dims):
            put(k, (page, 0, 2, d), 256.0)
        put(k, (page, 0, 2, 64), extra)
        put(v, (page, 0, 2), value)
    x = [2 * (dims * size * 256 + unit * e) for e in extras]
    assert x[1] - x[0] == step and all(np.float32(y) == y for y in x)
    sel = torch.arange(25, dtype=torch.int32, device=cuda_device)[None, None].contiguous()
    cnt = torch.full((1, 1), 25, dtype=torch.int32, device=cuda_device)
    want = (3 + 2 ** step * 5) / (1 + 2 ** step)
    for splits in (1, 2, 4, 8):
        out = api.sparse_decode(case.q, case.kc, case.vc, case.bt, case.cl, sel, cnt, scale, 1.0, splits=splits)
        off = (out.float() - want).abs().max().item()
        assert off <= 2.0 ** -8 * want, off
