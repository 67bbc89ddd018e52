"""Block summary, block choice and block-sparse decode against their
definitions in 64 bits: bit for bit where they give whole numbers, within a
derived bound where they give attention outputs."""
import numpy as np
import pytest
import torch

import ops_reference as R
from gpu_helpers import Guarded
from paged_kv_cache_193_gb300 import _lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api(cuda_device):
    from paged_kv_cache_193_gb300 import api as a
    a._lib_handle()
    return a


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def pool(shape, fp8, g, device, gain=1.0):
    x = torch.randn(shape, generator=g) * gain
    return ((x * 16).to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else x.to(torch.bfloat16)).to(device)


# ---- block summary --------------------------------------------------------------

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,B,Hkv,T", [(128, 16, 8, 1), (128, 16, 3, 33), (128, 32, 8, 257), (64, 16, 1, 100), (64, 32, 2, 64),
                                       (64, 32, 5, 2000), (64, 16, 9, 600), (128, 32, 20, 300), (64, 16, 2, 5000)])
def test_summary_bit_exact(api, cuda_device, D, B, Hkv, T, fp8):
    g = torch.Generator().manual_seed(D + B + Hkv + T)
    NB = max(4, T // 4)
    kc = pool((NB, Hkv, B, D), fp8, g, cuda_device)
    if not fp8:  # values over the exponents' whole range, and past both of its ends
        kc *= (2.0 ** torch.randint(-80, 70, (NB, Hkv, 1, 1), generator=g).float()).to(cuda_device)
    else:
        kc[0] = 0
        kc[1] = 0x80  # minus zero
    slots = torch.randint(-3, NB * B, (T,), generator=g).to(torch.int32)
    slots[::2] = (slots[::2].abs() // B) * B + B - 1  # every other one ends a block, some of them the same block
    s, e = Guarded((NB, Hkv, 2, D), torch.int8, cuda_device, 5), Guarded((NB, Hkv), torch.int8, cuda_device, 6)
    api.block_summary(kc, slots.to(cuda_device), s.tensor, e.tensor)
    want_s, want_e = np.full((NB, Hkv, 2, D), 5, np.int8), np.full((NB, Hkv), 6, np.int8)
    R.block_summary(R.values(kc), slots.numpy(), want_s, want_e)
    assert np.array_equal(e.tensor.cpu().numpy(), want_e)
    assert np.array_equal(s.tensor.cpu().numpy(), want_s)
    s.check()
    e.check()
    assert api.device_errors() == 0


@pytest.mark.parametrize("fp8,bad", [(False, float("nan")), (False, float("inf")), (False, float("-inf")), (True, float("nan"))])
def test_summary_of_a_page_that_is_not_finite(api, cuda_device, fp8, bad):
    g = torch.Generator().manual_seed(3)
    kc = pool((3, 2, 16, 64), fp8, g, cuda_device)
    if fp8:
        kc[1, 0, 7, 63] = 0x7F
    else:
        kc[1, 0, 7, 63] = bad
    s, e = api.alloc_block_summary(kc)
    api.block_summary(kc, torch.tensor([15, 31, 47], dtype=torch.int32, device=cuda_device), s, e)
    want_s, want_e = np.zeros((3, 2, 2, 64), np.int8), np.zeros((3, 2), np.int8)
    R.block_summary(R.values(kc), [15, 31, 47], want_s, want_e)
    assert want_e[1, 0] == 127
    assert np.array_equal(s.cpu().numpy(), want_s) and np.array_equal(e.cpu().numpy(), want_e)


def test_summary_slot_outside_the_pool_is_flagged(api, cuda_device):
    kc = torch.ones(2, 1, 16, 64, dtype=torch.bfloat16, device=cuda_device)
    s, e = api.alloc_block_summary(kc)
    api.block_summary(kc, torch.tensor([47, 2 ** 31 - 1, 31], dtype=torch.int32, device=cuda_device), s, e)
    assert api.device_errors() == _lib.PA_DEVERR_BAD_SLOT
    assert (s[0] == 0).all() and (s[1] == 64).all()
    api.block_summary(kc, torch.empty(0, dtype=torch.int32, device=cuda_device), s, e)


def test_summary_of_as_many_slots_as_an_int_counts(api, cuda_device):
    kc = torch.ones(2, 1, 16, 64, dtype=torch.bfloat16, device=cuda_device)
    s, e = api.alloc_block_summary(kc)
    slots = torch.full((2 ** 31 - 1,), -1, dtype=torch.int32, device=cuda_device)
    slots[-1] = 31
    api.block_summary(kc, slots, s, e)
    assert api.device_errors() == 0
    assert (s[0] == 0).all() and (s[1] == 64).all()


# ---- a paged case ---------------------------------------------------------------

class Case:
    def __init__(self, device, lens, Hq, Hkv, D=128, B=16, fp8=False, per_head=False, seed=0, spare=3, width=None):
        g = torch.Generator().manual_seed(seed + 17 * len(lens) + Hq)
        self.device, self.B, self.fp8 = device, B, fp8
        S = len(lens)
        need = [-(-n // B) for n in lens]
        NB = sum(need) + spare
        self.kc = pool((NB, Hkv, B, D), fp8, g, device)
        self.vc = pool((NB, Hkv, B, D), fp8, g, device)
        perm = torch.randperm(NB, generator=g).tolist()
        self.tables = np.full((S, width or max(1, max(need))), -1, np.int32)
        for s in range(S):
            self.tables[s, :need[s]] = [perm.pop() for _ in range(need[s])]
        self.lens = np.array(lens, np.int32)
        # rows behind each context, and pages that no table names: NaN
        live = np.zeros((NB, B), bool)
        for s in range(S):
            for t in range(lens[s]):
                live[self.tables[s, t // B], t % B] = True
        dead = torch.from_numpy(~live)[:, None, :, None].to(device)
        for c in (self.kc, self.vc):
            c.masked_fill_(dead, 0x7F if fp8 else float("nan"))
        self.q = torch.randn(S, Hq, D, generator=g).to(torch.bfloat16).to(device)
        self.k_scales = self.v_scales = None
        self.kv_scale = 1 / 16 if fp8 else 1.0
        ks = vs = np.full(Hkv, self.kv_scale)
        if per_head:
            self.k_scales, self.v_scales = ((0.04 + 0.04 * torch.rand(Hkv, generator=g)).to(device) for _ in range(2))
            ks, vs = f64(self.k_scales), f64(self.v_scales)
        self.ref_scales = (ks, vs)
        self.bt, self.cl = torch.from_numpy(self.tables).to(device), torch.from_numpy(self.lens).to(device)
        self.scale = 1.0 / D ** 0.5
        self.Hkv = Hkv

    def summaries(self, api):
        s, e = api.alloc_block_summary(self.kc)
        full = [self.tables[i, j] * self.B + self.B - 1 for i, n in enumerate(self.lens) for j in range(n // self.B)]
        api.block_summary(self.kc, torch.tensor(full, dtype=torch.int32, device=self.device), s, e)
        return s, e

    def check(self, out, sel, cnt):
        ref, bound = R.attend(f64(self.q), R.values(self.kc), R.values(self.vc), self.tables, self.lens, sel, cnt, self.scale,
                              *self.ref_scales, probability="fp16" if self.fp8 else "bf16")
        off = np.abs(f64(out) - ref) - bound
        assert np.isfinite(f64(out)).all()
        assert off.max() <= 0, f"{off.max()} at {np.unravel_index(off.argmax(), off.shape)}"

    def attend(self, api, s, e, top_k, sink=1, recent=2, **kw):
        S, Hq, D = self.q.shape
        sel = Guarded((S, self.Hkv, top_k), torch.int32, self.device, -9)
        cnt = Guarded((S, self.Hkv), torch.int32, self.device, -9)
        out = Guarded((S, Hq, D), torch.bfloat16, self.device, float("nan"))
        api.sparse_attend(self.q, self.kc, self.vc, s, e, self.bt, self.cl, top_k, sink, recent, self.scale, self.kv_scale,
                          self.k_scales, self.v_scales, sel.tensor, cnt.tensor, out.tensor, **kw)
        torch.cuda.synchronize()
        for gd in (sel, cnt, out):
            gd.check()
        return sel.tensor.cpu().numpy(), cnt.tensor.cpu().numpy(), out.tensor


SHAPES = [
    dict(lens=[1], Hq=4, Hkv=1, top_k=4),
    dict(lens=[0, 1, 15, 16, 17, 300, 0], Hq=8, Hkv=2, top_k=6),
    dict(lens=[700, 64, 333], Hq=16, Hkv=1, top_k=9),
    dict(lens=[500, 501, 512], Hq=5, Hkv=5, D=64, top_k=8, sink=0, recent=1),
    dict(lens=[900, 31, 32, 33], Hq=6, Hkv=2, B=32, top_k=7, sink=2, recent=3),
    dict(lens=[900, 31, 32, 33], Hq=24, Hkv=2, D=64, B=32, top_k=5),
    dict(lens=[640, 5, 129], Hq=8, Hkv=2, fp8=True, top_k=10),
    dict(lens=[640, 5, 129], Hq=11, Hkv=1, fp8=True, per_head=True, top_k=11),
    dict(lens=[1000, 77], Hq=4, Hkv=4, D=64, B=32, fp8=True, per_head=True, top_k=6),
    dict(lens=[1000, 77], Hq=32, Hkv=2, B=32, fp8=True, top_k=13),
    dict(lens=[333, 444], Hq=10, Hkv=2, D=64, fp8=True, top_k=5, sink=1, recent=4),   # nothing left to choose
    dict(lens=[5000], Hq=8, Hkv=2, top_k=40),
    dict(lens=[20000], Hq=4, Hkv=1, D=64, top_k=100),
    dict(lens=[3000] * 40, Hq=16, Hkv=8, D=64, top_k=16),
    dict(lens=[400, 100], Hq=4, Hkv=2, D=64, top_k=1000),                              # more than there are
]


@pytest.mark.parametrize("kw", SHAPES, ids=[",".join(f"{k}={v if k != 'lens' else len(v)}" for k, v in c.items()) + f"-{i}"
                                            for i, c in enumerate(SHAPES)])
def test_choice_bit_exact_and_attention_in_bounds(api, cuda_device, kw):
    kw = dict(kw)
    top_k, sink, recent = kw.pop("top_k"), kw.pop("sink", 1), kw.pop("recent", 2)
    case = Case(cuda_device, **kw)
    s, e = case.summaries(api)
    sel, cnt, out = case.attend(api, s, e, top_k, sink, recent)
    want_sel, want_cnt = R.select(f64(case.q), s.cpu().numpy(), e.cpu().numpy(), case.tables, case.lens, case.B, top_k, sink, recent)
    assert np.array_equal(cnt, want_cnt)
    assert np.array_equal(sel, want_sel)
    case.check(out, sel, cnt)
    # the two calls apart give the same
    sel2, cnt2 = api.sparse_select(case.q, s, e, case.bt, case.cl, case.B, top_k, sink, recent)
    assert np.array_equal(sel2.cpu().numpy(), sel) and np.array_equal(cnt2.cpu().numpy(), cnt)
    out2 = api.sparse_decode(case.q, case.kc, case.vc, case.bt, case.cl, sel2, cnt2, case.scale, case.kv_scale, case.k_scales,
                             case.v_scales)
    case.check(out2, sel, cnt)  # its parts may be joined in another order
    assert api.device_errors() == 0


@pytest.mark.parametrize("splits", [1, 2, 4, 8])
@pytest.mark.parametrize("D,B,Hq,fp8", [(128, 16, 4, False), (64, 32, 9, True)])
def test_every_split(api, cuda_device, splits, D, B, Hq, fp8):
    case = Case(cuda_device, [1, 2 * B, 1111, 0, 40], Hq, 1, D, B, fp8)
    s, e = case.summaries(api)
    sel, cnt = api.sparse_select(case.q, s, e, case.bt, case.cl, B, 23)
    out = api.sparse_decode(case.q, case.kc, case.vc, case.bt, case.cl, sel, cnt, case.scale, case.kv_scale, splits=splits)
    case.check(out, sel.cpu().numpy(), cnt.cpu().numpy())
    assert api.device_errors() == 0


def test_all_pages_is_the_dense_decode(api, cuda_device):
    case = Case(cuda_device, [500, 1, 77, 0], 8, 2)
    s, e = case.summaries(api)
    _, _, out = case.attend(api, s, e, 32)
    dense = api.decode(case.q, case.kc, case.vc, case.bt, case.cl, case.scale)
    # both are within the bound of the same exact value
    sel = np.tile(np.arange(32, dtype=np.int32), (4, 2, 1))
    cnt = np.array([[-(-n // 16)] * 2 for n in case.lens], np.int32)
    case.check(out, sel, cnt)
    case.check(dense, sel, cnt)


@pytest.mark.parametrize("D,Hq,S,pages", [(128, 1, 1, 1025), (128, 4, 1, 4097), (64, 16, 3, 513), (128, 16, 40, 130), (64, 2, 320, 70)])
def test_choice_among_many_ties(api, cuda_device, D, Hq, S, pages):
    """Random bounds with few values, so that most scores are shared: the lower index wins, across warps and CTAs."""
    g = torch.Generator().manual_seed(pages)
    NB, Hkv = 300, 1
    s = torch.randint(0, 2, (NB, Hkv, 2, D), generator=g).to(torch.int8)
    s[:, :, :, 2:] = 0
    s[:, :, 1] = -s[:, :, 1]
    e = torch.randint(0, 2, (NB, Hkv), generator=g).to(torch.int8)
    e[7] = 127
    q = torch.randn(S, Hq, D, generator=g).to(torch.bfloat16)
    tables = torch.randint(0, NB, (S, pages), generator=g).to(torch.int32)
    lens = torch.full((S,), pages * 16, dtype=torch.int32)
    lens[-1] = max(1, pages * 16 - 131)
    for top_k, sink, recent in ((pages // 2, 3, 5), (7, 0, 1), (pages - 1, 1, 1), (pages, 1, 1)):
        sel, cnt = api.sparse_select(*(t.to(cuda_device) for t in (q, s, e, tables, lens)), 16, top_k, sink, recent)
        want_sel, want_cnt = R.select(f64(q), s.numpy(), e.numpy(), tables.numpy(), lens.numpy(), 16, top_k, sink, recent)
        assert np.array_equal(cnt.cpu().numpy(), want_cnt)
        assert np.array_equal(sel.cpu().numpy(), want_sel)
    assert api.device_errors() == 0


@pytest.mark.parametrize("D,G,S,pages,top_k,sink,recent", [
    # candidates up to and just past the numbers that are ranked directly (one to a thread, 500 in a cluster)
    (64, 2, 304, 131, 20, 1, 2), (64, 2, 304, 132, 20, 1, 2), (64, 2, 304, 259, 20, 1, 2), (64, 2, 304, 260, 20, 1, 2), (128, 1, 2, 503, 90, 1, 2), (128, 1, 2, 504, 90, 1, 2),
    (128, 9, 3, 257, 40, 0, 1), (64, 16, 1, 513, 200, 0, 1),
    # one candidate more than is wanted, and lists longer than the candidates
    (128, 4, 1, 65, 64, 1, 2), (64, 1, 5, 130, 129, 60, 68), (128, 2, 2, 900, 700, 300, 350), (64, 3, 320, 900, 700, 300, 350),
    # a few pages to a warp of the last CTA, and none
    (128, 4, 1, 1029, 100, 1, 2), (64, 4, 3, 2081, 33, 1, 1), (64, 4, 60, 700, 33, 1, 1),
])
def test_choice_at_its_borders(api, cuda_device, D, G, S, pages, top_k, sink, recent):
    """Alone and followed by the attention, bit for bit; scores of any value, then few values."""
    g = torch.Generator().manual_seed(pages + top_k)
    NB, Hkv, B = 400, 2, 16
    kc, vc = (torch.randn(NB, Hkv, B, D, generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(S, G * Hkv, D, generator=g).to(torch.bfloat16)
    tables = torch.randint(0, NB, (S, pages), generator=g).to(torch.int32)
    lens = torch.full((S,), pages * B, dtype=torch.int32) - torch.randint(0, B, (S,), generator=g).to(torch.int32)
    dev = [t.to(cuda_device) for t in (q, kc, vc, tables, lens)]
    rows = sorted({0, S // 2, S - 1})
    for few_values in (False, True):
        s = torch.randint(-127, 128, (NB, Hkv, 2, D), generator=g).to(torch.int8).sort(dim=2, descending=True).values
        e = torch.randint(-9, -6, (NB, Hkv), generator=g).to(torch.int8)
        if few_values:
            s[:, :, :, 1:] = 0
            s[:, :, :, 0] = s[:, :, :, 0].sign()
            e[:] = -7
        se, ee = s.to(cuda_device), e.to(cuda_device)
        sel, cnt = api.sparse_select(dev[0], se, ee, dev[3], dev[4], B, top_k, sink, recent)
        sel2, cnt2 = torch.zeros_like(sel), torch.zeros_like(cnt)
        out = api.sparse_attend(*dev[:3], se, ee, *dev[3:], top_k, sink, recent, selected=sel2, counts=cnt2)
        assert torch.equal(sel, sel2) and torch.equal(cnt, cnt2)
        want_sel, want_cnt = R.select(f64(q)[rows], s.numpy(), e.numpy(), tables.numpy()[rows], lens.numpy()[rows], B, top_k, sink, recent)
        assert np.array_equal(sel.cpu().numpy()[rows], want_sel) and np.array_equal(cnt.cpu().numpy()[rows], want_cnt)
        one = np.ones(Hkv)
        ref, bound = R.attend(f64(q)[rows], R.values(kc), R.values(vc), tables.numpy()[rows], lens.numpy()[rows], want_sel, want_cnt,
                              D ** -0.5, one, one)
        for o in (out, api.sparse_decode(*dev[:3], *dev[3:], sel, cnt)):
            assert (np.abs(f64(o)[rows] - ref) <= bound).all()
    assert api.device_errors() == 0


@pytest.mark.parametrize("D", [64, 128])
def test_the_largest_whole_sums(api, cuda_device, D):
    """Queries and bounds at +-127 throughout: sums of up to 127 * 127 * D that differ by single units."""
    g = torch.Generator().manual_seed(D)
    NB, S = 90, 4
    s = torch.full((NB, 1, 2, D), 127, dtype=torch.int8)
    s[:, :, 1] = -127
    s[torch.arange(NB), 0, 0, torch.randint(0, D, (NB,), generator=g)] -= torch.randint(0, 3, (NB,), generator=g).to(torch.int8)
    s[torch.arange(NB), 0, 1, torch.randint(0, D, (NB,), generator=g)] += torch.randint(0, 3, (NB,), generator=g).to(torch.int8)
    e = torch.zeros(NB, 1, dtype=torch.int8)
    q = torch.full((S, 9, D), 127.0)
    q[1] = -127
    q[2] = torch.randint(0, 2, (9, D), generator=g) * 254.0 - 127
    q[3, :, ::2] = -127
    q = (q + torch.randint(-1, 1, q.shape, generator=g) * q.sign()).to(torch.bfloat16)
    tables, lens = torch.arange(NB).to(torch.int32)[None].repeat(S, 1), torch.full((S,), NB * 16, dtype=torch.int32)
    sel, _ = api.sparse_select(*(t.to(cuda_device) for t in (q, s, e, tables, lens)), 16, 30, 0, 1)
    want, _ = R.select(f64(q), s.numpy(), e.numpy(), tables.numpy(), lens.numpy(), 16, 30, 0, 1)
    assert np.array_equal(sel.cpu().numpy(), want)


def test_choice_with_extreme_bounds_and_queries(api, cuda_device):
    """Exponents at both ends, the largest whole numbers, zero and non-finite queries."""
    g = torch.Generator().manual_seed(12)
    NB, D, pages = 64, 128, 64
    s = torch.randint(-127, 128, (NB, 1, 2, D), generator=g).to(torch.int8)
    s, _ = s.sort(dim=2, descending=True)
    s[3, 0] = torch.tensor([[127], [-127]], dtype=torch.int8)
    e = torch.randint(-60, 41, (NB, 1), generator=g).to(torch.int8)
    e[0:4] = 40
    e[10] = 127
    tables = torch.randperm(NB, generator=g).to(torch.int32)[None].repeat(6, 1)
    q = torch.randn(6, 3, D, generator=g).to(torch.bfloat16)
    q[1] = 0
    q[2, 0, 5] = float("nan")
    q[3] = float("inf")
    q[4] *= 2.0 ** 100
    q[5] *= 2.0 ** -100
    lens = torch.full((6,), pages * 16 - 1, dtype=torch.int32)
    sel, cnt = api.sparse_select(*(t.to(cuda_device) for t in (q, s, e, tables, lens)), 16, 20, 1, 1)
    want_sel, _ = R.select(f64(q), s.numpy(), e.numpy(), tables.numpy(), lens.numpy(), 16, 20, 1, 1)
    assert np.array_equal(sel.cpu().numpy(), want_sel)


def test_nan_key_reaches_the_output_and_nan_query_only_its_head(api, cuda_device):
    case = Case(cuda_device, [800], 4, 2, D=64)
    b = int(case.tables[0, 20])
    case.kc[b, 1, 3, 3] = float("nan")
    case.q[0, 0, 0] = float("nan")
    s, e = case.summaries(api)
    sel, _, out = case.attend(api, s, e, 8)
    assert 20 in sel[0, 1]  # a page that is not finite is always taken
    nan = out.isnan().all(-1)[0].tolist()
    assert nan == [True, False, True, True]
    assert out[0, 1].isfinite().all()


def test_scores_of_minus_infinity(api, cuda_device):
    """Keys at minus infinity along the query: their tokens weigh nothing, whole pages of them too."""
    D, B = 64, 16
    kc = torch.zeros(4, 1, B, D, dtype=torch.bfloat16, device=cuda_device)
    vc = torch.randn(4, 1, B, D, device=cuda_device).to(torch.bfloat16)
    q = torch.zeros(1, 1, D, dtype=torch.bfloat16, device=cuda_device)
    q[..., 0] = 1
    kc[:2, :, :, 0] = float("-inf")
    kc[2, :, 3, 0] = float("-inf")
    bt, cl = torch.arange(4, dtype=torch.int32, device=cuda_device)[None], torch.tensor([64], dtype=torch.int32, device=cuda_device)
    sel = torch.arange(4, dtype=torch.int32, device=cuda_device).view(1, 1, 4)
    z = kc[:, 0, :, 0].flatten().float()
    want = torch.softmax(z.double(), 0) @ vc[:, 0].flatten(0, 1).double()
    for splits in (1, 4):
        out = api.sparse_decode(q, kc, vc, bt, cl, sel, torch.full((1, 1), 4, dtype=torch.int32, device=cuda_device), 0.125, splits=splits)
        # 31 equal probabilities: exact in bf16 up to their rounding and the output's
        assert (out[0, 0].double() - want).abs().max() <= 2.0 ** -7 * want.abs().max() + 2.0 ** -8 * vc.float().abs().max()


def test_own_lists_in_any_order(api, cuda_device):
    case = Case(cuda_device, [700, 260], 8, 2)
    rng = np.random.default_rng(2)
    sel = np.full((2, 2, 50), -1, np.int32)
    cnt = np.zeros((2, 2), np.int32)
    for s in range(2):
        for h in range(2):
            n = [44, 3][s] if h else [1, 17][s]
            sel[s, h, :n] = rng.permutation(-(-int(case.lens[s]) // 16))[:n]
            cnt[s, h] = n
    cnt[0, 0] = 0
    out = api.sparse_decode(case.q, case.kc, case.vc, case.bt, case.cl, torch.from_numpy(sel).to(cuda_device),
                            torch.from_numpy(cnt).to(cuda_device), case.scale)
    case.check(out, sel, cnt)
    assert (out[0, :4] == 0).all()
    assert api.device_errors() == 0


def test_entries_outside_the_sequence_are_flagged_and_left_out(api, cuda_device):
    case = Case(cuda_device, [100, 40], 4, 1, D=64, width=12)
    case.tables[1, 1] = 10 ** 6  # outside the pool: read as zeros, as the dense decode does
    bt = torch.from_numpy(case.tables).to(cuda_device)
    sel = torch.tensor([[[2, 7, -1, 100000, 0, 6]], [[0, 3, 2, 11, -5, -1]]], dtype=torch.int32, device=cuda_device)
    cnt = torch.tensor([[6], [500]], dtype=torch.int32, device=cuda_device)  # a count above the list is held to it
    for splits in (1, 8):
        out = api.sparse_decode(case.q, case.kc, case.vc, bt, case.cl, sel, cnt, case.scale, splits=splits)
        assert api.device_errors() == _lib.PA_DEVERR_BAD_BLOCK
        case.check(out, np.array([[[2, 0, 6]], [[0, 2, -1]]], np.int32), np.array([[3], [2]], np.int32))
    cnt[:] = -3
    out = api.sparse_decode(case.q, case.kc, case.vc, bt, case.cl, sel, cnt, case.scale)
    assert (out == 0).all() and api.device_errors() == 0


def test_choice_flags_bad_table_entries_and_contexts(api, cuda_device):
    case = Case(cuda_device, [640, 640], 4, 1, D=64)
    s, e = case.summaries(api)
    case.tables[0, 9], case.tables[0, 12] = -1, case.kc.shape[0]
    bt = torch.from_numpy(case.tables).to(cuda_device)
    sel, _ = api.sparse_select(case.q, s, e, bt, case.cl, 16, 30)
    assert api.device_errors() == _lib.PA_DEVERR_BAD_BLOCK
    want, _ = R.select(f64(case.q), s.cpu().numpy(), e.cpu().numpy(), case.tables, case.lens, 16, 30, 1, 2)
    assert np.array_equal(sel.cpu().numpy(), want)
    lens = torch.tensor([640, 10 ** 6], dtype=torch.int32, device=cuda_device)
    sel, _ = api.sparse_select(case.q, s, e, case.bt, lens, 16, 10)
    assert api.device_errors() == _lib.PA_DEVERR_BAD_CONTEXT
    assert sel[1, 0, -1] == 39
    out = api.sparse_attend(case.q, case.kc, case.vc, s, e, case.bt, lens, 64)
    assert api.device_errors() == _lib.PA_DEVERR_BAD_CONTEXT
    assert out.isfinite().all()


@pytest.mark.parametrize("G,S", [(2, 10), (2, 40), (2, 110), (2, 240), (2, 310), (2, 700), (9, 40), (9, 60), (9, 90), (9, 130),
                                 (9, 190), (9, 300)])
def test_every_number_of_ctas_to_a_row(api, cuda_device, G, S):
    """Row counts for which a row gets 8, 4 and 1 CTAs of eight warps, and 8, 6, 4, 3, 2 and 1 of four."""
    rng = np.random.default_rng(S)
    case = Case(cuda_device, [int(n) for n in rng.integers(0, 330, S)], G, 1, D=64, seed=S, width=260)
    s, e = case.summaries(api)
    top_k = 34 if S < 100 else 16
    sel, cnt, out = case.attend(api, s, e, top_k)
    want_sel, want_cnt = R.select(f64(case.q), s.cpu().numpy(), e.cpu().numpy(), case.tables, case.lens, 16, top_k, 1, 2)
    assert np.array_equal(sel, want_sel) and np.array_equal(cnt, want_cnt)
    case.check(out, sel, cnt)
    assert api.device_errors() == 0


@pytest.mark.parametrize("G,S,width,top_k,B,fp8", [
    (2, 85, 900, 20, 16, False), (2, 85, 900, 50, 16, True), (2, 96, 200, 60, 16, False), (3, 90, 390, 49, 32, True),   # six of four warps
    (2, 140, 900, 20, 16, False), (2, 152, 800, 33, 16, True), (1, 70, 900, 20, 32, False),                             # two of eight
    (9, 190, 1000, 40, 16, False), (9, 190, 200, 40, 16, True), (16, 60, 100, 20, 16, False),                           # groups above 8
    (2, 72, 900, 40, 16, False), (2, 36, 900, 40, 32, False), (2, 85, 900, 10, 16, False), (2, 100, 799, 40, 16, False),
])
def test_clusters_by_length_of_the_tables(api, cuda_device, G, S, width, top_k, B, fp8):
    """Row counts at which the tables' width and the lists' length say how many CTAs a row gets; some rows with as many
    pages as fit, some with few, some with none."""
    rng = np.random.default_rng(S + width)
    lens = [int(n) for n in rng.integers(0, 25 * B, S)]
    lens[1], lens[S // 2], lens[-1], lens[3] = width * B, (width // 2 + 3) * B - 1, width * B - B // 2, 300
    case = Case(cuda_device, lens, G, 1, D=64, B=B, fp8=fp8, seed=S, width=width)
    s, e = case.summaries(api)
    sel, cnt, out = case.attend(api, s, e, top_k)
    want_sel, want_cnt = R.select(f64(case.q), s.cpu().numpy(), e.cpu().numpy(), case.tables, case.lens, B, top_k, 1, 2)
    assert np.array_equal(sel, want_sel) and np.array_equal(cnt, want_cnt)
    case.check(out, sel, cnt)
    assert api.device_errors() == 0


@pytest.mark.parametrize("G,S,width", [(2, 9, 257), (2, 9, 128), (9, 30, 400), (2, 30, 2100), (2, 50, 2000), (2, 70, 1000), (2, 70, 400),
                                       (9, 100, 2000), (2, 140, 2000), (2, 160, 300), (9, 160, 500), (2, 200, 1000), (2, 310, 999),
                                       (9, 310, 5000), (2, 240, 5000)])
def test_choice_alone_by_rows_and_tables(api, cuda_device, G, S, width):
    """Every number of threads and CTAs that the choice alone gives a row, bit for bit."""
    D, NB = 64, 700
    g = torch.Generator().manual_seed(S + width)
    q = torch.randn(S, G, D, generator=g).to(torch.bfloat16)
    s = torch.randint(-127, 128, (NB, 1, 2, D), generator=g).to(torch.int8).sort(dim=2, descending=True).values
    e = torch.randint(-9, -6, (NB, 1), generator=g).to(torch.int8)
    tables = torch.randint(0, NB, (S, width), generator=g).to(torch.int32)
    lens = torch.randint(0, 60 * 16, (S,), generator=g).to(torch.int32)
    lens[::S // 4] = width * 16 - torch.randint(0, 16 * 16, lens[::S // 4].shape, generator=g).to(torch.int32)
    sel, cnt = api.sparse_select(*(t.to(cuda_device) for t in (q, s, e, tables, lens)), 16, 37)
    want_sel, want_cnt = R.select(f64(q), s.numpy(), e.numpy(), tables.numpy(), lens.numpy(), 16, 37, 1, 2)
    assert np.array_equal(sel.cpu().numpy(), want_sel) and np.array_equal(cnt.cpu().numpy(), want_cnt)
    assert api.device_errors() == 0


@pytest.mark.parametrize("S,Hkv", [(125, 5), (70, 9), (128, 5), (128, 9)])
def test_rows_taken_by_length(api, cuda_device, S, Hkv):
    """A few more clusters than places with 128 rows or fewer: the rows are taken longest first, equal ones in their
    order; with many more, in the order given."""
    case = Case(cuda_device, ([700, 16, 700, 0, 33] * 26)[:S], Hkv, Hkv, D=64)
    s, e = case.summaries(api)
    sel, cnt, out = case.attend(api, s, e, 8)
    want_sel, want_cnt = R.select(f64(case.q), s.cpu().numpy(), e.cpu().numpy(), case.tables, case.lens, 16, 8, 1, 2)
    assert np.array_equal(sel, want_sel) and np.array_equal(cnt, want_cnt)
    case.check(out, sel, cnt)


def test_rows_may_share_a_sequence(api, cuda_device):
    """Several query tokens of one sequence, each with its own length."""
    case = Case(cuda_device, [613], 8, 2)
    s, e = case.summaries(api)
    lens = torch.tensor([610, 611, 612, 613], dtype=torch.int32, device=cuda_device)
    q = torch.randn(4, 8, 128, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16).to(cuda_device)
    bt = case.bt.repeat(4, 1)
    many = api.sparse_attend(q, case.kc, case.vc, s, e, bt, lens, 12)
    for i in range(4):
        one = api.sparse_attend(q[i:i + 1], case.kc, case.vc, s, e, case.bt, lens[i:i + 1], 12)
        assert torch.equal(many[i:i + 1], one)


def test_captured_graphs_and_two_streams(api, cuda_device):
    """No state is shared: two captured calls and an eager one, replayed in turn and at once on two streams."""
    cases = [Case(cuda_device, [900, 41], 8, 2, seed=i) for i in range(2)]
    eager, graphs, outs = [], [], []
    for c in cases:
        s, e = c.summaries(api)
        eager.append(api.sparse_attend(c.q, c.kc, c.vc, s, e, c.bt, c.cl, 9))
        out, sel, cnt = torch.zeros_like(c.q), torch.zeros(2, 2, 9, dtype=torch.int32, device=cuda_device), torch.zeros(2, 2, dtype=torch.int32, device=cuda_device)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            api.sparse_attend(c.q, c.kc, c.vc, s, e, c.bt, c.cl, 9, selected=sel, counts=cnt, out=out)
        graphs.append((graph, s, e, sel, cnt))
        outs.append(out)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, (graph, *_) in zip(streams, graphs):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(eager, outs):
        assert torch.equal(a, b)


def test_a_timed_out_wait_is_flagged_and_the_next_call_is_right(api, cuda_device):
    case = Case(cuda_device, [500, 20], 8, 2)
    s, e = case.summaries(api)
    want = api.sparse_attend(case.q, case.kc, case.vc, s, e, case.bt, case.cl, 12)
    lib = _lib.load()
    torch.cuda.synchronize()
    try:
        assert lib.pa_test_set_wait(2_000_000, 1) == 0
        api.sparse_attend(case.q, case.kc, case.vc, s, e, case.bt, case.cl, 12)
        assert api.device_errors() == _lib.PA_DEVERR_TIMEOUT
    finally:
        lib.pa_test_set_wait(0, 0)
    again = api.sparse_attend(case.q, case.kc, case.vc, s, e, case.bt, case.cl, 12)
    assert torch.equal(want, again) and api.device_errors() == 0


def test_a_long_table(api, cuda_device):
    """2^20 tokens in 16-token pages: 65,536 candidates, few of them distinct pages."""
    g = torch.Generator().manual_seed(8)
    NB, D, pages = 2000, 64, 65536
    kc = torch.randn(NB, 1, 16, D, generator=g).to(torch.bfloat16).to(cuda_device)
    vc = torch.randn(NB, 1, 16, D, generator=g).to(torch.bfloat16).to(cuda_device)
    s, e = api.alloc_block_summary(kc)
    api.block_summary(kc, torch.arange(15, NB * 16, 16, dtype=torch.int32, device=cuda_device), s, e)
    tables = torch.randint(0, NB, (1, pages), generator=g).to(torch.int32)
    q = torch.randn(1, 2, D, generator=g).to(torch.bfloat16)
    lens = torch.tensor([pages * 16 - 5], dtype=torch.int32)
    sel, cnt = api.sparse_select(q.to(cuda_device), s, e, tables.to(cuda_device), lens.to(cuda_device), 16, 500)
    want, _ = R.select(f64(q), s.cpu().numpy(), e.cpu().numpy(), tables.numpy(), lens.numpy(), 16, 500, 1, 2)
    assert np.array_equal(sel.cpu().numpy(), want)
    out = api.sparse_decode(q.to(cuda_device), kc, vc, tables.to(cuda_device), lens.to(cuda_device), sel, cnt, 0.125)
    one = np.ones(1)
    ref, bound = R.attend(f64(q), R.values(kc), R.values(vc), tables.numpy(), lens.numpy(), want, cnt.cpu().numpy(), 0.125, one, one)
    assert (np.abs(f64(out) - ref) <= bound).all()


def test_a_cache_past_32_bits(api, cuda_device):
    """Pages whose bytes and elements lie past 2^32, at the end of an 8.6 GB E4M3 cache."""
    NB, Hkv, B, D = 2 ** 18, 16, 16, 128
    assert NB * Hkv * B * D > 2 ** 32
    g = torch.Generator().manual_seed(31)
    kc, vc = (torch.zeros(NB, Hkv, B, D, dtype=torch.uint8, device=cuda_device) for _ in range(2))
    s, e = api.alloc_block_summary(kc)
    n = 10 * B
    blocks = torch.tensor([NB - 1, 5, NB - 3, NB - 2, 9, NB - 200, 0, NB - 77, NB - 4, NB - 5], dtype=torch.int32)
    slots = (blocks[:, None] * B + torch.arange(B)).flatten().to(torch.int32).to(cuda_device)
    q, k, v = (torch.randn(n, h, D, generator=g).to(torch.bfloat16).to(cuda_device) for h in (Hkv, Hkv, Hkv))
    pos = torch.arange(n, dtype=torch.int32, device=cuda_device)
    freq = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).to(cuda_device)
    rq = api.rope_append(q, k, v, pos, freq, slots, kc, vc, kv_scale=1 / 32)
    api.block_summary(kc, slots, s, e)
    used = blocks.long().to(cuda_device)
    small = [t[used].clone() for t in (kc, vc, s, e)]
    # the same tokens in a cache of ten pages
    k2, v2 = torch.zeros_like(small[0]), torch.zeros_like(small[1])
    s2, e2 = api.alloc_block_summary(k2)
    slots2 = torch.arange(n, dtype=torch.int32, device=cuda_device)
    assert torch.equal(rq, api.rope_append(q, k, v, pos, freq, slots2, k2, v2, kv_scale=1 / 32))
    api.block_summary(k2, slots2, s2, e2)
    for big, want in zip(small, (k2, v2, s2, e2)):
        assert torch.equal(big, want)
    assert int((kc[NB - 300:] != 0).any(-1).any(-1).any(-1).sum()) == 7
    lens = torch.tensor([n], dtype=torch.int32, device=cuda_device)
    last = rq[-1:].contiguous()
    far = api.sparse_attend(last, kc, vc, s, e, blocks[None].to(cuda_device), lens, 6, kv_scale=1 / 32)
    near = api.sparse_attend(last, k2, v2, s2, e2, torch.arange(10, dtype=torch.int32, device=cuda_device)[None], lens, 6,
                             kv_scale=1 / 32)
    assert torch.equal(far, near) and far.isfinite().all() and api.device_errors() == 0


# ---- the operators as they are used together ------------------------------------

def _decode_loop(api, device, step_of, steps, S=3, Hq=8, Hkv=2, D=128, B=16, top_k=6, fp8=False):
    """`steps` decode steps of SparseDecodeStep from given prefixes, each against the reference on the device's own cache."""
    g = torch.Generator().manual_seed(21)
    prefix = [150, 14, 0]
    MB = 16
    NB = S * MB
    dtype = torch.uint8 if fp8 else torch.bfloat16
    kc = torch.zeros(NB, Hkv, B, D, dtype=dtype, device=device)
    vc = torch.zeros_like(kc)
    tables = torch.randperm(NB, generator=g).to(torch.int32).view(S, MB).to(device)
    lens = torch.tensor(prefix, dtype=torch.int32, device=device)
    positions = (lens - 1).clone()
    freq = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).to(device)
    kv_scale = 1 / 32 if fp8 else 1.0
    step = api.SparseDecodeStep(kc, vc, tables, lens, positions, freq, Hq, top_k, kv_scale=kv_scale)
    # the prompts' tokens, appended and summarised as chunks
    start = torch.tensor([0, 150, 164, 164], dtype=torch.int32, device=device)
    slots = api.chunk_slot_mapping(tables, lens, start, B)
    k0, v0 = (torch.randn(164, Hkv, D, generator=g).to(torch.bfloat16).to(device) for _ in range(2))
    pos0 = torch.cat([torch.arange(n) for n in prefix]).to(torch.int32).to(device)
    api.rope_append(None, k0, v0, pos0, freq, slots, kc, vc, kv_scale=kv_scale)
    api.block_summary(kc, slots, step.summary, step.exponents)
    q, k, v = (torch.zeros(S, h, D, dtype=torch.bfloat16, device=device) for h in (Hq, Hkv, Hkv))
    run = step_of(step, (q, k, v))
    # whatever a captured run did at its making is undone: the lengths, cache and summaries start here
    ones = np.full(Hkv, kv_scale)
    for _ in range(steps):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g).to(torch.bfloat16))
        lens += 1
        positions += 1
        run()
        torch.cuda.synchronize()
        rq = f64(step.q_rotated)
        assert np.abs(rq - R.rotate(f64(q), positions.cpu().numpy(), freq.cpu().numpy(), None, False)).max() < 2.0 ** -6
        kv = R.values(kc)
        for s in range(S):  # every full block's bounds are those of what the cache holds
            full = int(lens[s]) // B
            want_s, want_e = step.summary.cpu().numpy().copy(), step.exponents.cpu().numpy().copy()
            R.block_summary(kv, [int(b) * B + B - 1 for b in tables[s, :full]], want_s, want_e)
            assert np.array_equal(want_s, step.summary.cpu().numpy()) and np.array_equal(want_e, step.exponents.cpu().numpy())
        sel, cnt = R.select(rq, want_s, want_e, tables.cpu().numpy(), lens.cpu().numpy(), B, top_k, 1, 2)
        assert np.array_equal(step.selected.cpu().numpy(), sel) and np.array_equal(step.counts.cpu().numpy(), cnt)
        ref, bound = R.attend(rq, kv, R.values(vc), tables.cpu().numpy(), lens.cpu().numpy(), sel, cnt, D ** -0.5, ones, ones,
                              probability="fp16" if fp8 else "bf16")
        assert (np.abs(f64(step.out) - ref) <= bound).all()
    assert api.device_errors() == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_loop(api, cuda_device, fp8):
    _decode_loop(api, cuda_device, lambda step, io: (lambda: step(*io)), 20, fp8=fp8)


def test_decode_loop_captured(api, cuda_device):
    def captured(step, io):
        graph = api.StepGraph([step], [io])
        assert graph.launches() == 4
        return graph.replay
    _decode_loop(api, cuda_device, captured, 20)


def test_steps_one_after_the_other_equal_steps_that_wait(api, cuda_device):
    """A chain of the kernels with nothing between them (each is put on the SMs while the one before still runs), the
    dense decode and the plain append among them: bit for bit what the same calls give when each is waited for."""
    g = torch.Generator().manual_seed(41)
    S, Hq, Hkv, D, B, MB, steps = 6, 16, 4, 128, 16, 40, 40
    q, k, v = (torch.randn(steps, S, h, D, generator=g).to(torch.bfloat16).to(cuda_device) for h in (Hq, Hkv, Hkv))
    freq = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).to(cuda_device)
    tables = torch.randperm(S * MB, generator=g).to(torch.int32).view(S, MB).to(cuda_device)
    first = torch.tensor([0, 15, 100, 333, 500, 599], dtype=torch.int32, device=cuda_device)
    start = torch.randn(2, S * MB, Hkv, B, D, generator=g).to(torch.bfloat16).to(cuda_device)
    full = torch.arange(B - 1, S * MB * B, B, dtype=torch.int32, device=cuda_device)

    def chain(after):
        kc, vc = start[0].clone(), start[1].clone()
        lens, pos = first.clone(), first - 1
        step = api.SparseDecodeStep(kc, vc, tables, lens, pos, freq, Hq, 9)
        api.block_summary(kc, full, step.summary, step.exponents)
        got = []
        for i in range(steps):
            lens += 1
            pos += 1
            after()
            got.append(step(q[i], k[i], v[i]).clone())
            after()
            got.append(api.decode(step.q_rotated, kc, vc, tables, lens, partition_size=128))
            after()
            api.cache_append(k[i], v[i], step.slots, kc, vc)  # over the rotated row
            after()
            sel, cnt = api.sparse_select(q[i], step.summary, step.exponents, tables, lens, B, 7)
            after()
            got.append(api.sparse_decode(q[i], kc, vc, tables, lens, sel, cnt))
            after()
            api.rope_append(None, k[i], v[i], pos, freq, step.slots, kc, vc)  # and back
            after()
            api.block_summary(kc, step.slots, step.summary, step.exponents)
            after()
        return got + [kc, vc, step.summary, step.exponents]

    want = chain(torch.cuda.synchronize)
    for _ in range(3):
        got = chain(lambda: None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert api.device_errors() == 0


def test_captured_behind_copies_joins_and_other_kernels(api, cuda_device):
    """In one graph: behind a memory copy, behind a memset, behind two streams that join, and with a branch after."""
    case = Case(cuda_device, [900, 41, 300], 8, 2)
    s, e = case.summaries(api)
    want = api.sparse_attend(case.q, case.kc, case.vc, s, e, case.bt, case.cl, 9)
    other = api.decode(case.q, case.kc, case.vc, case.bt, case.cl, case.scale)
    full = [case.tables[i, j] * 16 + 15 for i, n in enumerate(case.lens) for j in range(n // 16)]
    full = torch.tensor(full, dtype=torch.int32, device=cuda_device)
    q, s2, e2 = torch.zeros_like(case.q), torch.zeros_like(s), torch.zeros_like(e)
    sel, cnt = torch.zeros(3, 2, 9, dtype=torch.int32, device=cuda_device), torch.zeros(3, 2, dtype=torch.int32, device=cuda_device)
    outs = [torch.zeros_like(case.q) for _ in range(3)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        q.zero_()
        q.copy_(case.q)                                    # a copy, then a kernel of ours
        api.sparse_attend(q, case.kc, case.vc, s, e, case.bt, case.cl, 9, selected=sel, counts=cnt, out=outs[0])
        side.wait_stream(main)
        s2.zero_()
        with torch.cuda.stream(side):
            api.block_summary(case.kc, full, s2, e2)       # on its own branch, after the attention
            api.decode(q, case.kc, case.vc, case.bt, case.cl, case.scale, out=outs[2])
        main.wait_stream(side)                             # the join, then a kernel of ours
        api.block_summary(case.kc, full, s2, e2)
        api.sparse_attend(q, case.kc, case.vc, s2, e2, case.bt, case.cl, 9, selected=sel, counts=cnt, out=outs[1])
    for _ in range(5):
        for t in (q, s2, e2, *outs):
            t.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want) and torch.equal(outs[2], other)
        done = full.long() // 16  # the others' exponents are left as they were: filled above
        assert torch.equal(s2, s) and torch.equal(e2[done], e[done])
    assert api.device_errors() == 0


def test_tensors_made_for_another_stream_belong_to_it(api, cuda_device):
    """What a call on a busy stream allocates is not memory that the current stream hands out, or has in use."""
    case = Case(cuda_device, [900, 41, 300], 8, 2)
    s, e = case.summaries(api)
    T, Hq, D = case.q.shape
    want_sel, want_cnt = api.sparse_select(case.q, s, e, case.bt, case.cl, 16, 9)
    want = api.sparse_attend(case.q, case.kc, case.vc, s, e, case.bt, case.cl, 9)
    none = torch.full((T,), -1, dtype=torch.int32, device=cuda_device)
    zero = none + 1  # the inputs outlive the calls: they are the caller's
    kv = case.q[:, :2].contiguous()
    freq = torch.ones(D // 2, dtype=torch.float64, device=cuda_device)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    got = api.sparse_attend(case.q, case.kc, case.vc, s, e, case.bt, case.cl, 9, stream=side)
    sel, cnt = api.sparse_select(case.q, s, e, case.bt, case.cl, 16, 9, stream=side)
    out = api.sparse_decode(case.q, case.kc, case.vc, case.bt, case.cl, sel, cnt, stream=side)
    rot = api.rope_append(case.q, kv, kv, zero, freq, none, case.kc, case.vc, stream=side)
    # the sizes of what those calls made, now on the current stream
    mine = [torch.full(t.shape, 5, dtype=t.dtype, device=cuda_device) for _ in range(4) for t in (sel, cnt, got)]
    torch.cuda.synchronize()
    assert all((t == 5).all() for t in mine)
    assert torch.equal(got, want) and torch.equal(sel, want_sel) and torch.equal(cnt, want_cnt)
    case.check(out, want_sel.cpu().numpy(), want_cnt.cpu().numpy())
    assert torch.equal(rot, case.q)  # position 0 turns nothing
