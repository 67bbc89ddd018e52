"""Shared-prefix decode as it is called by a server: chains of calls, tables wider than what they hold, bounds that say
little, groups that are none."""
import pytest
import torch

from paged_kv_cache_193_gb300 import _lib
from rows_cases import Shared, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api(cuda_device):
    from paged_kv_cache_193_gb300 import api as a
    a._lib_handle()
    return a


@pytest.fixture(autouse=True)
def every_prefix_is_shared():
    """Small batches would be attended to sequence by sequence."""
    lib = _lib.load()
    assert lib.pa_test_set_share(0, -1) == 0
    yield
    assert lib.pa_test_set_share(-1, -1) == 0


@pytest.mark.parametrize("apart", [0, 1])
@pytest.mark.parametrize("S,fp8", [(2, False), (9, True), (128, False)])
def test_longest_first_in_calls_that_feed_each_other(api, cuda_device, S, fp8, apart):
    """One group of 2 to 128 sequences with 16 pages of their own and more: CTAs rank the lengths where the first pages land
    next.  Each call's output is the next one's query; bit for bit what the same calls give when each is waited for, and
    the first of them the definition."""
    _lib.load().pa_test_set_share(0, apart)
    case = Shared(cuda_device, [(12, [(53 * i) % 290 for i in range(S - 1)] + [16 * 18])], 8, 2, fp8=fp8)
    ws = api.alloc_shared_prefix_workspace(case.q, case.pool.kd, case.gs, case.most)

    def chain(after):
        x, got = case.q.clone(), []
        for _ in range(40):
            y = case.call(api, q=x, workspace=ws)
            after()
            x = (y * 3).contiguous()
            after()
            got.append(y)
        return got

    want = chain(torch.cuda.synchronize)
    within(want[0], case.expected())
    for _ in range(5):
        got = chain(lambda: None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert api.device_errors() == 0


@pytest.mark.parametrize("share", [0, 10 ** 7, -1])
@pytest.mark.parametrize("groups,Hkv", [([(40, [-300, -17, -639]), (9, [5, 100, 0]), (30, [-1])], 2), ([(200, [9, -100, 30, None])], 8)])
def test_a_workspace_for_the_bound_or_for_the_width(api, cuda_device, groups, Hkv, share):
    """A bound past the tables' width counts as the width, so a workspace for either does, and none where the width says
    that nothing is shared."""
    lib = _lib.load()
    lib.pa_test_set_share(share, -1)
    case = Shared(cuda_device, groups, 8, Hkv)
    S, Hq, D = case.q.shape
    width, want = case.bt.shape[1], case.expected()
    taken = set()
    for most in (width, width + 1, 3 * width, 4096, 1 << 20):
        shared = lib.pa_shared_prefix_launches(S, len(case.pb), Hq, Hkv, D, case.pool.B, width, most, 0) > 1
        for sized in (most, width):
            ws = api.alloc_shared_prefix_workspace(case.q, case.pool.kd, case.gs, sized)
            assert ws is not None or not shared
            if ws is not None:
                ws.fill_(0xff)
            within(case.call(api, max_prefix_blocks=most, workspace=ws), want, f"{most} {sized}")
        taken.add(shared)
    assert len(taken) == 1 and api.device_errors() == 0


@pytest.mark.parametrize("kw", [dict(groups=[(9, [i % 113 for i in range(86)])], Hq=6, Hkv=6),
                                dict(groups=[(70, [i % 60 for i in range(175)])], Hq=9, Hkv=3, D=64, B=32),
                                dict(groups=[(40, [i % 101 for i in range(108)] + [-1, None])], Hq=20, Hkv=5, fp8=True, per_head=True),
                                dict(groups=[(12, [(211 * i) % 1100 for i in range(9)] + [None, -3])], Hq=8, Hkv=2)])
def test_both_ways_of_joining_are_the_ways_meant(api, cuda_device, kw):
    """Two and three kernels by the library's own answer, for lists so short that a warp takes a head too; each against the
    definition, and twice the same bits with a workspace of NaN."""
    lib = _lib.load()
    case = Shared(cuda_device, **kw)
    S, Hq, D = case.q.shape
    ws, want = api.alloc_shared_prefix_workspace(case.q, case.pool.kd, case.gs, case.most), case.expected()
    for apart in (0, 1):
        lib.pa_test_set_share(0, apart)
        assert lib.pa_shared_prefix_launches(S, len(case.pb), Hq, case.pool.Hkv, D, case.pool.B, case.bt.shape[1], case.most,
                                             int(case.pool.fp8)) == 2 + apart
        outs = []
        for _ in range(2):
            ws.fill_(0xff)
            outs.append(case.call(api, workspace=ws))
            within(outs[-1], want, f"apart: {apart}")
        assert torch.equal(*outs)
    assert api.device_errors() == 0


@pytest.mark.parametrize("apart", [0, 1])
@pytest.mark.parametrize("fp8", [False, True])
def test_groups_that_are_no_ranges_are_reported(api, cuda_device, fp8, apart):
    """Whichever group it is, among few and among more than a CTA has threads; and not those that are, empty ones, sequences
    of none and prefixes of none among them."""
    _lib.load().pa_test_set_share(0, apart)
    case = Shared(cuda_device, [(4, [8, 9]), (0, []), (3, [1, 2])], 4, 2, alone=[20], fp8=fp8)
    want = case.expected()
    within(case.call(api), want)
    assert api.device_errors() == 0
    for start in ([-1, 2, 2, 4], [0, 2, 2, 6], [0, 2, 1, 4], [3, 1, 0, 0], [0, 2, 2, -4], [2 ** 31 - 1, 0, -2 ** 31, 1], [6, 6, 6, 6]):
        case.gs.copy_(torch.tensor(start, dtype=torch.int32))
        case.call(api)
        assert api.device_errors() == _lib.PA_DEVERR_BAD_CONTEXT, start
    case.gs.copy_(torch.tensor([0, 2, 2, 4], dtype=torch.int32))
    case.pb[1:] = -7
    within(case.call(api), want)
    assert api.device_errors() == 0
    many = Shared(cuda_device, [(1 + i % 2, [i % 3]) for i in range(1500)], 2, 2, D=64, fp8=fp8)
    within(many.call(api), many.expected())
    assert api.device_errors() == 0
    for g in (1, 31, 700, 1499):
        was = int(many.gs[g])
        many.gs[g] = was + 2  # behind the start of the next
        many.call(api)
        assert api.device_errors() == _lib.PA_DEVERR_BAD_CONTEXT, g
        many.gs[g] = was
    within(many.call(api), many.expected())
    assert api.device_errors() == 0


def test_groups_are_not_read_where_nothing_is_shared(api, cuda_device):
    _lib.load().pa_test_set_share(1 << 60, -1)
    case = Shared(cuda_device, [(4, [8, 9]), (3, [1, 2])], 4, 2)
    case.gs.copy_(torch.tensor([3, 1, 0], dtype=torch.int32))
    within(case.call(api), case.expected())
    assert api.device_errors() == 0


@pytest.mark.parametrize("kw", [dict(groups=[(9, [(53 * i) % 400 for i in range(257)])], Hq=8, Hkv=8, D=64, fp8=True),       # a warp to a head
                                dict(groups=[(9, [(53 * i) % 330 for i in range(100)] + [None, -7])], Hq=16, Hkv=8, extra=40),  # a CTA
                                dict(groups=[(4, [(7 * i) % 90 for i in range(40)]), (20, [3, 700, -100])], Hq=8, Hkv=2, extra=3000),
                                dict(groups=[(140, [(i * 5) % 60 for i in range(69)] + [-1])], Hq=8, Hkv=8, alone=[1500, 3]),
                                dict(groups=[(30, [(i * 5) % 60 for i in range(69)] + [-1])], Hq=8, Hkv=8, alone=[300, 0])])
def test_without_a_bound_and_in_wide_tables(api, cuda_device, kw):
    """The bound is the tables' width, or they have room for far more than they hold; sequences without their prefix, and
    of no group, among others with little of their own."""
    lib = _lib.load()
    case = Shared(cuda_device, **kw)
    want = case.expected()
    for apart in (-1, 0, 1):
        lib.pa_test_set_share(0, apart)
        for most in (None, case.most):
            within(case.call(api, max_prefix_blocks=most), want, f"{apart} {most}")
    assert api.device_errors() == 0


def _time(call, n=5):
    call()
    best = float("inf")
    for _ in range(4):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        for _ in range(n):
            call()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) / n)
    return best


@pytest.mark.parametrize("S,P,own,Hq,extra", [(64, 64, 8000, 32, 0), (64, 2048, 2048, 64, 0), (64, 2048, 2048, 64, 6000), (16, 512, 1000, 32, 7000)])
def test_what_no_bound_and_wide_tables_cost(api, cuda_device, S, P, own, Hq, extra):
    """Neither sends a batch the long way round: within twice the time of the exact bound over exact tables (two and a half
    to five times, when a bound was taken for what is there)."""
    _lib.load().pa_test_set_share(-1, -1)
    Hkv, D, B = 8, 128, 16
    g = torch.Generator(device=cuda_device).manual_seed(1)
    mine = -(-own // B)
    NB = P + S * mine
    kv = torch.randn(2, NB, Hkv, B, D, generator=g, device=cuda_device, dtype=torch.bfloat16)
    q = torch.randn(S, Hq, D, generator=g, device=cuda_device).to(torch.bfloat16)
    exact = torch.cat([torch.arange(P, device=cuda_device).expand(S, P), P + torch.arange(S * mine, device=cuda_device).view(S, mine)], 1).to(torch.int32)
    wide = torch.cat([exact, torch.full((S, extra), -1, dtype=torch.int32, device=cuda_device)], 1).contiguous()
    lens = (P * B + torch.randint(1, own + 1, (S,), generator=g, device=cuda_device)).to(torch.int32)
    gs = torch.tensor([0, S], dtype=torch.int32, device=cuda_device)
    pb = torch.tensor([P], dtype=torch.int32, device=cuda_device)
    out = torch.empty_like(q)

    def call(tables, bound):
        ws = api.alloc_shared_prefix_workspace(q, kv[0], gs, tables.shape[1] if bound is None else bound)
        return lambda: api.shared_prefix_decode(q, kv[0], kv[1], tables, lens, gs, pb, bound, workspace=ws, out=out)

    least = _time(call(exact, P))
    assert _time(call(wide, P if extra else None)) < 2 * least
    assert api.device_errors() == 0


@pytest.mark.parametrize("apart", [0, 1])
@pytest.mark.parametrize("norm,fp8", [(False, False), (True, True)])
def test_every_step_against_the_definition(api, cuda_device, norm, fp8, apart):
    """Twenty tokens through SharedPrefixDecodeStep, over the ends of pages: the attention of each, eager and from a graph,
    against the definition over the cache that the steps wrote.  (A cache only grows, so the last one serves them all.)"""
    _lib.load().pa_test_set_share(0, apart)
    B, D, Hq, Hkv, steps = 16, 128, 8, 2, 20
    case = Shared(cuda_device, [(6, [1, 5, 14, 16]), (3, [2, 2])], Hq, Hkv, fp8=fp8, extra=2)
    S, dev = case.q.shape[0], cuda_device
    g = torch.Generator().manual_seed(6)
    more = torch.zeros(40, Hkv, B, D, dtype=case.pool.kd.dtype, device=dev)
    kc, vc = torch.cat([case.pool.kd, more]), torch.cat([case.pool.vd, more])
    fresh = iter(range(case.pool.kd.shape[0], kc.shape[0]))
    bt = case.bt.clone()
    for s in range(S):  # blocks for what is to come
        for j in range(-(-case.lens[s] // B), bt.shape[1]):
            if j * B < case.lens[s] + steps:
                bt[s, j] = next(fresh)
    freq = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).to(dev)
    w = (1 + 0.2 * torch.randn(2, D, generator=g)).to(torch.bfloat16).to(dev)
    extra = dict(q_weight=w[0], k_weight=w[1], eps=1e-5) if norm else {}
    new = [[torch.randn(S, h, D, generator=g).to(torch.bfloat16).to(dev) for h in (Hq, Hkv, Hkv)] for _ in range(steps)]

    def run(captured):
        k, v, lens = kc.clone(), vc.clone(), case.cl.clone()
        pos, buf, got = lens.clone(), [x.clone() for x in new[0]], []
        lens += 1
        step = api.SharedPrefixDecodeStep(k, v, bt, lens, pos, freq, Hq, case.gs, case.pb, case.most, kv_scale=1 / 16, **extra)
        assert step.launches() == 4 + apart
        graph = api.StepGraph([step], [buf]) if captured else None
        for x in new:
            for a, b in zip(buf, x):
                a.copy_(b)
            if captured:
                graph.replay()
            else:
                step(*buf)
            got.append((step.out.clone(), step.q_rotated.clone(), lens.tolist()))
            lens += 1
            pos += 1
        torch.cuda.synchronize()
        assert api.device_errors() == 0
        return k, v, got

    case.tables, case.scale = bt.cpu(), D ** -0.5
    for captured in (False, True):
        k, v, got = run(captured)
        case.pool.k, case.pool.v = k.cpu(), v.cpu()
        for i, (out, q, lens) in enumerate(got):
            case.q, case.lens = q, lens
            within(out, case.expected(), f"captured {captured}, step {i}")


@pytest.mark.parametrize("apart", [0, 1])
def test_groups_that_change_between_replays(api, cuda_device, apart):
    """One graph for all ways to group a batch: in each replay other groups, prefixes and lengths, an empty group, one of
    all sequences and sequences of none among them."""
    _lib.load().pa_test_set_share(0, apart)
    case = Shared(cuda_device, [(20, [(17 * i) % 150 for i in range(37)])], 8, 2)
    S, G, most = len(case.lens), 4, 20
    out = torch.empty_like(case.q)
    gs, pb = torch.zeros(G + 1, dtype=torch.int32, device=cuda_device), torch.zeros(G, dtype=torch.int32, device=cuda_device)
    ws = api.alloc_shared_prefix_workspace(case.q, case.pool.kd, gs, most)
    case.gs, case.pb = gs, pb

    def call():
        case.call(api, max_prefix_blocks=most, workspace=ws, out=out)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    full = list(case.lens)
    for start, pages in (([0, 0, 0, 0, 0], [20] * 4), ([0, 37, 37, 37, 37], [20, 1, 1, 1]), ([0, 1, 2, 36, 37], [3, 20, 19, 7]),
                         ([5, 5, 20, 20, 30], [9, 0, 8, 20]), ([0, 9, 18, 27, 37], [20, 0, 13, 40])):
        gs.copy_(torch.tensor(start, dtype=torch.int32))
        pb.copy_(torch.tensor(pages, dtype=torch.int32))
        for cut in (0, 200):  # some shorter than their prefix
            case.lens = [max(0, n - cut * (i % 3)) for i, n in enumerate(full)]
            case.cl.copy_(torch.tensor(case.lens, dtype=torch.int32))
            ws.fill_(0xff)
            out.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            within(out, case.expected(), f"{start} {pages} {cut}")
    assert api.device_errors() == 0
