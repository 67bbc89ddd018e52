"""Shared-prefix decode against its definition, the softmax over each sequence's whole context, in 64 bits."""
import numpy as np
import pytest
import torch

from gpu_helpers import Guarded
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
    """Small batches would be attended to sequence by sequence; the tests of that restore it."""
    lib = _lib.load()
    assert lib.pa_test_set_share(0, -1) == 0
    yield
    assert lib.pa_test_set_share(-1, -1) == 0


CASES = [
    dict(groups=[(1, [1])], Hq=1, Hkv=1, D=64),
    dict(groups=[(1, [0, 1])], Hq=8, Hkv=2),
    dict(groups=[(4, [5, 16, 0, 33])], Hq=8, Hkv=2),
    dict(groups=[(5, [5, 17, 40])], Hq=6, Hkv=2, D=64, B=32),
    dict(groups=[(63, [1, 2, 90, 100])], Hq=32, Hkv=8),
    dict(groups=[(20, [7] * 33)], Hq=4, Hkv=1),                     # two tiles, the second of one sequence
    dict(groups=[(9, [3] * 65)], Hq=8, Hkv=2),                      # three tiles, two pairs
    dict(groups=[(9, list(range(40)))], Hq=7, Hkv=1, D=64),         # 18 sequences of 7 heads to a tile
    dict(groups=[(11, [4] * 9)], Hq=16, Hkv=1, B=32),
    dict(groups=[(70, [30, 31, 500])], Hq=10, Hkv=2, fp8=True),
    dict(groups=[(33, [0, 1, 30, 31, 200])], Hq=16, Hkv=2, D=64, B=32, fp8=True, per_head=True),
    dict(groups=[(13, [9] * 21)], Hq=12, Hkv=2, D=64, fp8=True),
    dict(groups=[(17, [9] * 21)], Hq=24, Hkv=2, B=32, fp8=True, per_head=True),
    dict(groups=[(0, [3, 40]), (3, [1]), (30, [0, 9, 70]), (7, [5] * 11)], Hq=8, Hkv=4),
    dict(groups=[(6, [5, -1, 3, -96, None, -50]), (2, [-1, -2]), (0, [None, None])], Hq=8, Hkv=2),
    dict(groups=[(6, [5, -1, 3, -90, None, -50]), (2, [-32, 1])], Hq=8, Hkv=2, fp8=True),
    dict(groups=[(4, [8, 9]), (5, [1, 2, 3])], alone=[1, 100, 0, 17], Hq=8, Hkv=2, D=64),
    dict(groups=[(150, [900, 3])], Hq=8, Hkv=2),
    dict(groups=[(2 + i % 5, [i % 7]) for i in range(70)], Hq=2, Hkv=2, D=64),  # more groups than lanes
    dict(groups=[(8, [20, 30])], Hq=8, Hkv=2, extra=200),           # tables wider than the sequences
    # a warp to a KV head: many rows and short lists
    dict(groups=[(9, [i % 113 for i in range(86)])], Hq=6, Hkv=6),
    dict(groups=[(9, [i % 60 for i in range(175)])], Hq=9, Hkv=3, D=64, B=32),   # and a warp without one
    dict(groups=[(5, [i % 120 for i in range(130)])], Hq=64, Hkv=4),
    dict(groups=[(40, [i % 101 for i in range(110)])], Hq=20, Hkv=5, fp8=True, per_head=True),
    dict(groups=[(9, [i % 90 for i in range(260)] + [-1, None, -100])], Hq=2, Hkv=2, D=64, fp8=True),
    # the same beside the prefix, of more than eight pages
    dict(groups=[(9, [(7 * i) % 190 for i in range(226)] + [-1, None, -100])], Hq=7, Hkv=7, D=64),
    dict(groups=[(4, [(7 * i) % 120 for i in range(150)]), (0, [9]), (3, [(5 * i) % 160 for i in range(120)])], Hq=24, Hkv=6),
    dict(groups=[(30, [(11 * i) % 400 for i in range(200)])], Hq=16, Hkv=8, fp8=True, per_head=True),
    # by eight warps: one CTA to a row, two, four
    dict(groups=[(12, [(29 * i) % 380 for i in range(31)])], Hq=16, Hkv=4),
    dict(groups=[(5, [(29 * i) % 300 for i in range(40)]), (9, [3, 70, 200, None, -5])], Hq=8, Hkv=4, D=64, B=32, fp8=True),
    dict(groups=[(12, [1700, 20, 900, 0, 1])], Hq=8, Hkv=2, D=64),
    dict(groups=[(12, [3500, 40, -7])], Hq=16, Hkv=2),
    # longest first, and several CTAs to a row
    dict(groups=[(12, [(37 * i) % 400 for i in range(30)])], Hq=8, Hkv=2),
    dict(groups=[(12, [(211 * i) % 1100 for i in range(9)] + [None, -3])], Hq=8, Hkv=2),
    dict(groups=[(12, [3, 2500, 1, 1000])], Hq=4, Hkv=1, fp8=True),
]


@pytest.mark.parametrize("kw", CASES, ids=[f"{i}" for i in range(len(CASES))])
def test_matches_the_definition(api, cuda_device, kw):
    case = Shared(cuda_device, **kw)
    S, Hq, D = case.q.shape
    n = api.shared_prefix_workspace_size(S, len(case.pb), Hq, case.pool.Hkv, D, case.pool.B, case.most, int(case.pool.fp8))
    ws = Guarded((n,), torch.uint8, cuda_device)
    out = Guarded(case.q.shape, torch.bfloat16, cuda_device, fill=float("nan"))
    k0, v0, q0 = case.pool.kd.clone(), case.pool.vd.clone(), case.q.clone()
    got = case.call(api, workspace=ws.tensor if n else None, out=out.tensor)
    torch.cuda.synchronize()
    assert got.data_ptr() == out.tensor.data_ptr() and api.device_errors() == 0
    want = case.expected()
    within(got, want)
    for s, length in enumerate(case.lens):
        assert length or (got[s] == 0).all()
    ws.check("workspace")
    out.check("out")
    for a, b in ((case.pool.kd, k0), (case.pool.vd, v0), (case.q, q0)):  # NaN stays what it is: compare bits
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    # again, in place, and without a bound on the prefix
    again = case.call(api)
    assert torch.equal(again, got)
    q = case.q.clone()
    assert torch.equal(case.call(api, q=q, out=q), got)
    within(case.call(api, max_prefix_blocks=None), want, "no bound")
    within(case.call(api, max_prefix_blocks=min(3, case.bt.shape[1])), want, "a bound below the prefix")
    within(case.call(api, max_prefix_blocks=0), want, "nothing shared")
    for apart in (0, 1):
        _lib.load().pa_test_set_share(0, apart)
        ws.tensor.fill_(0xff)  # NaN wherever nothing is written
        within(case.call(api, workspace=ws.tensor if n else None, out=out.tensor), want, f"joined apart: {apart}")
        ws.check("workspace")
        out.check("out")
        within(case.call(api, max_prefix_blocks=None), want, f"joined apart, no bound: {apart}")
    _lib.load().pa_test_set_share(1 << 60, -1)
    assert api.alloc_shared_prefix_workspace(case.q, case.pool.kd, case.gs, case.most) is None
    within(case.call(api), want, "too little to share")


def test_no_groups_and_no_sequences(api, cuda_device):
    case = Shared(cuda_device, [(4, [8, 9])], 8, 2)
    none = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    args = (case.pool.kd, case.pool.vd, case.bt, case.cl, none, none[:0], 4, case.scale)
    within(api.shared_prefix_decode(case.q, *args), case.expected())
    e = case.q[:0]
    assert api.shared_prefix_decode(e, case.pool.kd, case.pool.vd, case.bt[:0], case.cl[:0], none, none[:0], 4).shape == e.shape


@pytest.mark.parametrize("fp8", [False, True])
def test_large_scores_and_odd_values(api, cuda_device, fp8):
    """Scores in the thousands, and a reference that has to move late; then an infinity in one sequence's own values, which
    stays in its outputs."""
    case = Shared(cuda_device, [(40, [9, 50, 300])], 8, 2, fp8=fp8, spread=30.0 if not fp8 else 20.0)
    want = case.expected()
    within(case.call(api), want)
    b = int(case.tables[1, 40])
    case.pool.vd[b, 0, 3, 5] = 0x7f if fp8 else float("inf")
    got = case.call(api).float().cpu()
    assert not torch.isfinite(got[1, :4, 5]).any()
    keep = torch.ones_like(got, dtype=torch.bool)
    keep[1, :4, 5] = False
    ref, bound = want
    off = (got.numpy() - ref)
    assert (np.abs(off) <= bound)[keep.numpy()].all()


def test_a_nan_in_the_prefix_reaches_all_that_share_it(api, cuda_device):
    case = Shared(cuda_device, [(4, [8, 9, -20])], 4, 2, alone=[33])
    b = int(case.tables[0, 3])  # the last of the prefix; the third sequence ends in the page before
    case.pool.vd[b, 1, 2, 7] = float("nan")
    got = case.call(api)
    nan = torch.isnan(got)
    assert nan[0, 2:, 7].all() and nan[1, 2:, 7].all() and int(nan.sum()) == 4


def test_bad_blocks_are_reported(api, cuda_device):
    case = Shared(cuda_device, [(8, [8, 9])], 4, 2, alone=[20])
    within(case.call(api), case.expected())
    case.bt[0, 2] = 10 ** 6
    case.call(api)
    assert api.device_errors() == _lib.PA_DEVERR_BAD_BLOCK
    case.bt[0, 2] = -5
    got = case.call(api)
    assert api.device_errors() == _lib.PA_DEVERR_BAD_BLOCK and torch.isfinite(got).all()
    case.bt.copy_(case.tables)
    case.cl[2] = 10 ** 6  # longer than its table: clamped, and what lies there is NaN
    case.call(api)
    assert api.device_errors() & _lib.PA_DEVERR_BAD_CONTEXT


def test_groups_that_are_no_ranges_stay_in_bounds(api, cuda_device):
    case = Shared(cuda_device, [(4, [8, 9]), (3, [1, 2])], 4, 2)
    out = Guarded(case.q.shape, torch.bfloat16, cuda_device, fill=0.0)
    for start in ([-5, 2, 4], [0, 2, 100], [3, 1, 0], [2 ** 31 - 1, 0, -2 ** 31]):
        case.gs.copy_(torch.tensor(start, dtype=torch.int32))
        case.call(api, out=out.tensor)
        torch.cuda.synchronize()
        out.check(str(start))
    case.gs.copy_(torch.tensor([0, 2, 4], dtype=torch.int32))
    case.pb.copy_(torch.tensor([-3, 2 ** 31 - 1], dtype=torch.int32))  # none; as much as the bound allows
    case.call(api, max_prefix_blocks=3)
    api.device_errors()


@pytest.mark.parametrize("apart", [0, 1])
def test_captured_and_replayed(api, cuda_device, apart):
    """Two graphs of one workspace, replayed in turn on one stream, with lengths and queries that change."""
    _lib.load().pa_test_set_share(0, apart)
    case = Shared(cuda_device, [(30, [40, 9, 3, 70]), (5, [9, 9])], 8, 2)
    want = case.expected()
    ws = api.alloc_shared_prefix_workspace(case.q, case.pool.kd, case.gs, case.most)
    assert ws is not None
    outs = [torch.empty_like(case.q) for _ in range(2)]
    case.call(api, workspace=ws, out=outs[0])
    torch.cuda.synchronize()
    graphs = []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            case.call(api, workspace=ws, out=o)
        graphs.append(g)
    q0, lens = case.q.clone(), case.cl.clone()
    for i in range(6):
        for o in outs:
            o.fill_(float("nan"))
        case.q.copy_(q0 if i % 2 == 0 else -q0)
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1])
        if i % 2 == 0:
            within(outs[0], want)
    case.q.copy_(q0)
    case.cl[1] = 30 * 16 - 1  # now shorter than its prefix
    case.lens[1] = 30 * 16 - 1
    graphs[1].replay()
    torch.cuda.synchronize()
    within(outs[1], case.expected())
    assert not torch.equal(case.cl, lens) and api.device_errors() == 0


def test_on_another_stream_behind_its_work(api, cuda_device):
    case = Shared(cuda_device, [(60, [40, 9, 3, 70])], 8, 2)
    want = case.expected()
    side = torch.cuda.Stream()
    q = torch.zeros_like(case.q)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
        q.copy_(case.q)
    for _ in range(20):
        with torch.cuda.stream(side):
            q.zero_()
            q.copy_(case.q)
        out = case.call(api, q=q, stream=side)
    side.synchronize()
    within(out, want)


@pytest.mark.parametrize("apart", [0, 1])
@pytest.mark.parametrize("groups", [[(50, [40, 9, 3, 70, 300]), (9, [5, 100])], [(9, [i % 113 for i in range(264)])]])
def test_back_to_back_calls_that_feed_each_other(api, cuda_device, groups, apart):
    """Each call's output is the next one's query, in one workspace: bit for bit what the same calls give when each is
    waited for."""
    _lib.load().pa_test_set_share(0, apart)
    case = Shared(cuda_device, groups, 8, 2)
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
    for _ in range(3):
        got = chain(lambda: None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("apart", [0, 1])
def test_a_wait_that_runs_out(api, cuda_device, apart):
    """The kernels give up, say so and end; the next call is right."""
    lib = _lib.load()
    lib.pa_test_set_share(0, apart)
    for fp8 in (False, True):
        case = Shared(cuda_device, [(30, [40, 9])], 8, 2, fp8=fp8)
        assert lib.pa_test_set_wait(1_000_000, 1) == 0
        try:
            case.call(api)
            torch.cuda.synchronize()
        finally:
            assert lib.pa_test_set_wait(0, 0) == 0
        assert api.device_errors() & _lib.PA_DEVERR_TIMEOUT
        within(case.call(api), case.expected())
        assert api.device_errors() == 0


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_the_step_eager_and_captured(api, cuda_device, norm, fp8):
    """Twelve tokens through SharedPrefixDecodeStep: the attention of each against the definition over the cache that the
    step itself wrote, and the same bits from a graph."""
    B, D, Hq, Hkv = 16, 128, 8, 2
    case = Shared(cuda_device, [(6, [1, 5, 14, 16]), (3, [2, 2])], Hq, Hkv, fp8=fp8, extra=2)
    S, dev = case.q.shape[0], cuda_device
    g = torch.Generator().manual_seed(5)
    spare = iter(case.pool.free)
    more = torch.zeros(40, Hkv, B, D, dtype=case.pool.kd.dtype, device=dev)
    kc, vc = torch.cat([case.pool.kd, more]), torch.cat([case.pool.vd, more])
    fresh = iter(range(case.pool.kd.shape[0], kc.shape[0]))
    del spare
    bt, lens = case.bt.clone(), case.cl.clone()
    for s in range(S):  # blocks for what is to come
        for j in range(-(-case.lens[s] // B), bt.shape[1]):
            if j * B < case.lens[s] + 13:
                bt[s, j] = next(fresh)
    pos = lens.clone()
    freq = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).to(dev)
    w = (1 + 0.2 * torch.randn(2, D, generator=g)).to(torch.bfloat16).to(dev)
    extra = dict(q_weight=w[0], k_weight=w[1], eps=1e-5) if norm else {}
    new = [[torch.randn(S, h, D, generator=g).to(torch.bfloat16).to(dev) for h in (Hq, Hkv, Hkv)] for _ in range(12)]

    def make(kc, vc, lens, pos):
        return api.SharedPrefixDecodeStep(kc, vc, bt, lens, pos, freq, Hq, case.gs, case.pb, case.most, kv_scale=1 / 16, **extra)

    k1, v1, l1, p1 = kc.clone(), vc.clone(), lens.clone(), pos.clone()
    step, outs = make(k1, v1, l1, p1), []
    for x in new:
        l1 += 1
        out = step(*x)
        outs.append(out.clone())
        p1 += 1
    torch.cuda.synchronize()
    assert api.device_errors() == 0 and step.launches() == 4
    case.pool.k, case.pool.v = k1.cpu(), v1.cpu()
    case.tables, case.scale = bt.cpu(), D ** -0.5
    case.q, case.lens = step.q_rotated, l1.tolist()
    within(outs[-1], case.expected())
    # the same from a graph
    k2, v2, l2, p2 = kc.clone(), vc.clone(), lens.clone(), pos.clone()
    l2 += 1
    buf = [x.clone() for x in new[0]]
    graph = api.StepGraph([make(k2, v2, l2, p2)], [buf])
    for i, x in enumerate(new):
        for a, b in zip(buf, x):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(graph.steps[0].out, outs[i])
        l2 += 1
        p2 += 1
    assert torch.equal(k2.view(torch.uint8), k1.view(torch.uint8))


@pytest.mark.parametrize("apart", [0, 1])
def test_a_bound_past_the_tables_width(api, cuda_device, apart):
    """Prefixes that no sequence holds to their end: the tables are narrower than the longest one."""
    _lib.load().pa_test_set_share(0, apart)
    case = Shared(cuda_device, [(40, [-300, -17, -639]), (9, [5, 100, 0]), (30, [-1])], 8, 2)
    assert case.bt.shape[1] < case.most
    for most in (case.most, 1000, 100000):
        ws = api.alloc_shared_prefix_workspace(case.q, case.pool.kd, case.gs, most)
        within(case.call(api, max_prefix_blocks=most, workspace=ws), case.expected())
    case.pb.fill_(2 ** 31 - 1)  # no sequence has so much: each by itself
    within(case.call(api, max_prefix_blocks=1000), case.expected())
    assert api.device_errors() == 0


def _launches(lib, *sizes):
    return lib.pa_shared_prefix_launches(*sizes)


def test_a_large_batch_by_its_sizes_alone(api, cuda_device):
    """As the call's own rules launch it: few sequences of a short prefix by themselves, more of them joined by the rest's
    kernel, long ones joined apart; sampled rows against the definition, and every one of them the same bits again."""
    lib = _lib.load()
    lib.pa_test_set_share(-1, -1)
    g = torch.Generator(device=cuda_device).manual_seed(11)
    seen = set()
    for S, P, own, Hq, Hkv, D, B, fp8 in ((3, 20, 200, 8, 8, 128, 16, False), (40, 64, 90, 32, 8, 128, 16, False), (64, 520, 900, 16, 4, 128, 16, True),
                                          (70, 300, 1500, 32, 8, 64, 32, False), (300, 40, 200, 32, 8, 128, 16, True)):
        mine = -(-own // B)
        NB = P + S * mine
        kv = torch.randn(2, NB, Hkv, B, D, generator=g, device=cuda_device)
        kv = (kv * 16).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else kv.to(torch.bfloat16)
        q = torch.randn(S, Hq, D, generator=g, device=cuda_device).to(torch.bfloat16)
        perm = torch.randperm(NB, generator=g, device=cuda_device).to(torch.int32)
        tables = torch.cat([perm[:P].expand(S, P), perm[P:].view(S, mine)], 1).contiguous()
        lens = (P * B + torch.randint(0, own + 1, (S,), generator=g, device=cuda_device)).to(torch.int32)
        gs = torch.tensor([0, S], dtype=torch.int32, device=cuda_device)
        pb = torch.tensor([P], dtype=torch.int32, device=cuda_device)
        seen.add(_launches(lib, S, 1, Hq, Hkv, D, B, P + mine, P, int(fp8)))
        call = lambda: api.shared_prefix_decode(q, kv[0], kv[1], tables, lens, gs, pb, P, kv_scale=1 / 16)  # noqa: E731
        outs = [call() for _ in range(5)]
        assert all(torch.equal(o, outs[0]) for o in outs) and api.device_errors() == 0
        for s in (0, S // 2, S - 1):
            n = int(lens[s])
            k, v = ((c.view(torch.float8_e4m3fn).double() / 16 if fp8 else c.double())[tables[s].long()].transpose(0, 1).flatten(1, 2)[:, :n]
                    for c in (kv[0], kv[1]))
            p = torch.softmax(q[s].double().view(Hkv, -1, D) @ k.transpose(1, 2) * D ** -0.5, -1)
            want, mass = (p @ v).view(Hq, D), (p @ v.abs()).view(Hq, D)
            # the output's rounding and one of each probability
            assert ((outs[0][s].double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -11 if fp8 else 2.0 ** -8) * mass + 2.0 ** -14).all()
    assert seen == {1, 2, 3}


def test_a_cache_past_32_bits(api, cuda_device):
    """A prefix and rows of its own at the end of a cache of 4.6 GB a side, appended there with a norm and read back by all
    three operators."""
    B, Hkv, D, Hq = 16, 8, 128, 32
    NB = 2 ** 32 // (Hkv * B * D * 2) + 9000
    kc = torch.zeros(NB, Hkv, B, D, dtype=torch.bfloat16, device=cuda_device)
    vc = torch.zeros_like(kc)
    g = torch.Generator().manual_seed(2)
    T = 700
    first = NB - 60
    slots = (first * B + torch.arange(T)).to(torch.int32).to(cuda_device)
    q, k, v = (torch.randn(T, h, D, generator=g).to(torch.bfloat16).to(cuda_device) for h in (Hq, Hkv, Hkv))
    pos = torch.arange(T, dtype=torch.int32, device=cuda_device)
    freq = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).to(cuda_device)
    low_k, low_v = torch.zeros(44, Hkv, B, D, dtype=torch.bfloat16, device=cuda_device), torch.zeros(44, Hkv, B, D, dtype=torch.bfloat16, device=cuda_device)
    rq = api.norm_rope_append(q, k, v, pos, freq, slots, kc, vc)
    low = api.norm_rope_append(q, k, v, pos, freq, slots - first * B, low_k, low_v)
    assert torch.equal(rq, low) and torch.equal(kc[first:first + 44], low_k) and torch.equal(vc[first:first + 44], low_v)
    assert not kc[:first].any() and not kc[first + 44:].any()
    tables = torch.arange(44, dtype=torch.int32, device=cuda_device).expand(3, 44).contiguous()
    lens = torch.tensor([700, 650, 641], dtype=torch.int32, device=cuda_device)
    gs = torch.tensor([0, 3], dtype=torch.int32, device=cuda_device)
    pb = torch.tensor([40], dtype=torch.int32, device=cuda_device)
    a = api.shared_prefix_decode(rq[:3].contiguous(), kc, vc, tables + first, lens, gs, pb, 40)
    assert torch.equal(a, api.shared_prefix_decode(rq[:3].contiguous(), low_k, low_v, tables, lens, gs, pb, 40))
    for rows in (2, 100):
        qs = torch.tensor([0, rows, 2 * rows, 2 * rows + 1], dtype=torch.int32, device=cuda_device)
        x = rq[:2 * rows + 1].contiguous()
        a = api.cross_attention(x, kc, vc, tables + first, lens, qs, rows)
        assert torch.equal(a, api.cross_attention(x, low_k, low_v, tables, lens, qs, rows)) and a.any()
    assert api.device_errors() == 0


def test_as_many_sequences_as_there_may_be(api, cuda_device):
    """65,535 of them in groups of all sizes, against the same call without sharing."""
    B, Hkv, D, S = 16, 1, 64, 65535
    g = torch.Generator().manual_seed(6)
    kc, vc = (torch.randn(200, Hkv, B, D, generator=g).to(torch.bfloat16).to(cuda_device) for _ in range(2))
    q = torch.randn(S, 2, D, generator=g).to(torch.bfloat16).to(cuda_device)
    start = torch.cat([torch.tensor([0, 0, 1]), torch.randint(2, S, (500,), generator=g).sort().values, torch.tensor([S])]).to(torch.int32).to(cuda_device)
    G = start.numel() - 1
    pb = torch.randint(0, 7, (G,), generator=g).to(torch.int32).to(cuda_device)
    of = torch.searchsorted(start, torch.arange(S, dtype=torch.int32, device=cuda_device), right=True) - 1
    tables = torch.randint(0, 200, (G, 8), generator=g).to(torch.int32).to(cuda_device)[of]
    tables[:, 6:] = torch.randint(0, 200, (S, 2), generator=g).to(torch.int32).to(cuda_device)
    lens = torch.randint(0, 8 * B + 1, (S,), generator=g).to(torch.int32).to(cuda_device)
    a = api.shared_prefix_decode(q, kc, vc, tables, lens, start, pb, 6)
    b = api.shared_prefix_decode(q, kc, vc, tables, lens, start, pb, 0)
    # each within 2^-8 of its size for the output's rounding and 2^-8 of the values' for the probabilities'
    assert ((a.float() - b.float()).abs() <= 2.0 ** -7 * (b.float().abs() + vc.float().abs().max())).all()
    assert (a.float() - b.float()).abs().mean() < 2.0 ** -8 and (a[lens == 0] == 0).all() and api.device_errors() == 0
