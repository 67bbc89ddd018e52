"""Cross attention over the paged cache against its definition in 64 bits."""
import numpy as np
import pytest
import torch

from gpu_helpers import Guarded
from paged_kv_cache_193_gb300 import _lib
from rows_cases import Cross, Shared, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api(cuda_device):
    from paged_kv_cache_193_gb300 import api as a
    a._lib_handle()
    return a


CASES = [
    dict(rows=[1], states=[1], Hq=1, Hkv=1, D=64),
    dict(rows=[1], states=[1500], Hq=4, Hkv=4, D=64),
    dict(rows=[1, 1, 1], states=[63, 64, 65], Hq=8, Hkv=2),
    dict(rows=[5, 5], states=[700, 333], Hq=8, Hkv=2),
    dict(rows=[0, 3, 0, 7], states=[10, 0, 0, 40], Hq=6, Hkv=2, B=32),
    dict(rows=[33, 1, 129], states=[15, 16, 17], Hq=4, Hkv=1),
    dict(rows=[64, 65, 31], states=[100, 48, 256], Hq=2, Hkv=1, D=64, B=32),
    dict(rows=[18, 19, 37], states=[90, 5, 128], Hq=7, Hkv=1),                # 18 rows of 7 heads to a tile
    dict(rows=[9, 17, 2], states=[64, 300, 2], Hq=16, Hkv=1, D=64),
    dict(rows=[11, 40], states=[130, 31], Hq=10, Hkv=2, fp8=True),
    dict(rows=[11, 40, 1], states=[130, 31, 900], Hq=6, Hkv=2, D=64, fp8=True, per_head=True),
    dict(rows=[3, 70], states=[1000, 65], Hq=8, Hkv=2, B=32, fp8=True, per_head=True),
    dict(rows=[0, 2, 5], states=[7, 0, 1], Hq=8, Hkv=2, D=64, B=32, fp8=True),
    dict(rows=[2, 3], states=[40, 50], Hq=8, Hkv=2, gap=4),                   # rows of no sequence
    dict(rows=[2, 3], states=[40, 50], Hq=8, Hkv=2, extra=300),               # a table wider than its states
    dict(rows=[4, 1], states=[3000, 2999], Hq=8, Hkv=2),
    dict(rows=[2] * 80, states=[(37 * i) % 90 for i in range(80)], Hq=4, Hkv=2, D=64),  # one part
    dict(rows=[130] * 5, states=[200, 0, 64, 65, 1], Hq=16, Hkv=8, D=64),
    dict(rows=[2, 3], states=[40, 50], Hq=8, Hkv=2, extra=200000),            # far wider: few rows, a tile, two
    dict(rows=[20, 3], states=[40, 50], Hq=8, Hkv=2, extra=200000),
    dict(rows=[70, 3], states=[40, 50], Hq=8, Hkv=2, extra=200000),
    # taken by length: ties, none, bad ends
    dict(rows=[(7 * i) % 90 for i in range(45)], states=[(53 * i) % 200 for i in range(45)], Hq=8, Hkv=4, D=64),
    dict(rows=[40] * 33, states=[64] * 33, Hq=6, Hkv=3, fp8=True, gap=3),
    dict(rows=[0] * 30 + [70], states=[100] * 31, Hq=20, Hkv=5),
    dict(rows=[70] + [0] * 250, states=[i for i in range(251)], Hq=16, Hkv=8, D=64),
    dict(rows=[9] * 300, states=[(11 * i) % 70 for i in range(300)], Hq=2, Hkv=1, D=64),  # more than are sorted
    # few rows, by eight warps: one CTA to a row, eight
    dict(rows=[1] * 60, states=[(53 * i) % 400 for i in range(60)], Hq=8, Hkv=4),
    dict(rows=[2, 1, 0] * 25, states=[(31 * i) % 300 for i in range(75)], Hq=12, Hkv=3, D=64, fp8=True, per_head=True),
    dict(rows=[1, 3], states=[3000, 777], Hq=4, Hkv=2, D=64),
    dict(rows=[2], states=[5001], Hq=8, Hkv=2, B=32, fp8=True),
    dict(rows=[2] * 40, states=[(97 * i) % 300 for i in range(40)], Hq=16, Hkv=2, fp8=True, per_head=True),
]


@pytest.mark.parametrize("kw", CASES, ids=[f"{i}" for i in range(len(CASES))])
def test_matches_the_definition(api, cuda_device, kw):
    case = Cross(cuda_device, **kw)
    T, Hq, D = case.q.shape
    n = api.cross_workspace_size(T, len(case.rows), min(case.most, T), Hq, case.pool.Hkv, D, case.bt.shape[1], case.pool.B)
    ws = Guarded((n,), torch.uint8, cuda_device)
    out = Guarded(case.q.shape, torch.bfloat16, cuda_device, fill=-7.0)
    k0, q0 = case.pool.kd.clone(), case.q.clone()
    got = case.call(api, workspace=ws.tensor if n else None, out=out.tensor)
    torch.cuda.synchronize()
    assert got.data_ptr() == out.tensor.data_ptr() and api.device_errors() == 0
    want = case.expected()
    live = T - case.gap
    within(got[:live], want)
    assert (got[live:] == -7).all()
    for i, s in enumerate(case.seq):
        assert case.states[s] or (got[i] == 0).all()
    ws.check("workspace")
    out.check("out")
    assert torch.equal(case.q, q0) and torch.equal(case.pool.kd.view(torch.uint8), k0.view(torch.uint8))
    assert torch.equal(case.call(api)[:live], got[:live])
    q = case.q.clone()
    assert torch.equal(case.call(api, q=q, out=q)[:live], got[:live])
    assert torch.equal(q[live:], q0[live:])
    within(case.call(api, most=10 ** 6)[:live], want, "a bound far above the rows")


def test_one_row_is_the_decode(api, cuda_device):
    """One row a sequence is what the decode kernel computes over the same table."""
    case = Cross(cuda_device, [1] * 5, [1, 20, 333, 64, 1000], 8, 2)
    a = case.call(api)
    b = api.decode(case.q, case.pool.kd, case.pool.vd, case.bt, case.sl, case.scale)
    assert (a.float() - b.float()).abs().max() <= 2.0 ** -6


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows", [[3, 40], [300, 2]])
def test_large_scores(api, cuda_device, fp8, rows):
    case = Cross(cuda_device, rows, [900, 333], 8, 2, fp8=fp8, spread=30.0 if not fp8 else 20.0)
    within(case.call(api), case.expected())


def test_infinities_stay_where_they_are(api, cuda_device):
    case = Cross(cuda_device, [3, 3], [200, 100], 4, 2)
    want = case.expected()
    case.pool.vd[int(case.tables[0, 2]), 1, 4, 9] = float("inf")
    got = case.call(api).float().cpu()
    assert torch.isinf(got[:3, 2:, 9]).all()
    keep = np.ones(got.shape, bool)
    keep[:3, 2:, 9] = False
    assert (np.abs(got.numpy() - want[0]) <= want[1])[keep].all()


def test_refused_rows_are_reported_and_left(api, cuda_device):
    case = Cross(cuda_device, [3, 40, 2], [200, 100, 50], 4, 2)
    want = case.expected()
    out = Guarded(case.q.shape, torch.bfloat16, cuda_device, fill=-7.0)
    got = case.call(api, most=39, out=out.tensor)  # one sequence has more
    torch.cuda.synchronize()
    assert api.device_errors() == _lib.PA_DEVERR_BAD_CONTEXT
    assert (got[3:43] == -7).all()
    within(got[:3], tuple(x[:3] for x in want))
    within(got[43:], tuple(x[43:] for x in want))
    for start in ([0, 3, 43, 46], [0, 3, 2, 45], [-1, 3, 43, 45], [2 ** 31 - 1, -2 ** 31, 43, 45]):
        case.qs.copy_(torch.tensor(start, dtype=torch.int32))
        case.call(api, out=out.tensor)
        torch.cuda.synchronize()
        assert api.device_errors() == _lib.PA_DEVERR_BAD_CONTEXT
        out.check(str(start))


def test_bad_blocks_and_lengths(api, cuda_device):
    case = Cross(cuda_device, [3, 2], [200, 100], 4, 2)
    case.bt[0, 2] = 10 ** 6
    assert torch.isfinite(case.call(api)).all() and api.device_errors() == _lib.PA_DEVERR_BAD_BLOCK
    case.bt.copy_(case.tables)
    case.sl[1] = 10 ** 6
    case.call(api)
    assert api.device_errors() & _lib.PA_DEVERR_BAD_CONTEXT
    case.sl[1] = -4
    assert (case.call(api)[3:] == 0).all() and api.device_errors() == 0


@pytest.mark.parametrize("rows", [[1, 1], [300, 200]])
def test_captured_and_replayed(api, cuda_device, rows):
    case = Cross(cuda_device, rows, [700, 90], 8, 2, D=64)
    want = case.expected()
    out = torch.empty_like(case.q)
    ws = api.alloc_cross_workspace(case.q, case.pool.kd, case.bt, case.most)
    case.call(api, workspace=ws, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        case.call(api, workspace=ws, out=out)
    for _ in range(3):
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        within(out, want)
    case.sl[0], case.states = 77, [77, 90]
    g.replay()
    torch.cuda.synchronize()
    within(out, case.expected())


def test_on_another_stream_and_back_to_back(api, cuda_device):
    case = Cross(cuda_device, [2, 3], [500, 900], 8, 2)
    ws = api.alloc_cross_workspace(case.q, case.pool.kd, case.bt, case.most)

    def chain(after, stream=None):
        x, got = case.q.clone(), []
        torch.cuda.synchronize()
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            for _ in range(40):
                y = case.call(api, q=x, workspace=ws, stream=stream)
                after()
                x = (y * 3).contiguous()
                after()
                got.append(y)
        return got

    want = chain(torch.cuda.synchronize)
    for stream in (None, torch.cuda.Stream()):
        got = chain(lambda: None, stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_wait_that_runs_out(api, cuda_device):
    lib = _lib.load()
    for fp8 in (False, True):
        for rows in ([2, 3], [300, 3]):
            case = Cross(cuda_device, rows, [500, 900], 8, 2, fp8=fp8)
            assert lib.pa_test_set_wait(1_000_000, 1) == 0
            try:
                case.call(api)
                torch.cuda.synchronize()
            finally:
                assert lib.pa_test_set_wait(0, 0) == 0
            assert api.device_errors() & _lib.PA_DEVERR_TIMEOUT
            within(case.call(api), case.expected())
            assert api.device_errors() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fp8", [False, True])
def test_long_runs_give_the_same_bits_every_time(api, cuda_device, fp8, D):
    """Enough rows that no run is cut into parts, so every ring of stages goes round many times, and enough CTAs that a page
    landing too early would be seen; sampled rows against the definition."""
    g = torch.Generator(device=cuda_device).manual_seed(3)
    S, n, Hq, Hkv, B, rows = 40, 2029, 24, 8, 32, 126
    MB = -(-n // B)
    kv = torch.randn(2, S * MB, Hkv, B, D, generator=g, device=cuda_device)
    kv = (kv * 16).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else kv.to(torch.bfloat16)
    q = torch.randn(S * rows, Hq, D, generator=g, device=cuda_device).to(torch.bfloat16)
    tables = torch.randperm(S * MB, generator=g, device=cuda_device).view(S, MB).to(torch.int32)
    lens = torch.full((S,), n, dtype=torch.int32, device=cuda_device)
    start = torch.arange(0, S * rows + 1, rows, dtype=torch.int32, device=cuda_device)
    outs = [api.cross_attention(q, kv[0], kv[1], tables, lens, start, rows, kv_scale=1 / 16).clone() for _ in range(20)]
    assert all(torch.equal(o, outs[0]) for o in outs) and api.device_errors() == 0
    for s in (0, 17, 39):
        k, v = ((c.view(torch.float8_e4m3fn).double() / 16 if fp8 else c.double())[tables[s].long()].transpose(0, 1).flatten(1, 2)[:, :n]
                for c in kv)
        x = q[s * rows:(s + 1) * rows].double().view(rows, Hkv, 3, D).permute(1, 2, 0, 3).flatten(1, 2)
        p = torch.softmax(x @ k.transpose(1, 2) * D ** -0.5, -1)
        want, mass = p @ v, p @ v.abs()
        got = outs[0][s * rows:(s + 1) * rows].double().view(rows, Hkv, 3, D).permute(1, 2, 0, 3).flatten(1, 2)
        # the output's rounding, and one of each probability (2^-8 of it in bf16, 2^-11 in fp16)
        assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -11 if fp8 else 2.0 ** -8) * mass + 2.0 ** -14).all()


def test_refused_rows_among_many(api, cuda_device):
    """The same where sequences are taken by length."""
    case = Cross(cuda_device, [30] * 20, [(31 * i) % 150 for i in range(20)], 16, 8, D=64)
    want = case.expected()
    out = torch.full_like(case.q, -7.0)
    start = case.qs.clone()
    start[8] = 5 * 30  # sequence 7 has none that ascend, 8 twice as many as may be
    case.qs.copy_(start)
    case.call(api, out=out, most=30)
    torch.cuda.synchronize()
    assert api.device_errors() == _lib.PA_DEVERR_BAD_CONTEXT
    bad = slice(7 * 30, 9 * 30)
    assert (out[bad] == -7).all()
    keep = np.r_[0:7 * 30, 9 * 30:600]
    within(out[torch.from_numpy(keep)], tuple(x[keep] for x in want))


def test_as_many_sequences_as_there_may_be(api, cuda_device):
    """65,535 sequences of up to three rows, against the decode kernel over each row's table."""
    B, D, S = 16, 64, 65535
    g = torch.Generator().manual_seed(9)
    kc, vc = (torch.randn(200, 1, B, D, generator=g).to(torch.bfloat16).to(cuda_device) for _ in range(2))
    rows = torch.randint(0, 4, (S,), generator=g)
    start = torch.cat([torch.zeros(1, dtype=torch.int64), rows.cumsum(0)]).to(torch.int32).to(cuda_device)
    T = int(start[-1])
    q = torch.randn(T, 8, D, generator=g).to(torch.bfloat16).to(cuda_device)
    tables = torch.randint(0, 200, (S, 5), generator=g).to(torch.int32).to(cuda_device)
    lens = torch.randint(0, 5 * B + 1, (S,), generator=g).to(torch.int32).to(cuda_device)
    got = api.cross_attention(q, kc, vc, tables, lens, start, 3)
    seq = torch.repeat_interleave(torch.arange(S), rows).to(cuda_device)
    pick = torch.randint(0, T, (500,), generator=g).to(cuda_device)
    want = api.decode(q[pick].contiguous(), kc, vc, tables[seq[pick]].contiguous(), lens[seq[pick]].contiguous())
    assert ((got[pick].float() - want.float()).abs() <= 2.0 ** -7 * (want.float().abs() + vc.float().abs().max())).all()
    assert (got[lens[seq] == 0] == 0).all() and api.device_errors() == 0


def test_calls_at_once(api, cuda_device):
    """Cross attention in small and large tiles, shared prefixes joined in both ways, and a chunked prefill, each in a graph
    and a workspace of its own, replayed on streams that run together: the same bits as one after the other."""
    lib = _lib.load()
    small = Cross(cuda_device, [(5 * i) % 30 for i in range(40)], [(53 * i) % 900 for i in range(40)], 16, 8)
    large = Cross(cuda_device, [(7 * i) % 200 for i in range(25)], [(97 * i) % 600 for i in range(25)], 16, 4, D=64, fp8=True)
    shared = [Shared(cuda_device, [(60, [(7 * i) % 90 for i in range(40)])], 8, 4, seed=i) for i in range(2)]
    outs = [torch.zeros_like(c.q) for c in (small, large, *shared)]
    T = 300
    chunk = torch.tensor([0, T], dtype=torch.int32, device=cuda_device)
    table = torch.arange(30, dtype=torch.int32, device=cuda_device).view(1, 30)
    length = torch.tensor([400], dtype=torch.int32, device=cuda_device)
    kv = torch.randn(2, 30, 4, 16, 64, device=cuda_device).to(torch.bfloat16)
    qp = torch.randn(T, 16, 64, device=cuda_device).to(torch.bfloat16)
    outs.append(torch.zeros_like(qp))
    ws = [api.alloc_cross_workspace(c.q, c.pool.kd, c.bt, c.most) for c in (small, large)]

    def prefix(i):
        lib.pa_test_set_share(0, i)
        try:
            shared[i].call(api, out=outs[2 + i], workspace=ws[2 + i])
        finally:
            lib.pa_test_set_share(-1, -1)

    lib.pa_test_set_share(0, -1)
    ws += [api.alloc_shared_prefix_workspace(c.q, c.pool.kd, c.gs, c.most) for c in shared]
    lib.pa_test_set_share(-1, -1)
    calls = [lambda: small.call(api, out=outs[0], workspace=ws[0]), lambda: large.call(api, out=outs[1], workspace=ws[1]),
             lambda: prefix(0), lambda: prefix(1),
             lambda: api.prefill(qp, kv[0], kv[1], table, length, chunk, T, out=outs[4])]
    for c in calls:
        c()
        torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    graphs, streams = [], [torch.cuda.Stream() for _ in calls]
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(10):
                c()
        graphs.append(g)
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
    assert api.device_errors() == 0
