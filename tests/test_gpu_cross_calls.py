"""Cross attention and the normalised append as a server calls them: rows in front of the first sequence, a captured call whose
rows and states change, caches of torch's own 8-bit type, weights of two kinds in one call."""
import numpy as np
import pytest
import torch

from paged_kv_cache_193_gb300 import workloads as W
from rows_cases import Cross, Shared, within
from test_gpu_norm_rope import NormCase

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api(cuda_device):
    from paged_kv_cache_193_gb300 import api as a
    a._lib_handle()
    return a


@pytest.mark.parametrize("rows,states,Hkv", [([2, 3], [40, 500], 2), ([20, 0, 3], [40, 50, 900], 2), ([(7 * i) % 60 for i in range(30)], [(53 * i) % 200 for i in range(30)], 4)])
@pytest.mark.parametrize("front", [1, 19])
def test_rows_in_front_of_the_first_sequence(api, cuda_device, rows, states, Hkv, front):
    """They are no sequence's, like those behind the last, and stay as they were."""
    case = Cross(cuda_device, rows, states, 8, Hkv, D=64, gap=5)
    g = torch.Generator().manual_seed(1)
    q = torch.cat([torch.randn(front, *case.q.shape[1:], generator=g).to(torch.bfloat16).to(cuda_device), case.q])
    case.qs += front
    out = torch.full_like(q, -7.0)
    case.call(api, q=q, out=out)
    torch.cuda.synchronize()
    assert (out[:front] == -7).all() and (out[q.shape[0] - 5:] == -7).all() and api.device_errors() == 0
    within(out[front:q.shape[0] - 5], case.expected())


@pytest.mark.parametrize("most", [2, 40])
def test_rows_and_states_that_change_between_replays(api, cuda_device, most):
    """One graph for all batches of so many sequences and rows: in each replay others, none and all of them in one sequence
    among them."""
    rng = np.random.default_rng(most)
    S, T = 6, 4 * most
    case = Cross(cuda_device, [T // S] * S, [700] * S, 8, 2)
    T = case.q.shape[0]
    out = torch.empty_like(case.q)
    ws = api.alloc_cross_workspace(case.q, case.pool.kd, case.bt, most)
    case.call(api, most=most, workspace=ws, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        case.call(api, most=most, workspace=ws, out=out)
    for i in range(8):
        rows = [0] * S
        while i and sum(rows) < T and min(rows) < most:
            s = int(rng.integers(S))
            rows[s] += min(most - rows[s], T - sum(rows), int(rng.integers(1, most + 1)))
            if i == 1:
                break
        states = [int(x) for x in rng.integers(0, 701, S)]
        start = np.concatenate([[0], np.cumsum(rows)])
        case.rows, case.states, case.seq = rows, states, np.repeat(np.arange(S), rows)
        case.qs.copy_(torch.tensor(start, dtype=torch.int32))
        case.sl.copy_(torch.tensor(states, dtype=torch.int32))
        out.fill_(-7.0)
        graph.replay()
        torch.cuda.synchronize()
        within(out[:start[-1]], case.expected(), str(rows))
        assert (out[start[-1]:] == -7).all() and api.device_errors() == 0


def test_caches_of_the_8_bit_type(api, cuda_device):
    """float8_e4m3fn and the same bytes as uint8 are one cache."""
    as_type = lambda t: t.view(torch.float8_e4m3fn)  # noqa: E731
    for case in (Cross(cuda_device, [3, 30], [90, 200], 8, 2, fp8=True), Shared(cuda_device, [(200, [9, 50] * 40)], 16, 8, fp8=True)):
        want = case.call(api)
        case.pool.kd, case.pool.vd = as_type(case.pool.kd), as_type(case.pool.vd)
        assert torch.equal(case.call(api), want)
    case = NormCase(cuda_device, T=40, Hq=8, Hkv=2, fp8=True)
    out, kc, vc = case.call(api)
    o2, k2, v2 = case.call(api, kc=as_type(case.k0.clone()), vc=as_type(case.v0.clone()))
    assert torch.equal(out, o2) and np.array_equal(W.bits(kc), W.bits(k2.view(torch.uint8))) and np.array_equal(W.bits(vc), W.bits(v2.view(torch.uint8)))


@pytest.mark.parametrize("q_kind,k_kind", [("shared", "heads"), ("heads", "shared"), ("none", "heads"), ("heads", "none"), ("none", "shared"),
                                           ("shared", "none")])
@pytest.mark.parametrize("D,T", [(64, 5), (128, 700)])
def test_weights_of_two_kinds(api, oracle, cuda_device, q_kind, k_kind, D, T):
    case = NormCase(cuda_device, T=T, Hq=6, Hkv=3, D=D, fused=True, offset=1.0)
    g = torch.Generator().manual_seed(4)
    shape = {"shared": lambda h: (D,), "heads": lambda h: (h, D)}
    case.w = [None if kind == "none" else (0.3 * torch.randn(shape[kind](h), generator=g)).to(torch.bfloat16).to(cuda_device)
              for kind, h in ((q_kind, 6), (k_kind, 3))]
    out, kc, vc = case.call(api)
    torch.cuda.synchronize()
    case.check(oracle, out, kc, vc)
    k2, v2 = case.k0.clone(), case.v0.clone()  # the keys alone, their weights as they are
    assert api.norm_rope_append(None, case.k, case.v, case.pos[0].to(cuda_device), case.freq.to(cuda_device), case.slots.to(cuda_device), k2, v2,
                                k_weight=case.w[1], eps=case.eps, weight_offset=1.0, kv_scale=case.kv_scale) is None
    assert torch.equal(k2, kc) and torch.equal(v2, vc) and api.device_errors() == 0
