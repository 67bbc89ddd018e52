"""Calls of the block-sparse decode that its documentation allows, beside the ordinary ones."""
import pytest
import torch

from test_gpu_sparse import Case, api  # noqa: F401  (api: a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,Hq,Hkv,top_k", [([900, 41, 300], 8, 2, 9), ([5000], 16, 2, 64), ([400] * 200, 32, 4, 12), ([20000], 16, 1, 100)])
@pytest.mark.parametrize("fp8", [False, True])
def test_the_output_may_be_the_query(api, cuda_device, lens, Hq, Hkv, top_k, fp8):  # noqa: F811
    """Each KV head's queries are read before its outputs are written, however many CTAs share it."""
    case = Case(cuda_device, lens, Hq, Hkv, fp8=fp8)
    s, e = case.summaries(api)
    args = case.kc, case.vc, s, e, case.bt, case.cl, top_k, 1, 2, case.scale, case.kv_scale
    want = api.sparse_attend(case.q, *args)
    q = case.q.clone()
    assert torch.equal(api.sparse_attend(q, *args, out=q), want)
    sel, cnt = api.sparse_select(case.q, s, e, case.bt, case.cl, 16, top_k)
    for splits in (0, 1, 2, 4, 8):
        args = case.kc, case.vc, case.bt, case.cl, sel, cnt, case.scale, case.kv_scale
        want = api.sparse_decode(case.q, *args, splits=splits)
        q = case.q.clone()
        assert torch.equal(api.sparse_decode(q, *args, splits=splits, out=q), want)


def test_as_many_rows_as_there_may_be(api, cuda_device):  # noqa: F811
    """65,535 rows of one sequence, each with a length of its own."""
    case = Case(cuda_device, [2000], 2, 1, D=64)
    s, e = case.summaries(api)
    g = torch.Generator().manual_seed(8)
    n = 65535
    q = torch.randn(n, 2, 64, generator=g).to(torch.bfloat16).to(cuda_device)
    lens = torch.randint(0, 2001, (n,), generator=g).to(torch.int32).to(cuda_device)
    tables = case.bt.expand(n, -1).contiguous()
    out = api.sparse_attend(q, case.kc, case.vc, s, e, tables, lens, 9)
    pick = torch.randint(0, n, (40,), generator=g).to(cuda_device)
    few = api.sparse_attend(q[pick], case.kc, case.vc, s, e, tables[pick], lens[pick], 9)
    # another number of CTAs joins their parts in another order: an output apart by a rounding of bf16
    assert (out[pick].float() - few.float()).abs().max() <= 2.0 ** -7 * few.float().abs().max()
    assert (out[lens == 0] == 0).all() and api.device_errors() == 0
