"""Kernels that are put on the SMs while the one before them still runs read
its results by loads that their wait orders."""
import glob
import os
import re

import pytest
import torch

from paged_kv_cache_193_gb300 import build


def _code(path):
    with open(path) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def test_no_read_only_loads_in_dependent_kernels():
    """``__ldg``, ld.global.nc and what a compiler makes of const __restrict__ promise that nobody writes the memory for
    as long as the kernel is there, and nothing orders them behind griddepcontrol.wait: the kernel before may write it."""
    sources = [p for p in sorted(glob.glob(os.path.join(build.CSRC, "*.cu*")))
               if "launch_dependent(" in _code(p) or "dependent_wait()" in _code(p)
               or os.path.basename(p) == "pa_sparse_select.cuh"]  # called by two of them
    assert len(sources) >= 5
    for p in sources:
        assert not re.search(r"__ldg|\.nc\b|__restrict__", _code(p)), os.path.basename(p)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_a_rotated_query_goes_straight_into_the_choice_and_the_attention(cuda_device, fp8):
    """One output of rope_append, tables and scales that are rewritten all the time, and read by the next kernel: bit for
    bit what the same calls give when each is waited for."""
    from paged_kv_cache_193_gb300 import api
    g = torch.Generator().manual_seed(51)
    S, Hq, Hkv, D, B, MB, steps = 5, 8, 2, 128, 16, 48, 60
    NB = S * MB
    q = torch.randn(steps, S, Hq, D, generator=g).to(torch.bfloat16).to(cuda_device)
    kv = torch.randn(2, NB, Hkv, B, D, generator=g)
    kv = ((kv * 16).to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else kv.to(torch.bfloat16)).to(cuda_device)
    kc, vc = kv[0], kv[1]
    tables = torch.stack([torch.randperm(NB, generator=g).view(S, MB) for _ in range(steps)]).to(torch.int32).to(cuda_device)
    scales = (torch.rand(steps, Hkv, generator=g) / 16 + 1 / 32).to(cuda_device)
    lens = torch.tensor([700, 768, 512, 33, 600], dtype=torch.int32, device=cuda_device)
    pos = torch.randint(0, 5000, (steps, S), generator=g).to(torch.int32).to(cuda_device)
    none = torch.full((S,), -1, dtype=torch.int32, device=cuda_device)
    new = torch.zeros(S, Hkv, D, dtype=torch.bfloat16, device=cuda_device)
    freq = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).to(cuda_device)
    s, e = api.alloc_block_summary(kc)
    api.block_summary(kc, torch.arange(B - 1, NB * B, B, dtype=torch.int32, device=cuda_device), s, e)

    def chain(after):
        rq, table = torch.zeros_like(q[0]), torch.zeros_like(tables[0])
        ks = torch.ones(Hkv, device=cuda_device) if fp8 else None
        got = []
        for i in range(steps):
            table.copy_(tables[i])
            if fp8:
                ks.copy_(scales[i])
            for x in (q[i], q[i - 1]):
                after()
                api.rope_append(x, new, new, pos[i], freq, none, kc, vc, out=rq)
                after()
                got.append(api.sparse_attend(rq, kc, vc, s, e, table, lens, 9, k_scales=ks, v_scales=ks))
                after()
                api.rope_append(x, new, new, pos[i - 1], freq, none, kc, vc, out=rq)
                after()
                sel, cnt = api.sparse_select(rq, s, e, table, lens, B, 9)
                after()
                api.rope_append(x, new, new, pos[i], freq, none, kc, vc, out=rq)
                after()
                got += [sel, cnt, api.sparse_decode(rq, kc, vc, table, lens, sel, cnt, k_scales=ks, v_scales=ks)]
        return got

    want = chain(torch.cuda.synchronize)
    for _ in range(3):
        got = chain(lambda: None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert not torch.equal(want[0], want[4]) and api.device_errors() == 0
