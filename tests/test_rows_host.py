"""Refusals of the normalised append, shared-prefix decode and cross attention, in the C ABI and in the Python binding, their
workspaces' sizes, and the tests' own reference (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import rows_cases
from paged_kv_cache_193_gb300 import api

FAKE = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 8)
FAR = ctypes.c_void_p(1 << 30)
FARTHER = ctypes.c_void_p(1 << 32)
bf = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_193_gb300 import build, _lib
    build.build()
    return _lib.load()


def _norm(lib, **kw):
    a = dict(q=FAKE, qs=1024, k=FAKE, ks=256, v=FAKE, vs=256, qw=FAKE, qws=0, kw=FAKE, kws=0, off=0.0, eps=1e-6, pos=FAKE, axes=1,
             freq=FAKE, axis=None, R=128, adj=0, mag=1.0, slots=FAKE, T=4, Hq=8, qo=FAR, kc=FAKE, vc=FAKE, NB=64, Hkv=2, D=128, B=16,
             dt=0, kvs=1.0, ksc=None, vsc=None)
    a.update(kw)
    return lib.pa_norm_rope_append(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["qw"], a["qws"], a["kw"], a["kws"], a["off"],
                                   a["eps"], a["pos"], a["axes"], a["freq"], a["axis"], a["R"], a["adj"], a["mag"], a["slots"],
                                   a["T"], a["Hq"], a["qo"], a["kc"], a["vc"], a["NB"], a["Hkv"], a["D"], a["B"], a["dt"], a["kvs"],
                                   a["ksc"], a["vsc"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(D=96), 2), (dict(R=24), 2), (dict(axes=3), 1), (dict(mag=0.0), 1), (dict(k=None), 1), (dict(qo=None), 1),
    (dict(q=ODD), 1), (dict(qs=1016), 1), (dict(k=FAR), 1), (dict(dt=1, kvs=0.0), 1), (dict(NB=1 << 28), 2),
    (dict(eps=0.0), 1), (dict(eps=-1.0), 1), (dict(eps=1e-13), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(off=float("nan")), 1), (dict(off=float("-inf")), 1), (dict(qw=ODD), 1), (dict(kw=ODD), 1),
    (dict(qws=-128), 1), (dict(qws=120), 1), (dict(kws=132), 1), (dict(qw=FAR), 1), (dict(kw=FAR), 1),
    (dict(qw=ctypes.c_void_p((1 << 30) - 2032), qws=128), 1),      # the last head's weights lie on q_out
])
def test_norm_rope_append_rejects_on_host(lib, kw, status):
    assert _norm(lib, **kw) == status
    assert lib.pa_last_error()


def test_norm_rope_append_of_nothing_is_a_no_op(lib):
    assert _norm(lib, T=0, q=None, k=None, v=None) == 0


def _shared(lib, **kw):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, mb=4096, cl=FAKE, S=8, gs=FAKE, pb=FAKE, G=2, mp=4096, Hq=8, Hkv=2, D=128, NB=64, B=16,
             dt=0, kvs=1.0, ksc=None, vsc=None, sm=0.088, ws=FARTHER, wsb=1 << 30, out=FAR)
    a.update(kw)
    return lib.pa_shared_prefix_decode(a["q"], a["kc"], a["vc"], a["bt"], a["mb"], a["cl"], a["S"], a["gs"], a["pb"], a["G"], a["mp"],
                                       a["Hq"], a["Hkv"], a["D"], a["NB"], a["B"], a["dt"], a["kvs"], a["ksc"], a["vsc"], a["sm"],
                                       a["ws"], a["wsb"], a["out"], None)


def _cross(lib, **kw):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, mb=64, cl=FAKE, qs=FAKE, S=4, T=9, mq=5, Hq=8, Hkv=2, D=128, NB=64, B=16, dt=0, kvs=1.0,
             ksc=None, vsc=None, sm=0.088, ws=FARTHER, wsb=1 << 30, out=FAR)
    a.update(kw)
    return lib.pa_cross_attention(a["q"], a["kc"], a["vc"], a["bt"], a["mb"], a["cl"], a["qs"], a["S"], a["T"], a["mq"], a["Hq"],
                                  a["Hkv"], a["D"], a["NB"], a["B"], a["dt"], a["kvs"], a["ksc"], a["vsc"], a["sm"], a["ws"], a["wsb"],
                                  a["out"], None)


@pytest.mark.parametrize("call", [_shared, _cross])
@pytest.mark.parametrize("kw,status", [
    (dict(S=-1), 1), (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(Hkv=3), 1), (dict(Hq=64, Hkv=2), 2), (dict(D=96), 2), (dict(B=8), 2),
    (dict(NB=0), 1), (dict(mb=0), 1), (dict(mb=1 << 28), 1), (dict(mb=(1 << 27) - 1), 2), (dict(S=70000), 2), (dict(NB=1 << 27), 2), (dict(dt=3), 2),
    (dict(sm=0.0), 1), (dict(sm=-1.0), 1), (dict(sm=float("nan")), 1), (dict(sm=float("inf")), 1), (dict(ksc=FAKE), 1),
    (dict(ksc=FAKE, vsc=FAKE), 1), (dict(dt=1, kvs=0.0), 1), (dict(dt=1, ksc=FAKE), 1),
    (dict(q=None), 1), (dict(kc=None), 1), (dict(vc=None), 1), (dict(bt=None), 1), (dict(cl=None), 1), (dict(out=None), 1),
    (dict(q=ODD), 1), (dict(kc=ODD), 1), (dict(vc=ODD), 1), (dict(out=ODD), 1),
    (dict(out=ctypes.c_void_p((1 << 20) + 16)), 1), (dict(out=ctypes.c_void_p((1 << 20) - 16)), 1),
    (dict(ws=None), 3), (dict(wsb=1000), 3), (dict(ws=ctypes.c_void_p((1 << 32) + 8)), 1), (dict(ws=FAKE), 1), (dict(ws=FAR), 1),
])
def test_both_attentions_reject_on_host(lib, call, kw, status):
    assert call(lib, **kw) == status
    assert lib.pa_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(G=-1), 1), (dict(G=9), 1), (dict(mp=-1), 1), (dict(mp=1 << 28), 2), (dict(gs=None), 1), (dict(pb=None), 1),
])
def test_shared_prefix_rejects_on_host(lib, kw, status):
    assert _shared(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [(dict(T=-1), 1), (dict(mq=-1), 1), (dict(mq=0), 1), (dict(qs=None), 1)])
def test_cross_rejects_on_host(lib, kw, status):
    assert _cross(lib, **kw) == status


def test_the_share_hook_is_checked(lib):
    assert lib.pa_test_set_share(0, 2) == 1 and lib.pa_test_set_share(-1, -1) == 0


def test_nothing_to_do_is_a_no_op(lib):
    assert _shared(lib, S=0, G=0, q=None, out=None) == 0
    assert _cross(lib, S=0, q=None, out=None) == 0
    assert _cross(lib, T=0, mq=0, q=None, out=None) == 0


def test_workspace_sizes(lib):
    size = api.shared_prefix_workspace_size
    assert size(4, 0, 8, 2, 128, 16, 32) == 0 == size(4, 1, 8, 2, 128, 16, 0)  # nothing shared
    assert size(4, 1, 9, 2, 128, 16, 32) == 0                                  # the call refuses such heads
    assert size(4, 1, 32, 8, 128, 16, 63) == 0                                 # little to share: 16.5 MB
    assert size(23, 1, 32, 8, 128, 16, 65) == 0 != size(24, 1, 32, 8, 128, 16, 65)  # 98.0 and 102.2 MB
    assert size(46, 1, 32, 8, 128, 16, 65, 1) == 0 != size(48, 1, 32, 8, 128, 16, 65, 1)  # E4M3: half of that each
    assert size(7, 1, 32, 8, 128, 16, 435) == 0 != size(7, 1, 32, 8, 128, 16, 436)  # few sequences: 199.6 and 200.02 MB
    assert size(8, 1, 32, 8, 128, 16, 435) != 0 == size(8, 2, 32, 8, 128, 16, 381)  # eight to a group, four: 228 and 199.8 MB
    try:
        assert lib.pa_test_set_share(0, -1) == 0
        for n in (1, 4, 256, 65535):
            row = n * 32 * (128 + 2) * 4
            got = size(n, 1, 32, 8, 128, 16, 2048)
            assert got % row == 0 and 2 <= got // row <= 33                   # the prefix's parts and the rest's
        assert size(65535, 1, 32, 8, 128, 16, 128) == 2 * 65535 * 32 * 130 * 4  # enough tiles: one part
        assert size(4, 0, 8, 2, 128, 16, 32) == 0 == size(4, 1, 8, 2, 128, 16, 0)
    finally:
        assert lib.pa_test_set_share(-1, -1) == 0
    size = api.cross_workspace_size
    assert size(8192, 16, 512, 32, 8, 128, 128, 16) == 0                       # one part, which needs none
    assert size(1, 1, 1, 16, 16, 64, 94, 16) == 0                              # a handful of rows: a kernel that needs none
    row = 20 * 16 * (64 + 2) * 4
    got = size(20, 1, 20, 16, 16, 64, 94, 16)
    assert got % row == 0 and 2 <= got // row <= 32
    assert size(20, 1, 10 ** 6, 16, 16, 64, 94, 16) == got                     # no more rows than there are
    assert size(0, 1, 1, 16, 16, 64, 94, 16) == 0


# ---- the Python binding: host tensors meet every check but the device's, which comes last ----

def z(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype)


def _norm_args():
    return dict(q=z(3, 4, 64, dtype=bf), k=z(3, 2, 64, dtype=bf), v=z(3, 2, 64, dtype=bf), positions=z(3),
                inv_freq=torch.ones(32, dtype=torch.float64), slot_mapping=z(3), k_cache=z(4, 2, 16, 64, dtype=bf),
                v_cache=z(4, 2, 16, 64, dtype=bf), out=z(3, 4, 64, dtype=bf), q_weight=z(64, dtype=bf), k_weight=z(2, 64, dtype=bf))


@pytest.mark.parametrize("change,err,match", [
    (dict(q=z(2, 4, 64, dtype=bf)), ValueError, "inconsistent q and k"),
    (dict(k=z(3, 128, dtype=bf)), ValueError, "3 dimensions"),
    (dict(q_weight=z(64)), TypeError, "q_weight"),
    (dict(q_weight=z(32, dtype=bf)), ValueError, "q_weight"),
    (dict(q_weight=z(2, 64, dtype=bf)), ValueError, "q_weight"),
    (dict(q_weight=z(64, 4, dtype=bf).t()), ValueError, "contiguous"),
    (dict(k_weight=z(4, 64, dtype=bf)), ValueError, "k_weight"),
    (dict(k_weight=z(1, 2, 64, dtype=bf)), ValueError, "k_weight"),
    (dict(eps="small"), TypeError, None),
    (dict(weight_offset=None), TypeError, None),
    ({}, ValueError, "CUDA tensor"),
    (dict(q_weight=None, k_weight=None), ValueError, "CUDA tensor"),
    (dict(q_weight=z(4, 64, dtype=bf)), ValueError, "CUDA tensor"),
])
def test_norm_rope_append_binding_refuses(lib, change, err, match):
    with pytest.raises(err, match=match):
        api.norm_rope_append(**{**_norm_args(), **change})


def _caches():
    return dict(k_cache=z(4, 2, 16, 64, dtype=bf), v_cache=z(4, 2, 16, 64, dtype=bf))


def _shared_args():
    return dict(q=z(3, 4, 64, dtype=bf), block_tables=z(3, 8), context_lens=z(3), group_start=z(3), prefix_blocks=z(2),
                max_prefix_blocks=4, out=z(3, 4, 64, dtype=bf), **_caches())


def _cross_args():
    return dict(q=z(5, 4, 64, dtype=bf), block_tables=z(3, 8), state_lens=z(3), query_start=z(4), max_query_len=3,
                out=z(5, 4, 64, dtype=bf), **_caches())


@pytest.mark.parametrize("fns,change,err,match", [
    ("shared cross", dict(q=z(3, 4, 64, dtype=torch.float16)), TypeError, "q has dtype"),
    ("shared cross", dict(q=z(3, 4, 64, dtype=bf).transpose(0, 1)), ValueError, "contiguous"),
    ("shared cross", dict(block_tables=z(3, 8, dtype=torch.int64)), TypeError, "block_tables"),
    ("shared", dict(block_tables=z(2, 8)), ValueError, "block_tables"),
    ("shared", dict(context_lens=z(2)), ValueError, "context_lens"),
    ("shared", dict(prefix_blocks=z(3)), ValueError, "group_start"),
    ("shared", dict(group_start=z(3, dtype=torch.int64)), TypeError, "group_start"),
    ("shared", dict(group_start=z(3, 1)), ValueError, "group_start"),
    ("cross", dict(block_tables=z(2, 8)), ValueError, "state_lens"),
    ("cross", dict(state_lens=z(2)), ValueError, "state_lens"),
    ("cross", dict(query_start=z(3)), ValueError, "query_start"),
    ("cross", dict(max_query_len=2 ** 40), (ValueError, ctypes.ArgumentError), None),
    ("shared cross", dict(workspace=z(100)), TypeError, "workspace"),
    ("shared cross", dict(workspace=z(10, 10, dtype=torch.uint8)), ValueError, "workspace"),
    ("shared cross", dict(v_scales=torch.ones(2)), ValueError, "both"),
    ("shared cross", dict(out=z(2, 4, 64, dtype=bf)), ValueError, "out"),
    ("shared cross", dict(k_cache=z(4, 2, 16, 128, dtype=bf), v_cache=z(4, 2, 16, 128, dtype=bf)), ValueError, "inconsistent"),
    ("shared cross", {}, ValueError, "CUDA tensor"),
])
def test_attention_bindings_refuse(lib, fns, change, err, match):
    for fn in fns.split():
        args, call = (_shared_args(), api.shared_prefix_decode) if fn == "shared" else (_cross_args(), api.cross_attention)
        with pytest.raises(err, match=match):
            call(**{**args, **change})


def test_a_step_holds_its_buffers():
    kc = z(4, 2, 16, 64, dtype=bf)
    wide = 3, 20000  # 320,000 tokens of prefix: enough to share
    step = api.SharedPrefixDecodeStep(kc, kc, z(*wide), z(3), z(3), z(32, dtype=torch.float64), 4, z(2), z(1))
    assert step.launches() == 4 and not step.norm
    assert step.workspace.numel() == api.shared_prefix_workspace_size(3, 1, 4, 2, 64, 16, 20000)
    assert api.SharedPrefixDecodeStep(kc, kc, z(3, 8), z(3), z(3), z(32, dtype=torch.float64), 4, z(2), z(1), 5).launches() == 3
    assert api.SharedPrefixDecodeStep(kc, kc, z(3, 8), z(3), z(3), z(32, dtype=torch.float64), 4, z(2), z(1), 0).launches() == 3
    assert api.SharedPrefixDecodeStep(kc, kc, z(3, 8), z(3), z(3), z(32, dtype=torch.float64), 4, z(2), z(1), k_weight=z(64, dtype=bf)).norm


# ---- the reference ----

def test_the_reference_is_a_softmax_over_the_gathered_rows():
    """torch's own attention in 64 bits over each sequence's rows, brought together by hand."""
    case = rows_cases.Shared("cpu", [(2, [5, -1, None]), (0, [3])], 4, 2, D=64, alone=[7])
    out, _ = case.expected()
    for s, n in enumerate(case.lens):
        if not n:
            assert (out[s] == 0).all()
            continue
        k, v = (torch.cat([c[b] for b in case.tables[s, :-(-n // 16)].tolist()], 1)[:, :n].double() for c in (case.pool.k, case.pool.v))
        q = case.q[s].double().view(2, 2, 64)
        want = torch.nn.functional.scaled_dot_product_attention(q, k, v, scale=case.scale).reshape(4, 64)
        assert np.abs(out[s] - want.numpy()).max() < 1e-12


def test_a_planted_mistake_is_past_the_bound():
    """One page of the prefix taken twice, a row's states off by one, a prefix of one page less: none is within."""
    case = rows_cases.Shared("cpu", [(6, [40, 3])], 4, 2, D=64)
    good = case.expected()
    rows_cases.within(torch.from_numpy(good[0]), good)
    case.tables[:, 1] = case.tables[:, 0]
    wrong = [case.expected()[0]]
    cross = rows_cases.Cross("cpu", [3, 2], [60, 9], 4, 2, D=64)
    want = cross.expected()
    cross.states = [59, 9]
    with pytest.raises(AssertionError):
        rows_cases.within(torch.from_numpy(cross.expected()[0]), want)
    for w in wrong:
        with pytest.raises(AssertionError):
            rows_cases.within(torch.from_numpy(w), good)
