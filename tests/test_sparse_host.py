"""Host-side refusals of the rotate-and-append, block-summary, block-choice
and block-sparse decode entry points, in the C ABI and in the Python binding
(no GPU: every call fails validation before it reaches CUDA)."""
import ctypes

import pytest
import torch

from paged_kv_cache_193_gb300 import api

FAKE = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 8)
FAR = ctypes.c_void_p(1 << 30)


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_193_gb300 import build, _lib
    build.build()
    return _lib.load()


def _rope(lib, **kw):
    a = dict(q=FAKE, qs=1024, k=FAKE, ks=256, v=FAKE, vs=256, pos=FAKE, axes=1, freq=FAKE, axis=None, R=128, adj=0, mag=1.0,
             slots=FAKE, T=4, Hq=8, qo=FAR, kc=FAKE, vc=FAKE, NB=64, Hkv=2, D=128, B=16, dt=0, kvs=1.0, ksc=None, vsc=None)
    a.update(kw)
    return lib.pa_rope_append(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["pos"], a["axes"], a["freq"], a["axis"],
                              a["R"], a["adj"], a["mag"], a["slots"], a["T"], a["Hq"], a["qo"], a["kc"], a["vc"], a["NB"],
                              a["Hkv"], a["D"], a["B"], a["dt"], a["kvs"], a["ksc"], a["vsc"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(Hq=-1), 1), (dict(Hkv=0), 1), (dict(NB=0), 1),
    (dict(D=96), 2), (dict(B=8), 2), (dict(dt=5), 2),
    (dict(R=0), 1), (dict(R=144), 1), (dict(R=24), 2),
    (dict(axes=0), 1), (dict(axes=17, axis=FAKE), 2), (dict(axes=3), 1),
    (dict(mag=0.0), 1), (dict(mag=float("nan")), 1), (dict(mag=float("inf")), 1),
    (dict(ksc=FAKE), 1), (dict(ksc=FAKE, vsc=FAKE), 1), (dict(dt=1, kvs=0.0), 1), (dict(dt=1, kvs=float("inf")), 1),
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(pos=None), 1), (dict(freq=None), 1), (dict(slots=None), 1),
    (dict(qo=None), 1), (dict(kc=None), 1), (dict(vc=None), 1),
    (dict(q=ODD), 1), (dict(k=ODD), 1), (dict(vc=ODD), 1), (dict(qo=ODD), 1),
    (dict(qs=1020), 1), (dict(ks=260), 1), (dict(vs=248), 1), (dict(qs=1016), 1),
    (dict(qo=FAKE, qs=1536), 1),                                    # strided q cannot be its own output
    (dict(qo=ctypes.c_void_p((1 << 20) + 4096)), 1),                # q_out inside q
    (dict(NB=1 << 28), 2),
])
def test_rope_append_rejects_on_host(lib, kw, status):
    assert _rope(lib, **kw) == status
    assert lib.pa_last_error()


def test_rope_append_of_nothing_is_a_no_op(lib):
    assert _rope(lib, T=0, q=None, k=None, v=None) == 0


def _summary(lib, **kw):
    a = dict(kc=FAKE, slots=FAKE, T=4, NB=64, Hkv=2, D=128, B=16, dt=0, s=FAKE, e=FAKE)
    a.update(kw)
    return lib.pa_block_summary(a["kc"], a["slots"], a["T"], a["NB"], a["Hkv"], a["D"], a["B"], a["dt"], a["s"], a["e"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(NB=0), 1), (dict(Hkv=0), 1), (dict(D=32), 2), (dict(B=64), 2), (dict(dt=2), 2), (dict(kc=None), 1),
    (dict(slots=None), 1), (dict(s=None), 1), (dict(e=None), 1), (dict(kc=ODD), 1), (dict(s=ODD), 1), (dict(NB=1 << 28), 2),
])
def test_block_summary_rejects_on_host(lib, kw, status):
    assert _summary(lib, **kw) == status
    assert lib.pa_last_error()


def _select(lib, fn="select", **kw):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, s=FAKE, e=FAKE, bt=FAKE, mb=64, cl=FAKE, S=4, Hq=8, Hkv=2, D=128, NB=64, B=16, dt=0,
             kvs=1.0, ksc=None, vsc=None, sm=0.088, k=16, sink=1, recent=2, sel=FAKE, cnt=FAKE, split=0, out=FAKE)
    a.update(kw)
    if fn == "select":
        return lib.pa_sparse_select(a["q"], a["s"], a["e"], a["bt"], a["mb"], a["cl"], a["S"], a["Hq"], a["Hkv"], a["D"],
                                    a["NB"], a["B"], a["k"], a["sink"], a["recent"], a["sel"], a["cnt"], None)
    head = (a["bt"], a["mb"], a["cl"], a["S"], a["Hq"], a["Hkv"], a["D"], a["NB"], a["B"], a["dt"], a["kvs"], a["ksc"], a["vsc"],
            a["sm"])
    if fn == "decode":
        return lib.pa_sparse_decode(a["q"], a["kc"], a["vc"], *head, a["sel"], a["cnt"], a["k"], a["split"], a["out"], None)
    return lib.pa_sparse_attend(a["q"], a["kc"], a["vc"], a["s"], a["e"], *head, a["k"], a["sink"], a["recent"], a["sel"],
                                a["cnt"], a["out"], None)


@pytest.mark.parametrize("fn", ["select", "decode", "attend"])
@pytest.mark.parametrize("kw,status", [
    (dict(S=-1), 1), (dict(Hkv=3), 1), (dict(Hq=64, Hkv=2), 2), (dict(D=96), 2), (dict(B=8), 2), (dict(NB=0), 1), (dict(mb=0), 1),
    (dict(S=70000), 2), (dict(NB=1 << 27), 2), (dict(k=0), 1), (dict(mb=1 << 28), 1), (dict(mb=(1 << 18) + 1), 2),
    (dict(q=None), 1), (dict(bt=None), 1), (dict(cl=None), 1), (dict(sel=None), 1), (dict(cnt=None), 1), (dict(q=ODD), 1),
])
def test_sparse_entry_points_reject_on_host(lib, fn, kw, status):
    assert _select(lib, fn, **kw) == status
    assert lib.pa_last_error()


@pytest.mark.parametrize("fn", ["select", "attend"])
@pytest.mark.parametrize("kw", [dict(sink=-1), dict(recent=0), dict(k=2), dict(sink=15, recent=2), dict(sink=2 ** 31 - 1, recent=2),
                                dict(s=None), dict(e=None), dict(s=ODD)])
def test_choice_rejects_on_host(lib, fn, kw):
    assert _select(lib, fn, **kw) == 1


@pytest.mark.parametrize("fn", ["decode", "attend"])
@pytest.mark.parametrize("kw,status", [
    (dict(dt=3), 2), (dict(sm=0.0), 1), (dict(sm=-1.0), 1), (dict(sm=float("nan")), 1), (dict(ksc=FAKE), 1),
    (dict(ksc=FAKE, vsc=FAKE), 1), (dict(dt=1, kvs=-1.0), 1), (dict(kc=None), 1), (dict(vc=ODD), 1), (dict(out=None), 1),
    (dict(out=ODD), 1),
])
def test_attention_rejects_on_host(lib, fn, kw, status):
    assert _select(lib, fn, **kw) == status


@pytest.mark.parametrize("split", [-1, 3, 16])
def test_splits_are_checked(lib, split):
    assert _select(lib, "decode", split=split) == 1


@pytest.mark.parametrize("fn", ["select", "decode", "attend"])
def test_no_rows_is_a_no_op(lib, fn):
    assert _select(lib, fn, S=0, q=None, sel=None, out=None) == 0


# ---- the Python binding --------------------------------------------------------

@pytest.fixture
def on_gpu(monkeypatch, lib):
    """Host tensors that say they are on cuda:0, to reach the checks behind the device's."""
    monkeypatch.setattr(torch.Tensor, "device", property(lambda self: torch.device("cuda", 0)))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)


def _args(T=3, Hq=4, Hkv=2, D=64, NB=4, B=16):
    bf = torch.bfloat16
    cache = torch.zeros(NB, Hkv, B, D, dtype=bf)
    return dict(q=torch.zeros(T, Hq, D, dtype=bf), k=torch.zeros(T, Hkv, D, dtype=bf), v=torch.zeros(T, Hkv, D, dtype=bf),
                positions=torch.zeros(T, dtype=torch.int32), inv_freq=torch.ones(D // 2, dtype=torch.float64),
                slot_mapping=torch.zeros(T, dtype=torch.int32), k_cache=cache, v_cache=cache.clone(),
                out=torch.zeros(T, Hq, D, dtype=bf))


@pytest.mark.parametrize("change,err,match", [
    (dict(q=torch.zeros(3, 4, 128, dtype=torch.bfloat16)), ValueError, "inconsistent q and k"),
    (dict(q=torch.zeros(3, 4, 64)), TypeError, "bfloat16"),
    (dict(k=torch.zeros(3, 64, 2, dtype=torch.bfloat16).transpose(1, 2)), ValueError, "dense"),
    (dict(v=torch.zeros(4, 2, 64, dtype=torch.bfloat16)), ValueError, "inconsistent K/V"),
    (dict(positions=torch.zeros(4, dtype=torch.int32)), ValueError, "positions"),
    (dict(positions=torch.zeros(3, dtype=torch.int64)), TypeError, "positions"),
    (dict(inv_freq=torch.ones(32)), TypeError, "inv_freq"),
    (dict(pair_axis=torch.zeros(31, dtype=torch.int32)), ValueError, "pair_axis"),
    (dict(slot_mapping=torch.zeros(2, dtype=torch.int32)), ValueError, "slot_mapping"),
    (dict(k_scales=torch.ones(2)), ValueError, "both"),
    (dict(out=torch.zeros(3, 4, 32, dtype=torch.bfloat16)), ValueError, "out"),
    (dict(v_cache=torch.zeros(4, 2, 16, 32, dtype=torch.bfloat16)), ValueError, "v_cache"),
])
def test_rope_append_binding_refuses(on_gpu, change, err, match):
    with pytest.raises(err, match=match):
        api.rope_append(**{**_args(), **change})


def test_rope_append_binding_refuses_a_library_error(on_gpu):
    a = _args()
    a["inv_freq"] = torch.ones(12, dtype=torch.float64)  # 24 elements: not a multiple of 16
    with pytest.raises(api.PagedAttentionError, match="multiple of 16"):
        api.rope_append(**a, stream=type("S", (), {"cuda_stream": 0}))


def test_tensors_of_another_device_are_refused(on_gpu, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        api.rope_append(**_args())
    with pytest.raises(ValueError, match="current device"):
        api.block_summary(_args()["k_cache"], torch.zeros(3, dtype=torch.int32), torch.zeros(4, 2, 2, 64, dtype=torch.int8),
                          torch.zeros(4, 2, dtype=torch.int8))


def test_host_tensors_are_refused(lib):
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.rope_append(**_args())
    a = _args()
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.block_summary(a["k_cache"], a["slot_mapping"], *api.alloc_block_summary(a["k_cache"]))


@pytest.mark.parametrize("change,match", [
    (dict(summary=torch.zeros(4, 2, 2, 32, dtype=torch.int8)), "summary"),
    (dict(exponents=torch.zeros(4, 3, dtype=torch.int8)), "exponents"),
    (dict(context_lens=torch.zeros(2, dtype=torch.int32)), "context_lens"),
    (dict(block_tables=torch.zeros(2, 8, dtype=torch.int32)), "block_tables"),
    (dict(selected=torch.zeros(3, 2, 5, dtype=torch.int32)), "selected"),
    (dict(counts=torch.zeros(3, 1, dtype=torch.int32)), "counts"),
    (dict(v_scales=torch.ones(2)), "both"),
    (dict(out=torch.zeros(3, 2, 64, dtype=torch.bfloat16)), "out"),
])
def test_sparse_attend_binding_refuses(on_gpu, change, match):
    a = _args()
    args = dict(q=a["q"], k_cache=a["k_cache"], v_cache=a["v_cache"], summary=torch.zeros(4, 2, 2, 64, dtype=torch.int8),
                exponents=torch.zeros(4, 2, dtype=torch.int8), block_tables=torch.zeros(3, 8, dtype=torch.int32),
                context_lens=torch.ones(3, dtype=torch.int32), top_k=4, selected=torch.zeros(3, 2, 4, dtype=torch.int32),
                counts=torch.zeros(3, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match=match):
        api.sparse_attend(**{**args, **change})
