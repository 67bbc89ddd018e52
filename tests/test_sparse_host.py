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
    (dict(k=FAR), 1), (dict(v=FAR, vs=512), 1),                     # q_out on k or v
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
    (dict(S=70000), 2), (dict(NB=1 << 27), 2), (dict(k=0), 1), (dict(mb=1 << 28), 1), (dict(mb=(1 << 17) + 1), 2), (dict(k=(1 << 17) + 1), 2), (dict(k=2 ** 31 - 1), 2),
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


# ---- the Python binding: host tensors meet every check but the device's, which comes last ----

bf = torch.bfloat16


def z(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype)


def _append_args():
    return dict(q=z(3, 4, 64, dtype=bf), k=z(3, 2, 64, dtype=bf), v=z(3, 2, 64, dtype=bf), positions=z(3),
                inv_freq=torch.ones(32, dtype=torch.float64), slot_mapping=z(3), k_cache=z(4, 2, 16, 64, dtype=bf),
                v_cache=z(4, 2, 16, 64, dtype=bf), out=z(3, 4, 64, dtype=bf))


@pytest.mark.parametrize("change,err,match", [
    (dict(q=z(3, 4, 128, dtype=bf)), ValueError, "inconsistent q and k"),
    (dict(q=z(2, 4, 64, dtype=bf)), ValueError, "inconsistent q and k"),
    (dict(q=z(3, 4, 64, dtype=torch.float32)), TypeError, "q has dtype"),
    (dict(q=[1.0]), TypeError, "q must be a torch.Tensor"),
    (dict(k=z(3, 64, 2, dtype=bf).transpose(1, 2)), ValueError, "dense"),
    (dict(k=z(3, 128, dtype=bf)), ValueError, "3 dimensions"),
    (dict(v=z(4, 2, 64, dtype=bf)), ValueError, "inconsistent K/V"),
    (dict(k=None), TypeError, "k must be a torch.Tensor"),
    (dict(positions=z(4)), ValueError, "positions"),
    (dict(positions=z(2, 3, 1)), ValueError, "positions"),
    (dict(positions=z(3, dtype=torch.int64)), TypeError, "positions"),
    (dict(positions=z(3, 2).t()), ValueError, "contiguous"),
    (dict(inv_freq=torch.ones(32)), TypeError, "inv_freq"),
    (dict(inv_freq=torch.ones(2, 16, dtype=torch.float64)), ValueError, "inv_freq"),
    (dict(pair_axis=z(31)), ValueError, "pair_axis"),
    (dict(slot_mapping=z(2)), ValueError, "slot_mapping"),
    (dict(k_scales=torch.ones(2)), ValueError, "both"),
    (dict(k_scales=torch.ones(3), v_scales=torch.ones(3)), ValueError, "k_scales"),
    (dict(out=z(3, 4, 32, dtype=bf)), ValueError, "out"),
    (dict(out=z(3, 4, 64, dtype=torch.float16)), TypeError, "out"),
    (dict(v_cache=z(4, 2, 16, 32, dtype=bf)), ValueError, "v_cache"),
    (dict(v_cache=z(4, 2, 16, 64, dtype=torch.uint8)), ValueError, "v_cache"),
    (dict(k_cache=z(4, 2, 16, 64, dtype=torch.float32)), TypeError, "k_cache"),
    (dict(k_cache=z(4, 3, 16, 64, dtype=bf), v_cache=z(4, 3, 16, 64, dtype=bf)), ValueError, "inconsistent K/V and cache"),
    (dict(magnitude="much"), TypeError, None),
    ({}, ValueError, "CUDA tensor"),
])
def test_rope_append_binding_refuses(lib, change, err, match):
    with pytest.raises(err, match=match):
        api.rope_append(**{**_append_args(), **change})


def _summary_args():
    return dict(k_cache=z(4, 2, 16, 64, dtype=bf), slot_mapping=z(3), summary=z(4, 2, 2, 64, dtype=torch.int8),
                exponents=z(4, 2, dtype=torch.int8))


@pytest.mark.parametrize("change,err,match", [
    (dict(summary=z(4, 2, 64, dtype=torch.int8)), ValueError, "summary"),
    (dict(summary=z(4, 2, 2, 64, dtype=torch.uint8)), TypeError, "summary"),
    (dict(exponents=z(4, 3, dtype=torch.int8)), ValueError, "exponents"),
    (dict(slot_mapping=z(3, 1)), ValueError, "slot_mapping"),
    (dict(k_cache=z(4, 2, 64, dtype=bf)), ValueError, "k_cache"),
    ({}, ValueError, "CUDA tensor"),
])
def test_block_summary_binding_refuses(lib, change, err, match):
    with pytest.raises(err, match=match):
        api.block_summary(**{**_summary_args(), **change})


def test_alloc_block_summary():
    s, e = api.alloc_block_summary(z(4, 2, 16, 64, dtype=bf))
    assert s.shape == (4, 2, 2, 64) and e.shape == (4, 2) and s.dtype == e.dtype == torch.int8


def _sparse_args(fn):
    a = dict(q=z(3, 4, 64, dtype=bf), block_tables=z(3, 8), context_lens=z(3), selected=z(3, 2, 4), counts=z(3, 2))
    if fn != "select":
        a.update(k_cache=z(4, 2, 16, 64, dtype=bf), v_cache=z(4, 2, 16, 64, dtype=bf), out=z(3, 4, 64, dtype=bf))
    if fn != "decode":
        a.update(summary=z(4, 2, 2, 64, dtype=torch.int8), exponents=z(4, 2, dtype=torch.int8), top_k=4)
    if fn == "select":
        a["block_size"] = 16
    return a


@pytest.mark.parametrize("fns,change,err,match", [
    ("select decode attend", dict(q=z(3, 4, 64, dtype=torch.float16)), TypeError, "q has dtype"),
    ("select decode attend", dict(q=z(3, 256, dtype=bf)), (ValueError, IndexError), None),
    ("select decode attend", dict(block_tables=z(2, 8)), ValueError, "block_tables"),
    ("select decode attend", dict(block_tables=z(3, 8, dtype=torch.int64)), TypeError, "block_tables"),
    ("select decode attend", dict(context_lens=z(2)), ValueError, "context_lens"),
    ("select decode attend", dict(counts=z(3, 1)), ValueError, "counts"),
    ("select decode attend", dict(selected=z(3, 3, 4)), ValueError, "selected"),
    ("select attend", dict(selected=z(3, 2, 5)), ValueError, "selected"),
    ("select attend", dict(summary=z(4, 2, 2, 32, dtype=torch.int8)), ValueError, "summary"),
    ("select attend", dict(exponents=z(4, 2)), TypeError, "exponents"),
    ("select attend", dict(top_k=2 ** 40), ValueError, "top_k is out of range"),
    ("select attend", dict(top_k=4.5), TypeError, None),
    ("decode attend", dict(v_scales=torch.ones(2)), ValueError, "both"),
    ("decode attend", dict(out=z(3, 2, 64, dtype=bf)), ValueError, "out"),
    ("decode attend", dict(k_cache=z(4, 2, 16, 128, dtype=bf), v_cache=z(4, 2, 16, 128, dtype=bf)), ValueError, "inconsistent"),
    ("select decode attend", {}, ValueError, "CUDA tensor"),
])
def test_sparse_binding_refuses(lib, fns, change, err, match):
    for fn in fns.split():
        with pytest.raises(err, match=match):
            getattr(api, "sparse_" + fn)(**{**_sparse_args(fn), **change})


def test_binding_fails_loudly_when_it_is_not_built(monkeypatch, tmp_path):
    from paged_kv_cache_193_gb300 import _lib
    monkeypatch.setattr(_lib, "_binding", None)
    monkeypatch.setattr(_lib, "BINDING_PATH", str(tmp_path / "missing.so"))
    with pytest.raises(ImportError, match="build"):
        _lib.binding()


@pytest.mark.parametrize("given", ["summary", "exponents"])
def test_a_step_wants_summary_and_exponents_together(given):
    """One without the other: neither may be made up beside it."""
    kc = z(4, 2, 16, 64, dtype=bf)
    both = dict(zip(("summary", "exponents"), api.alloc_block_summary(kc)))
    args = (kc, kc, z(3, 8), z(3), z(3), z(32, dtype=torch.float64), 4, 4)
    with pytest.raises(ValueError, match="summary and exponents"):
        api.SparseDecodeStep(*args, **{given: both[given]})
    step = api.SparseDecodeStep(*args, **both)
    assert step.summary is both["summary"] and step.exponents is both["exponents"]
    assert api.SparseDecodeStep(*args).summary.shape == (4, 2, 2, 64)


@pytest.mark.parametrize("fn", ["decode", "attend"])
def test_an_output_that_overlaps_the_query_is_refused(lib, fn):
    """In place is fine, a shifted overlap is not: outputs would be written over queries still to be read."""
    rows = 4 * 8 * 128 * 2  # bytes of the query of _select's call
    for off in (16, rows - 16, -16, 16 - rows):
        assert _select(lib, fn, out=ctypes.c_void_p((1 << 20) + off)) == 1
        assert b"overlap" in lib.pa_last_error()
