"""Host-side argument checks of the operators that train drafts and grow
candidate trees: the C entry points return the documented codes before any
CUDA call, the Python binding refuses tensors it cannot take (no GPU)."""
import ctypes

import pytest
import torch

from token_verification_gb300 import _native, api, build

FAKE = 0x10000  # never dereferenced: every call below fails validation first
ODD = FAKE + 1
F = ctypes.c_float
NULL, SHAPE, DTYPE, TEMPERATURE, ALIAS = 1, 2, 3, 4, 9


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _native.lib()


def top(lib, **kw):
    a = dict(logits=FAKE, k=8, T=1.0, lens=None, ids=FAKE, vals=FAKE, lse=FAKE, st=None, dtype=1,
             B=2, P=3, V=100)
    a.update(kw)
    return lib.spec_top_logits(a["logits"], a["k"], F(a["T"]), a["lens"], a["ids"], a["vals"],
                               a["lse"], a["st"], a["dtype"], a["B"], a["P"], a["V"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(k=0), SHAPE), (dict(k=129), SHAPE), (dict(P=0), SHAPE), (dict(V=0), SHAPE),
    (dict(V=(1 << 24) + 1), SHAPE), (dict(B=-1), SHAPE), (dict(B=65537), SHAPE),
    (dict(B=65536, P=1 << 20), SHAPE), (dict(dtype=2), DTYPE), (dict(T=0.0), TEMPERATURE),
    (dict(T=-1.0), TEMPERATURE), (dict(T=float("nan")), TEMPERATURE),
    (dict(T=float("inf")), TEMPERATURE), (dict(logits=None), NULL), (dict(ids=None), NULL),
    (dict(vals=None), NULL), (dict(lse=None), NULL), (dict(logits=ODD), NULL),
    (dict(logits=FAKE + 2, dtype=0), NULL), (dict(B=0, logits=None), 0)])
def test_top_logits_codes(lib, kw, code):
    assert top(lib, **kw) == code


def distill(lib, **kw):
    a = dict(s=FAKE, ids=FAKE, t=FAKE, lse=None, lens=None, g=None, T=1.0, loss=FAKE, stats=None,
             grad=None, st=None, dtype=1, B=2, P=3, V=100, k=8)
    a.update(kw)
    return lib.spec_distill(a["s"], a["ids"], a["t"], a["lse"], a["lens"], a["g"], F(a["T"]),
                            a["loss"], a["stats"], a["grad"], a["st"], a["dtype"], a["B"], a["P"],
                            a["V"], a["k"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(k=0), SHAPE), (dict(k=129), SHAPE), (dict(P=0), SHAPE), (dict(V=0), SHAPE),
    (dict(V=786433), SHAPE), (dict(V=393217, dtype=0), SHAPE), (dict(dtype=-1), DTYPE),
    (dict(T=0.0), TEMPERATURE), (dict(T=float("nan")), TEMPERATURE), (dict(s=None), NULL),
    (dict(ids=None), NULL), (dict(t=None), NULL), (dict(loss=None), NULL), (dict(s=ODD), NULL),
    (dict(stats=FAKE + 8), NULL), (dict(g=FAKE), NULL), (dict(g=FAKE, grad=ODD), NULL),
    (dict(g=FAKE, grad=FAKE + 2), ALIAS), (dict(g=FAKE, grad=FAKE + 1198), ALIAS),
    (dict(g=FAKE, grad=FAKE - 1198), ALIAS), (dict(B=0, s=None), 0)])
def test_distill_codes(lib, kw, code):
    assert distill(lib, **kw) == code


def distill_grad(lib, **kw):
    a = dict(s=FAKE, ids=FAKE, t=FAKE, stats=FAKE, g=FAKE, grad=FAKE, T=1.0, dtype=0, V=100, k=8)
    a.update(kw)
    return lib.spec_distill_grad(a["s"], a["ids"], a["t"], None, None, a["stats"], a["g"],
                                 F(a["T"]), a["grad"], a["dtype"], 2, 3, a["V"], a["k"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(stats=None), NULL), (dict(g=None), NULL), (dict(grad=None), NULL),
    (dict(grad=FAKE + 2), NULL), (dict(stats=FAKE + 4), NULL), (dict(grad=FAKE + 4), ALIAS),
    (dict(k=200), SHAPE), (dict(V=0), SHAPE), (dict(T=-2.0), TEMPERATURE), (dict(dtype=7), DTYPE)])
def test_distill_grad_codes(lib, kw, code):
    assert distill_grad(lib, **kw) == code


def beam(lib, **kw):
    a = dict(x=FAKE, sc=FAKE, tok=FAKE, par=FAKE, out=FAKE, dtype=1, B=2, W=4, V=100, n=8,
             ws=None, ws_bytes=0)
    a.update(kw)
    return lib.spec_beam_select(a["x"], a["sc"], a["tok"], a["par"], a["out"], None, a["dtype"],
                                a["B"], a["W"], a["V"], a["n"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(W=0), SHAPE), (dict(W=65), SHAPE), (dict(n=0), SHAPE), (dict(n=129), SHAPE),
    (dict(V=0), SHAPE), (dict(W=64, V=262145), SHAPE), (dict(W=8, V=2097153), SHAPE),
    (dict(dtype=9), DTYPE), (dict(x=None), NULL), (dict(sc=None), NULL), (dict(tok=None), NULL),
    (dict(par=None), NULL), (dict(out=None), NULL), (dict(x=ODD), NULL), (dict(B=0, x=None), 0)])
def test_beam_select_codes(lib, kw, code):
    assert beam(lib, **kw) == code


def test_beam_workspace(lib):
    assert lib.spec_beam_workspace_size(1, 1, 4, 32000, 8) == 0
    big = dict(B=256, W=8, V=128256, n=16)
    need = lib.spec_beam_workspace_size(1, 256, 8, 128256, 16)
    assert need >= 256 * 8 * 16 * 8
    assert beam(lib, **big) == 6
    assert beam(lib, ws=FAKE, ws_bytes=need - 1, **big) == 6
    assert beam(lib, ws=FAKE + 8, ws_bytes=need, **big) == 6
    assert lib.spec_beam_workspace_size(1, 256, 65, 128256, 16) == 0


I5 = ctypes.c_int64 * 5


def reorder(lib, state=FAKE, ss=(4096, 2048, 512, 256, 64), parents=FAKE, out=0x90000,
            os=(4096, 2048, 512, 256, 64), G=2, B=2, W=4, Wo=4, H=2, L=4, row=64):
    return lib.spec_beam_reorder(state, I5(*ss) if ss else None, parents, None, out,
                                 I5(*os) if os else None, None, G, B, W, Wo, H, L, row, None)


@pytest.mark.parametrize("kw,code", [
    (dict(G=-1), SHAPE), (dict(B=65537), SHAPE), (dict(W=65536), SHAPE), (dict(Wo=-1), SHAPE),
    (dict(row=0), SHAPE), (dict(ss=(4096, 2048, -512, 256, 64)), SHAPE),
    (dict(os=(4096, 2048, 512, -256, 64)), SHAPE), (dict(state=None), NULL),
    (dict(out=None), NULL), (dict(parents=None), NULL), (dict(ss=None), NULL),
    (dict(os=None), NULL), (dict(out=FAKE), ALIAS), (dict(out=FAKE + 8191), ALIAS),
    (dict(out=FAKE - 8191), ALIAS), (dict(os=(0, 2048, 512, 256, 64)), ALIAS),
    (dict(os=(4096, 2048, 512, 256, 32)), ALIAS), (dict(os=(1 << 61, 2048, 512, 256, 64)), SHAPE),
    (dict(B=0, ss=None), 0), (dict(L=0), 0), (dict(G=0, state=None, out=None), 0),
    (dict(Wo=0, parents=None), 0)])
def test_beam_reorder_codes(lib, kw, code):
    assert reorder(lib, **kw) == code


def test_alias_status_string(lib):
    assert b"overlap" in lib.spec_verify_status_string(ALIAS)


def test_binding_refuses_host_tensors(lib):
    x = torch.zeros(2, 3, 10)
    ids, t = torch.zeros(2, 3, 4, dtype=torch.int32), torch.zeros(2, 3, 4)
    for call in (lambda: api.spec_top_logits(x, 4), lambda: api.spec_distill(x, ids, t),
                 lambda: api.spec_beam_select(x, torch.zeros(2, 3), 4),
                 lambda: api.spec_beam_reorder(torch.zeros(1, 2, 3, 1, 1, 8),
                                               torch.zeros(2, 3, dtype=torch.int32)),
                 lambda: api.spec_top_logits(x[0], 4), lambda: api.spec_distill(x, ids[0], t),
                 lambda: api.spec_distill_grad(x, ids, t, 1.0, None, None),
                 lambda: api.spec_beam_reorder(torch.zeros(2, 3), ids[0])):
        with pytest.raises(ValueError):
            call()
