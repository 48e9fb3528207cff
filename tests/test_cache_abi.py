"""Host-side argument checks of the 4-bit cache's operators: the C entry points
return the documented codes before any CUDA call, the Python functions
refuse tensors they cannot take (no GPU)."""
import ctypes
import math

import pytest
import torch

from token_verification_gb300 import _native, api, build

FAKE = 0x100000  # never dereferenced: every call below fails validation first
F = ctypes.c_float
NULL, SHAPE, DTYPE, TREE, ALIAS, SCORE = 1, 2, 3, 5, 9, 10
ROW = 128 * 2


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _native.lib()


def strides(*x):
    return (ctypes.c_int64 * 3)(*x) if x[0] is not None else None


def dense(**kw):
    a = dict(cache=FAKE, stride=1 << 20, k=FAKE, ks=(32 * ROW, 8 * ROW, ROW), v=FAKE,
             vs=(32 * ROW, 8 * ROW, ROW), table=FAKE, start=FAKE, lens=None, fill=0, st=None,
             dtype=1, pages=9, page=64, B=2, N=4, M=3, H=8, D=128)
    a.update(kw)
    return a


def write(lib, **kw):
    a = dense(**kw)
    return lib.spec_cache_write(a["cache"], a["stride"], a["k"], strides(*a["ks"]), a["v"],
                                strides(*a["vs"]), a["table"], a["start"], a["lens"], a["st"],
                                a["dtype"], a["pages"], a["page"], a["B"], a["N"], a["M"], a["H"],
                                a["D"], None)


def read(lib, **kw):
    a = dense(**kw)
    return lib.spec_cache_read(a["cache"], a["stride"], a["k"], strides(*a["ks"]), a["v"],
                               strides(*a["vs"]), a["table"], a["start"], a["lens"], a["fill"],
                               a["st"], a["dtype"], a["pages"], a["page"], a["B"], a["N"], a["M"],
                               a["H"], a["D"], None)


def keep(lib, **kw):
    a = dict(cache=FAKE, stride=1 << 20, table=FAKE, start=FAKE, path=FAKE, st=None, pages=9,
             page=64, B=2, P=4, M=3, H=8, D=128)
    a.update(kw)
    return lib.spec_cache_keep(a["cache"], a["stride"], a["table"], a["start"], a["path"], a["st"],
                               a["pages"], a["page"], a["B"], a["P"], a["M"], a["H"], a["D"], None)


def attend(lib, **kw):
    a = dict(q=4 * FAKE, qs=(128 * ROW, 32 * ROW, ROW), cache=FAKE, stride=1 << 20, table=FAKE,
             lens=FAKE, q_lens=None, parent=None, ps=0, slopes=None, scale=0.1, cap=0.0, window=0,
             out=FAKE, lse=None, st=None, dtype=1, pages=9, page=64, B=2, N=4, M=3, Hq=32, H=8,
             D=128)
    a.update(kw)
    return lib.spec_cache_attention(
        a["q"], strides(*a["qs"]), a["cache"], a["stride"], a["table"], a["lens"], a["q_lens"],
        a["parent"], a["ps"], a["slopes"], F(a["scale"]), F(a["cap"]), a["window"], a["out"],
        a["lse"], a["st"], a["dtype"], a["pages"], a["page"], a["B"], a["N"], a["M"], a["Hq"],
        a["H"], a["D"], None, 0, None)


CACHE = [  # (what every entry point refuses of a cache and its table)
    (dict(page=8), SHAPE), (dict(page=48), SHAPE), (dict(page=512), SHAPE), (dict(page=-16), SHAPE),
    (dict(D=32), SHAPE), (dict(D=96), SHAPE), (dict(D=512), SHAPE), (dict(D=0), SHAPE),
    (dict(pages=-1), SHAPE), (dict(B=-1), SHAPE), (dict(B=65537), SHAPE), (dict(M=-1), SHAPE),
    (dict(M=(1 << 21) + 1), SHAPE), (dict(stride=8), SHAPE), (dict(stride=(1 << 20) + 8), SHAPE),
    (dict(stride=-(1 << 20)), SHAPE), (dict(stride=1 << 32), SHAPE),
    (dict(stride=64 * 68 * 16 - 16), SHAPE),  # (a page of 8 heads: 64 * 68 * 2 * 8 bytes)
    (dict(cache=None), NULL), (dict(cache=FAKE + 8), NULL), (dict(table=None), NULL),
    (dict(start=None, lens=None), NULL), (dict(B=0, cache=None, table=None), 0)]


@pytest.mark.parametrize("kw,code", CACHE)
def test_cache_codes(lib, kw, code):
    assert write(lib, **kw) == code
    assert keep(lib, **kw) == code
    if "start" not in kw:
        assert read(lib, **kw) == code
    a = {k: v for k, v in kw.items() if k != "start"}
    assert attend(lib, **a) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), DTYPE), (dict(dtype=-1), DTYPE), (dict(N=-1), SHAPE), (dict(H=0), SHAPE),
    (dict(H=1025), SHAPE), (dict(B=65536, N=1 << 12), SHAPE), (dict(k=None), NULL),
    (dict(v=None), NULL), (dict(k=FAKE + 8), NULL), (dict(v=FAKE + 2), NULL),
    (dict(ks=(None,)), NULL), (dict(vs=(None,)), NULL), (dict(ks=(32 * ROW, 8 * ROW + 8, ROW)), NULL),
    (dict(vs=(32 * ROW, 8 * ROW, ROW + 2)), NULL), (dict(ks=(-32 * ROW, 8 * ROW, ROW)), SHAPE),
    (dict(vs=(1 << 61, 8 * ROW, ROW)), SHAPE)])
def test_dense_codes(lib, kw, code):
    assert write(lib, **kw) == code
    assert read(lib, **kw) == code


@pytest.mark.parametrize("ks", [(0, 8 * ROW, ROW), (32 * ROW, 0, ROW), (32 * ROW, 8 * ROW, 0),
                                (32 * ROW, 8 * ROW, ROW - 16), (32 * ROW - 16, 8 * ROW, ROW),
                                (ROW, 2 * ROW, 4 * ROW)])
def test_read_refuses_rows_that_overlap(lib, ks):
    assert read(lib, ks=ks) == ALIAS
    assert read(lib, vs=ks) == ALIAS


@pytest.mark.parametrize("kw,code", [(dict(P=-1), SHAPE), (dict(P=258), SHAPE), (dict(path=None), NULL),
                                     (dict(H=0), SHAPE)])
def test_keep_codes(lib, kw, code):
    assert keep(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), DTYPE), (dict(N=-1), SHAPE), (dict(N=258), SHAPE), (dict(Hq=0), SHAPE),
    (dict(Hq=30), SHAPE), (dict(Hq=1032), SHAPE), (dict(H=0), SHAPE), (dict(H=64), SHAPE),
    (dict(scale=math.nan), SCORE), (dict(scale=math.inf), SCORE), (dict(cap=-1.0), SCORE),
    (dict(cap=math.nan), SCORE), (dict(cap=math.inf), SCORE), (dict(cap=2e30), SCORE), (dict(window=-1), SCORE),
    (dict(parent=FAKE, ps=4), TREE), (dict(parent=FAKE, ps=-1), TREE), (dict(q=None), NULL),
    (dict(lens=None), NULL), (dict(out=None), NULL), (dict(qs=(None,)), NULL),
    (dict(q=4 * FAKE + 8), NULL), (dict(out=FAKE + 8), NULL), (dict(qs=(128 * ROW, 32 * ROW, 8)), NULL),
    (dict(qs=(-16, 32 * ROW, ROW)), SHAPE), (dict(qs=(1 << 61, 32 * ROW, ROW)), SHAPE),
    (dict(q=FAKE, out=FAKE + 16), ALIAS), (dict(q=FAKE + 2 * 4 * 32 * ROW - 16, out=FAKE), ALIAS),
    (dict(q=FAKE, out=FAKE + 7 * 32 * ROW + 31 * ROW), ALIAS), (dict(q=FAKE, out=FAKE), ALIAS),
    (dict(N=0, q=None), 0)])
def test_attention_codes(lib, kw, code):
    assert attend(lib, **kw) == code


def test_page_bytes_and_workspace(lib):
    for page in (16, 32, 64, 128, 256):
        for D in (64, 128, 256):
            assert lib.spec_cache_page_bytes(page, D) == page * (D // 2 + D // 32)
    for page, D in ((0, 64), (24, 64), (512, 64), (-16, 64), (64, 0), (64, 72), (64, 512)):
        assert lib.spec_cache_page_bytes(page, D) == 0
    for args in ((2, 1, 8, 8, 128), (1, -1, 8, 8, 128), (1, 258, 8, 8, 128), (1, 1, 9, 8, 128),
                 (1, 1, 8, 0, 128), (1, 1, 8, 8, 100)):
        assert lib.spec_cache_attention_workspace_size(*args) == 0


def test_python_refuses_what_it_cannot_take():
    cache = torch.zeros((3, 2, 2, 16 * 34), dtype=torch.uint8)
    table, start = torch.zeros((2, 1), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    k = torch.zeros((2, 1, 2, 64))
    path = torch.zeros((2, 1), dtype=torch.int32)
    for c in (cache, cache[0], None):  # (on the host; no cache)
        for call in (lambda: api.spec_cache_write(c, k, k, table, start),
                     lambda: api.spec_cache_read(c, table, 1, 64),
                     lambda: api.spec_cache_keep(c, table, start, path, 64),
                     lambda: api.spec_cache_attention(k, c, table, start)):
            with pytest.raises(ValueError):
                call()
    for k in (None, torch.zeros((2, 2, 64))):
        with pytest.raises(ValueError):
            api.spec_cache_write(cache, k, k, table, start)
        with pytest.raises(ValueError):
            api.spec_cache_attention(k, cache, table, start)
    for page, D in ((20, 64), (16, 96)):
        with pytest.raises(ValueError):
            api.spec_cache_alloc(1, 1, D, page, device="cpu")
    assert api.spec_cache_alloc(3, 2, 64, 16, device="cpu").shape == cache.shape
