"""Which state / out pairs spec_beam_reorder refuses as overlapping: those that
share a byte, and no others. Without a GPU a call that passes the checks ends at
its launch; with one, interleaved parts of one allocation are moved."""
import ctypes
import random

import pytest
import torch

import plain_draft as plain
from token_verification_gb300 import _native, api, build

FAKE = 1 << 20  # never dereferenced: there is no GPU to launch on
ALIAS, CUDA = 9, 7
I5 = ctypes.c_int64 * 5

host_only = pytest.mark.skipif(torch.cuda.is_available(), reason="the calls would be launched")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _native.lib()


def code(lib, at_in, ss, n_in, at_out, os, n_out, row):
    G, B, W, H, L = n_in
    return lib.spec_beam_reorder(FAKE + at_in, I5(*ss), FAKE, None, FAKE + at_out, I5(*os), None,
                                 G, B, W, n_out[2], H, L, row, None)


def cells(at, strides, n, row):
    starts = {at}
    for s, m in zip(strides, n):
        starts = {a + s * i for a in starts for i in range(m)}
    return {a + j for a in starts for j in range(row)}


def dense(n, row, order, pad):
    """Strides of a tensor whose dimensions lie in memory in `order` (outermost first), each
    extent `pad` entries longer than used."""
    strides, step = [0] * 5, row
    for i in reversed(order):
        strides[i] = step
        step *= n[i] + pad[i]
    return strides


@host_only
def test_interleaved_parts_of_one_allocation(lib):
    n, half = (2, 3, 16, 4, 8), (2, 3, 8, 4, 8)
    for order in ((0, 1, 2, 3, 4), (0, 1, 3, 2, 4), (4, 3, 2, 1, 0)):
        s = dense(n, 32, order, [0] * 5)
        assert code(lib, 0, s, half, 8 * s[2], s, half, 32) == CUDA
        assert code(lib, 8 * s[2], s, half, 0, s, half, 32) == CUDA
        assert code(lib, 7 * s[2], s, half, 0, s, half, 32) == ALIAS
        assert code(lib, 8 * s[2] - 1, s, half, 0, s, half, 32) == ALIAS
        # every other slot
        two = list(s)
        two[2] *= 2
        assert code(lib, 0, two, half, s[2], two, half, 32) == CUDA
        assert code(lib, 0, two, half, 2 * s[2], two, half, 32) == ALIAS
    # the halves of each entry of a wider cache
    s = dense(half, 64, (0, 1, 2, 3, 4), [0] * 5)
    assert code(lib, 0, s, half, 32, s, half, 32) == CUDA
    assert code(lib, 0, s, half, 31, s, half, 32) == ALIAS


@host_only
def test_large_caches(lib):
    n = (64, 64, 8, 128, 1 << 16)
    s = dense((64, 64, 16, 128, 1 << 16), 256, (0, 1, 2, 3, 4), [0] * 5)
    assert code(lib, 0, s, n, 8 * s[2], s, n, 256) in (CUDA, 2)  # (2: more runs than a call takes)
    m = (4, 16, 8, 8, 1 << 16)
    assert code(lib, 0, s, m, 8 * s[2], s, m, 256) == CUDA
    assert code(lib, 0, s, m, 7 * s[2] + 7 * s[3], s, m, 256) == ALIAS
    assert code(lib, 0, s, m, 7 * s[2] + 8 * s[3], s, m, 256) == CUDA  # 8 of 128 heads are used


@host_only
def test_random_layouts_against_their_bytes(lib):
    r = random.Random(5)
    seen = {ALIAS: 0, CUDA: 0}
    for _ in range(4000):
        row = r.choice([1, 2, 3, 4])
        n_in = [r.randint(1, 3) for _ in range(5)]
        n_out = list(n_in)
        n_out[2] = r.randint(1, 3)
        os = dense(n_out, row, r.sample(range(5), 5), [r.choice([0, 0, 1, 2]) for _ in range(5)])
        if r.random() < 0.6:
            ss = list(os)
        else:
            ss = dense(n_in, row, r.sample(range(5), 5), [r.choice([0, 0, 1]) for _ in range(5)])
        if r.random() < 0.2:
            ss[r.randrange(5)] = 0
        at = r.randint(-200, 200)
        meet = bool(cells(at, ss, n_in, row) & cells(0, os, n_out, row))
        got = code(lib, at, ss, n_in, 0, os, n_out, row)
        assert got == (ALIAS if meet else CUDA), (at, ss, n_in, os, n_out, row)
        seen[got] += 1
    assert min(seen.values()) > 500


@pytest.mark.gpu
@pytest.mark.parametrize("order", [(0, 1, 2, 3, 4, 5), (0, 1, 3, 2, 4, 5), (0, 3, 1, 4, 2, 5)])
@pytest.mark.parametrize("with_status", [False, True])  # the compiled binding, the long way
def test_double_buffered_cache_is_moved(order, with_status):
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    shape = (2, 3, 16, 4, 9, 24)
    mem = torch.randn([shape[i] for i in order], generator=g, device="cuda")
    cache = mem.permute([order.index(i) for i in range(6)])
    p = torch.tensor([[7, 6, 5, 4, 3, 2, 1, 0], [0, 0, -1, 1, 1, 2, 2, 3], [3] * 8],
                     dtype=torch.int32, device="cuda")
    lens = torch.tensor([9, 4, 0], dtype=torch.int32, device="cuda")
    status = torch.empty(3, dtype=torch.int32, device="cuda") if with_status else None
    for state, out in ((cache[:, :, :8], cache[:, :, 8:]), (cache[:, :, 1::2], cache[:, :, ::2])):
        before = state.clone()
        want = plain.reorder(state.cpu(), p.cpu(), out.cpu(), [9, 4, 0])
        api.spec_beam_reorder(state, p, out, lens=lens, status=status)
        assert torch.equal(out.cpu(), want) and torch.equal(state, before)
    with pytest.raises(api.VerifyError):
        api.spec_beam_reorder(cache[:, :, :8], p, cache[:, :, 7:15], lens=lens, status=status)
