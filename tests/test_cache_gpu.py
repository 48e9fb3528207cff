"""spec_cache_write, spec_cache_read and spec_cache_keep against the plain forms
(tests/plain_cache.py): every code and scale byte, and what is left alone (needs a
GPU)."""
import math

import pytest
import torch

import plain_cache as plain
from token_verification_gb300 import api

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def pages_for(B, slots, page, g, spare=2):
    """(table [B, M], pages): every page its own, in no order."""
    M = -(-slots // page)
    n = B * M + spare
    ids = torch.randperm(n, generator=g, device="cuda")[:B * M]
    return ids.int().view(B, M).contiguous(), n


def spread(shape, dtype, g):
    """Values over many magnitudes, group by group."""
    x = torch.randn(shape, generator=g, device="cuda")
    e = torch.randint(-24, 14, shape[:-1] + (shape[-1] // 32, 1), generator=g, device="cuda")
    return (x.unflatten(-1, (-1, 32)) * torch.exp2(e.float())).flatten(-2).to(dtype)


def expected(cache, k, v, table, start, lens, page):
    """The cache's bytes after a write, token by token from the definition."""
    want = cache.cpu().clone()
    B, N, H, D = k.shape
    codes = want[..., :page * D // 2].unflatten(-1, (page, D // 2))
    scales = want[..., page * D // 2:].unflatten(-1, (page // 16, D // 32, 16))
    bad = ~(torch.isfinite(k).all(-1) & torch.isfinite(v).all(-1)).cpu()
    for part, x in enumerate((k, v)):
        x = torch.where(bad[..., None], 0.0, x.cpu().double())
        q, byte, _ = plain.quantise(x)
        if part == 0:
            byte[bad] = 247
        w = (q + 8).unflatten(-1, (-1, 8))
        word = torch.zeros(w.shape[:-1], dtype=torch.int64)
        for i in range(8):
            word |= w[..., i].long() << (4 * (i // 2 + 4 * (i % 2)))
        packed = torch.stack([(word >> (8 * j)) & 255 for j in range(4)], -1).flatten(-2)
        for b in range(B):
            for i in range(N if lens is None else lens[b]):
                slot = start[b] + i
                p, t = int(table[b, slot // page]), slot % page
                codes[p, :, part, t] = packed[b, i].to(torch.uint8)
                scales[p, :, part, t // 16, :, t % 16] = byte[b, i].to(torch.uint8)
    return want


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,N,H,D,page,start,lens", [
    (1, 1, 1, 64, 16, [0], None), (1, 1, 3, 128, 64, [63], None), (2, 6, 8, 128, 64, [60, 7], None),
    (3, 40, 2, 64, 16, [0, 15, 33], [40, 0, 17]), (2, 33, 5, 256, 32, [31, 0], [33, 1]),
    (4, 300, 1, 128, 256, [5, 0, 255, 100], [300, 299, 1, 0])])
def test_write_and_read(B, N, H, D, page, start, lens, dtype):
    g = gen(B * N + H)
    table, n = pages_for(B, max(start) + N, page, g)
    cache = torch.randint(0, 256, (n, H, 2, page * (D // 2 + D // 32)), generator=g, device="cuda",
                          dtype=torch.uint8)
    before = cache.clone()
    k, v = spread((B, N, H, D), dtype, g), spread((B, N, H, D), dtype, g)
    status = torch.full((B,), 77, dtype=torch.int32, device="cuda")
    l = None if lens is None else ints(lens)
    assert api.spec_cache_write(cache, k, v, table, ints(start), lens=l, status=status) is cache
    assert torch.equal(cache.cpu(), expected(before, k, v, table, start, lens, page))
    assert not bool(status.any())
    for t in (BF16, F32):
        gk, gv = api.spec_cache_read(cache, table, N, D, start=ints(start), lens=l, dtype=t)
        for got, x in ((gk, k), (gv, v)):
            want = plain.quantise(x)[2]
            if lens is not None:
                for b in range(B):
                    want[b, lens[b]:] = 0
            assert got.dtype == t and torch.equal(got.cpu().double(), want)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_ties_and_borders(dtype):
    """Every scale byte against every half and its neighbours, magnitudes at 7 s and beside it,
    signed zeros, subnormals, values above the largest scale."""
    rows = []
    for byte in range(0, plain.TOP + 1):
        s = float(plain.SCALES[byte])
        top = torch.full((32,), 7 * s)
        x = torch.tensor([(h + 0.5) * s for h in range(-7, 7)] + [h * s for h in range(-7, 8)] + [7 * s] * 3)
        rows.append(x)
        top[1:] = 0.0
        rows.append(top)
        rows.append(torch.cat([torch.tensor([7 * s * (1 + 2.0 ** -7), 7 * s * (1 - 2.0 ** -8)]),
                               torch.tensor([0.5 * s * (1 + e * 2.0 ** -7) for e in range(-15, 15)])]))
        if dtype == F32:
            rows.append(torch.nextafter(x, torch.tensor(math.inf)))
            rows.append(torch.nextafter(x, torch.tensor(-math.inf)))
            t = torch.tensor([7 * s])
            rows.append(torch.nextafter(t, torch.tensor(math.inf)).expand(32))
            rows.append(torch.nextafter(t, torch.tensor(0.0)).expand(32))
    rows += [torch.zeros(32), torch.full((32,), -0.0), torch.full((32,), 1e-40),
             torch.full((32,), 6272.0), torch.full((32,), -1e30), torch.linspace(-9000, 9000, 32)]
    while len(rows) % 4:
        rows.append(torch.zeros(32))
    x = torch.stack(rows).view(1, -1, 1, 128).to(dtype).cuda()
    N = x.shape[1]
    table, n = pages_for(1, N, 64, gen(1))
    cache = api.spec_cache_alloc(n, 1, 128, 64)
    api.spec_cache_write(cache, x, -x, table, ints([0]))
    want = expected(torch.zeros_like(cache), x, -x, table, [0], None, 64)
    assert torch.equal(cache.cpu(), want)


def test_every_bf16_number():
    """All finite bf16 values, each against each scale of its group's top."""
    bits = torch.arange(0, 0x7f80, dtype=torch.int32)
    x = bits.to(torch.int16).view(BF16)
    big = x.float()
    tops = [x, (big * 1.09375).to(BF16), (big * 2.7).to(BF16), (big * 6.9).to(BF16),
            (big * 13.2).to(BF16)]
    tops = [torch.where(torch.isfinite(t), t, x) for t in tops]
    rows = torch.stack([torch.stack([x, t], -1) for t in tops], 0).flatten(0, 1)  # [n, 2]
    rows = rows.repeat_interleave(16, dim=1)
    pad = (-rows.shape[0]) % 8
    rows = torch.cat([rows, rows[:pad]])
    k = rows.view(1, -1, 1, 256).cuda()
    table, n = pages_for(1, k.shape[1], 128, gen(2))
    cache = api.spec_cache_alloc(n, 1, 256, 128)
    api.spec_cache_write(cache, k, k, table, ints([0]))
    gk, gv = api.spec_cache_read(cache, table, k.shape[1], 256)
    want = plain.quantise(k)[2]
    assert torch.equal(gk.cpu().double(), want) and torch.equal(gv.cpu().double(), want)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_not_finite(bad):
    """A head of a token with NaN or infinity is NaN in keys and values; its neighbours hold."""
    g = gen(3)
    for D in (64, 128, 256):
        k = torch.randn((2, 5, 3, D), generator=g, device="cuda").to(BF16)
        v = torch.randn((2, 5, 3, D), generator=g, device="cuda").to(BF16)
        k[0, 1, 2, D - 1] = bad
        v[1, 4, 0, 0] = bad
        table, n = pages_for(2, 5, 16, g)
        cache = api.spec_cache_alloc(n, 3, D, 16)
        api.spec_cache_write(cache, k, v, table, ints([0, 0]))
        gk, gv = api.spec_cache_read(cache, table, 5, D)
        wk, wv = plain.held(k, v)
        assert torch.equal(torch.isnan(gk).cpu(), torch.isnan(wk)) and int(torch.isnan(wk).sum()) == 2 * D
        assert torch.equal(gk.cpu().double().nan_to_num(0), wk.nan_to_num(0))
        assert torch.equal(gv.cpu().double().nan_to_num(7), wv.nan_to_num(7))


def test_strided_parts_and_layers():
    """Keys and values as parts of a fused projection, heads before tokens, and a cache whose pages
    interleave the layers of a model; a read into parts of a larger tensor."""
    g = gen(4)
    B, N, H, D, page, layers = 2, 21, 2, 128, 16, 3
    table, n = pages_for(B, 40, page, g)
    pool = torch.randint(0, 256, (n, layers, H, 2, page * (D // 2 + D // 32)), generator=g,
                         device="cuda", dtype=torch.uint8)
    before = pool.clone()
    qkv = torch.randn((B, N, 4 + 2 * H, D), generator=g, device="cuda").to(BF16)
    k, v = qkv[:, :, 4:4 + H], qkv[:, :, 4 + H:]
    api.spec_cache_write(pool[:, 1], k, v, table, ints([3, 19]))
    want = expected(before[:, 1], k, v, table, [3, 19], None, page)
    assert torch.equal(pool[:, 1].cpu(), want)
    assert torch.equal(pool[:, 0], before[:, 0]) and torch.equal(pool[:, 2], before[:, 2])
    heads_first = torch.randn((2, B, H, N, D), generator=g, device="cuda")
    k2, v2 = heads_first[0].transpose(1, 2), heads_first[1].transpose(1, 2)
    api.spec_cache_write(pool[:, 2], k2, v2, table, ints([0, 1]))
    assert torch.equal(pool[:, 2].cpu(), expected(before[:, 2], k2, v2, table, [0, 1], None, page))
    out = torch.full((2, B, H, N, D), 9.0, device="cuda")
    api.spec_cache_read(pool[:, 2], table, N, D, out[0].transpose(1, 2), out[1].transpose(1, 2),
                        start=ints([0, 1]), lens=ints([N, 4]))
    for part, x in ((0, k2), (1, v2)):
        want = plain.quantise(x)[2].float()
        got = out[part].transpose(1, 2).cpu()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1, :4], want[1, :4])
        assert bool((got[1, 4:] == 9).all())


def test_data_errors():
    """Lengths, starts and pages out of range: a status, nothing of theirs written, the others'
    tokens in place."""
    g = gen(5)
    B, N, H, D, page = 6, 20, 2, 64, 16
    table, n = pages_for(B, 64, page, g)
    start, lens = [0, 60, -1, 5, 0, 3], [20, 20, 3, 21, -1, 20]
    table[5, 1] = n
    table[0, 3] = -5  # not touched: no error
    cache = torch.randint(0, 256, (n, H, 2, page * 34), generator=g, device="cuda", dtype=torch.uint8)
    before = cache.clone()
    k = torch.randn((B, N, H, D), generator=g, device="cuda").to(BF16)
    status = torch.zeros(B, dtype=torch.int32, device="cuda")
    api.spec_cache_write(cache, k, k, table, ints(start), lens=ints(lens), status=status)
    assert status.tolist() == [0, 4, 4, 4, 4, 32]
    want = expected(before, k[[0]], k[[0]], table[[0]], [0], [20], page)
    want = expected(want, k[[5]], k[[5]], table[[5]], [3], [13], page)  # up to the page that is none
    assert torch.equal(cache.cpu(), want)
    out = torch.full((2, B, N, H, D), 5.0, device="cuda")
    status.zero_()
    api.spec_cache_read(cache, table, N, D, out[0], out[1], start=ints(start), lens=ints(lens),
                        status=status)
    assert status.tolist() == [0, 4, 4, 4, 4, 32]
    assert bool((out[:, 1:5] == 5).all()) and bool((out[:, 5, 13:] == 5).all())
    assert torch.equal(out[0, 5, :13].cpu().double(), plain.quantise(k[5, :13])[2])


def paths(B, N, P, g):
    """Ascending paths from the root on, -1 after; some empty, some in place."""
    out = torch.full((B, P), -1, dtype=torch.int32)
    for b in range(B):
        n = int(torch.randint(0, P + 1, (1,), generator=g, device="cuda"))
        if n == 0:
            continue
        rest = torch.randperm(N - 1, generator=g, device="cuda")[:n - 1].cpu() + 1
        out[b, :len(rest) + 1] = torch.cat([torch.zeros(1, dtype=torch.int64), rest.sort().values]).int()
    return out


@pytest.mark.parametrize("B,N,P,H,D,page", [
    (1, 2, 2, 1, 64, 16), (5, 61, 6, 8, 128, 64), (9, 257, 30, 3, 128, 16), (4, 30, 30, 2, 256, 32),
    (300, 12, 5, 1, 64, 256)])
def test_keep(B, N, P, H, D, page):
    g = gen(B + N)
    table, n = pages_for(B, 300 + N, page, g)
    cache = torch.randint(0, 256, (n, H, 2, page * (D // 2 + D // 32)), generator=g, device="cuda",
                          dtype=torch.uint8)
    start = torch.randint(0, 300, (B,), generator=g, device="cuda").int()
    path = paths(B, N, P, g)
    want = cache.cpu().clone()
    codes = want[..., :page * D // 2].unflatten(-1, (page, D // 2))
    scales = want[..., page * D // 2:].unflatten(-1, (page // 16, D // 32, 16))
    old_c, old_s = codes.clone(), scales.clone()
    for b in range(B):
        for i, x in enumerate(path[b].tolist()):
            if x < 0:
                break
            s, d = int(start[b]) + x, int(start[b]) + i
            ps, pd = int(table[b, s // page]), int(table[b, d // page])
            s, d = s % page, d % page
            codes[pd, :, :, d] = old_c[ps, :, :, s]
            scales[pd, :, :, d // 16, :, d % 16] = old_s[ps, :, :, s // 16, :, s % 16]
    status = torch.full((B,), 9, dtype=torch.int32, device="cuda")
    assert api.spec_cache_keep(cache, table, start, path.cuda(), D, status=status) is cache
    assert torch.equal(cache.cpu(), want) and not bool(status.any())


def test_keep_errors():
    g = gen(6)
    page, D = 16, 64
    table, n = pages_for(7, 64, page, g)
    table[6, 2] = -1
    cache = torch.randint(0, 256, (n, 2, 2, page * 34), generator=g, device="cuda", dtype=torch.uint8)
    before = cache.clone()
    path = ints([[0, 3, 2], [0, 0, 1], [-2, 1, 2], [0, 5, 64], [0, 5, 9], [2, 3, 5], [0, 1, 40]])
    start = ints([0, 0, 0, 0, -3, 56, 0])
    status = torch.zeros(7, dtype=torch.int32, device="cuda")
    api.spec_cache_keep(cache, table, start, path, D, status=status)
    assert status.tolist() == [16, 16, 16, 4, 4, 0, 32]
    own = set(table[5].tolist())
    rest = torch.tensor([i for i in range(n) if i not in own], device="cuda")
    assert torch.equal(cache[rest], before[rest])
    assert not torch.equal(cache, before)


def test_nothing_to_do():
    cache = api.spec_cache_alloc(0, 2, 64, 16)
    none = torch.empty((0, 3), dtype=torch.int32, device="cuda")
    zero = torch.empty((0,), dtype=torch.int32, device="cuda")
    k = torch.empty((0, 4, 2, 64), device="cuda")
    api.spec_cache_write(cache, k, k, none, zero)
    api.spec_cache_keep(cache, none, zero, none, 64)
    a, b = api.spec_cache_read(cache, none, 0, 64)
    assert a.shape == (0, 0, 2, 64)
    cache = api.spec_cache_alloc(2, 2, 64, 16)
    one = ints([[0]])
    k = torch.empty((1, 0, 2, 64), device="cuda")
    st = ints([5])
    api.spec_cache_write(cache, k, k, one, ints([16]), status=st)
    assert st.tolist() == [0]
    api.spec_cache_keep(cache, one, ints([0]), torch.empty((1, 0), dtype=torch.int32, device="cuda"),
                        64, status=st)
    assert st.tolist() == [0] and not bool(cache.any())
