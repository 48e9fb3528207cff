"""Scores of any size that fp32 holds in spec_cache_attention: rows whose weights follow
from the scores' order alone (needs a GPU).

Keys and queries have one value each that is not 0, so scores are single products, the keys' value
7 * 2^i, which the cache holds exactly.  In rows of large scores those of two slots are either equal to the
bit or 2^12 apart and more: the exact weights are equal ones on the largest scores and 0 elsewhere,
however the scores were rounded, and all that is off is (tests/plain_cache.py) the weights' rounding
of 2^-11 (2^-22 in fp32), the running sums and the result's half step.  Rows of ordinary scores
(|x| <= 2) share their tile; their weights are off by 2 E, E = 4 u (|x| + |m|) + 2^-20 < 2^-18 in addition."""
import math

import pytest
import torch

import plain_cache as plain
from test_cache_attention_gpu import BF16, F32, gen, ints
from token_verification_gb300 import api

pytestmark = pytest.mark.gpu
SHAPES = [(1, 4, 1), (3, 8, 2), (6, 8, 2), (6, 8, 1), (17, 8, 1)]  # rows a head: 4, 12, 24, 48, 136


def levels(pattern, L, sign, g):
    """Exponents i of the slots' keys 7 * 2^i; the largest scores are at 2^7 (sign > 0) or 2^-3."""
    up = torch.empty(L, dtype=torch.int64, device="cuda")
    if pattern == "ties":
        up[:] = 0
    elif pattern == "few":  # three slots and the first, which every row sees
        up[:] = 1
        up[torch.randint(0, L, (3,), generator=g, device="cuda")] = 0
        up[0] = 0
    else:  # ever larger along the slots
        up[:] = 10 - 11 * torch.arange(L, device="cuda") // L
    return 7 - up if sign > 0 else -3 + up


def check(B, L, N, Hq, Hkv, D, dtype, top, pattern, g, **kw):
    """`top`: the rows' largest score; its sign is every score's."""
    sign = 1 if top > 0 else -1
    i = levels(pattern, L, sign, g)
    k = torch.zeros((1, L, Hkv, D), device="cuda")
    k[..., 5] = (7 * torch.exp2(i.double())).float()[:, None]
    v = torch.randn((1, L, Hkv, D), generator=g, device="cuda")
    page = 64
    M = -(-L // page)
    cache = api.spec_cache_alloc(M, Hkv, D, page)
    table = torch.arange(M, device="cuda").int()[None].contiguous()
    api.spec_cache_write(cache, k, v, table, ints([0]))
    # every third row's scores are 2 at most
    unit = 7 * 2.0 ** int(i.max() if sign > 0 else i.min())
    a = 2.0 ** min(100, max(0, math.frexp(top)[1] - 20))
    scale = float(torch.tensor(top / (unit * a), dtype=torch.float32))
    q = torch.zeros((1, N, Hq, D), device="cuda")
    q[..., 5] = a
    plainly = (torch.arange(N * Hq, device="cuda") % 3 == 1).view(N, Hq)
    most = 7 * 2.0 ** int(i.max())
    q[0, ..., 5][plainly] = 2.0 ** math.floor(math.log2(2 / (most * abs(scale))))
    q = q.to(dtype)
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    out = api.spec_cache_attention(q.expand(B, N, Hq, D), cache, table.expand(B, M).contiguous(), lens,
                                   lse=True, scale=scale, **kw)
    assert not bool(out.status.any())
    kv = plain.slots(plain.decode(cache, page, D), table[0], L)
    assert torch.equal(kv[:, :, 0].cpu(), k[0].cpu().double())
    sees = torch.arange(L) <= L - N + torch.arange(N)[:, None]
    if kw.get("window"):
        sees &= torch.arange(L) > L - N + torch.arange(N)[:, None] - kw["window"]
    for h in range(Hq):
        x = (q[0, :, h].cpu().double() @ kv[:, h * Hkv // Hq, 0].T) * scale
        x = x.masked_fill(~sees, -math.inf)
        p, vv = x.softmax(-1), kv[:, h * Hkv // Hq, 1]
        o = p @ vv
        E = torch.where(plainly[:, h].cpu(), 2.0 ** -17, 0.0)[:, None]
        rounding = 2.0 ** (-22 if dtype == F32 else -11)
        tol = (rounding + E + 2 * (64 + L / 4) * plain.U) * (p @ vv.abs())
        tol += plain.HALF_STEP[dtype] * o.abs() * 1.01 + 2.0 ** -30 * vv.abs().max()
        off = (out.out[:, :, h].cpu().double() - o).abs()
        assert bool((off <= tol).all()), (h, float((off / tol).nan_to_num(math.inf).max()))
        lse = x.logsumexp(-1)
        # scaled by log2 e, by ln 2 and added to the log of the sum: three roundings, and the tanh's two places
        ltol = (64 + L / 4) * plain.U + 2.0 ** -18 + (8 if kw.get("softcap") else 4) * plain.U * lse.abs()
        assert bool(((out.lse[:, :, h].cpu().double() - lse).abs() <= ltol).all()), h


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("N,Hq,Hkv", SHAPES)
def test_large_scores(N, Hq, Hkv, D, dtype):
    """Largest scores of 2^17 to 2^125 of both signs, for one slot, several and all of them."""
    g = gen(N * Hq + D)
    for e in (17, 20, 23, 24, 25, 26, 27, 28, 29, 30, 33, 60, 100, 125):
        for top in (1.37 * 2.0 ** e, -1.37 * 2.0 ** (e - 1), 1.99 * 2.0 ** e):
            check(1, N + 500, N, Hq, Hkv, D, dtype, top, ("ties", "few", "rising")[e % 3], g)
    for e in (24, 26, 28, 31):
        for pattern in ("ties", "few", "rising"):
            check(1, N, N, Hq, Hkv, D, dtype, 1.71 * 2.0 ** e, pattern, g)
            check(1, N + 777, N, Hq, Hkv, D, dtype, -1.71 * 2.0 ** e, pattern, g)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,Hq,Hkv", SHAPES)
def test_large_scores_of_long_pieces(N, Hq, Hkv, dtype):
    """As many requests as there are places for CTAs: each walks all chunks of its rows."""
    g = gen(N + Hq)
    for D in (64, 128, 256):
        for e in (24, 28, 90):
            for pattern in ("few", "rising"):
                check(620, 900, N, Hq, Hkv, D, dtype, 1.37 * 2.0 ** e, pattern, g)
                check(620, 900, N, Hq, Hkv, D, dtype, -1.37 * 2.0 ** e, pattern, g)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_large_scores_capped_biased_and_windowed(D, dtype):
    g = gen(D)
    for N, Hq, Hkv in SHAPES:
        none = torch.zeros(Hq, device="cuda")
        for kw in (dict(softcap=1e30), dict(slopes=none), dict(window=130),
                   dict(softcap=1e30, slopes=none, window=300)):
            for e in (24, 27, 30):
                check(1, N + 400, N, Hq, Hkv, D, dtype, 1.37 * 2.0 ** e, "ties", g, **kw)
                check(1, N + 400, N, Hq, Hkv, D, dtype, -1.37 * 2.0 ** e, "rising", g, **kw)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_largest_queries(D):
    """Queries of fp32's largest numbers, whose scores are ordinary ones."""
    g = gen(D)
    most = torch.finfo(F32).max
    for N, Hq, Hkv in SHAPES:
        for big in (most, -most, 1.75 * 2.0 ** 127):
            L = N + 90
            k = torch.zeros((1, L, Hkv, D), device="cuda")
            i = torch.randint(-17, 0, (L,), generator=g, device="cuda")
            k[..., 3] = (7 * torch.exp2(i.double())).float()[:, None]
            v = torch.randn((1, L, Hkv, D), generator=g, device="cuda")
            cache = api.spec_cache_alloc(4, Hkv, D, 64)
            table = ints([[3, 0, 1, 2]])
            api.spec_cache_write(cache, k, v, table, ints([0]))
            q = torch.zeros((1, N, Hq, D), device="cuda")
            q[..., 3] = big
            scale = 2.0 ** -127
            out = api.spec_cache_attention(q, cache, table, ints([L]), scale=scale, lse=True)
            plain.check_attention(q, cache, 64, table, ints([L]), out.out, out.lse, scale=scale)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_largest_scales(D, dtype):
    """Scales up to fp32's largest number, over queries that are 0 or give ordinary scores."""
    g = gen(D + 1)
    most = torch.finfo(F32).max
    for N, Hq, Hkv in SHAPES:
        L = N + 90
        k = torch.zeros((1, L, Hkv, D), device="cuda")
        i = torch.randint(-17, 0, (L,), generator=g, device="cuda")
        k[..., 3] = (7 * torch.exp2(i.double())).float()[:, None]
        v = torch.randn((1, L, Hkv, D), generator=g, device="cuda")
        cache = api.spec_cache_alloc(4, Hkv, D, 64)
        table = ints([[3, 0, 1, 2]])
        api.spec_cache_write(cache, k, v, table, ints([0]))
        q = torch.zeros((1, N, Hq, D), device="cuda")
        zero = q.to(dtype)
        q[..., 3] = 2.0 ** -126
        for x in (zero, q.to(dtype)):
            for scale in (most, -most, 2.5e38):
                out = api.spec_cache_attention(x, cache, table, ints([L]), scale=scale, lse=True)
                plain.check_attention(x, cache, 64, table, ints([L]), out.out, out.lse, scale=scale)
