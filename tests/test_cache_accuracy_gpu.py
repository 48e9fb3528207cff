"""spec_cache_attention to the last places that its formula leaves: whole numbers throughout, so that a
score's sum is exact and its bound shrinks to a few roundings (needs a GPU).

Keys are whole numbers of -7 to 7 with a 7 in each group of 32 and queries of -8 to 8: products and their
sums are whole numbers below 2^14, exact in 32 bits. What is left of plain_cache's bound is, for slot j,
    E_j = 4 u (|x_j| + |m| + |b_j|) + 2^-20
(scaling, the bias b and the exponent's sum; the exponential), and each slot counts with its own:
    |out - o| <= sum_j p_j (round + E_j) |v_j| + |o| sum_j p_j E_j + L step max |v| + sums + half a step of o.
step: fp16's least step is 2^-24 and a row's largest weight is 2^7 or more (2^14 or more in tiles of few
rows), so that a small weight is off by 2^-25 and by 2^-32 (2^-39) of the largest at most.
sums: the weighted values of L slots are added 16 at a time, a step cut off by at most 2^-23 of the sum
so far; the weights' own sum is off by at most u of it for each of a lane's terms."""
import math

import pytest
import torch

import plain_cache as plain
from test_cache_attention_gpu import BF16, F32, gen, ints, tree
from token_verification_gb300 import api

pytestmark = pytest.mark.gpu
U = plain.U
SHAPES = [(1, 4, 1), (3, 8, 2), (6, 8, 2), (6, 8, 1), (17, 8, 1)]  # rows a head: 4, 12, 24, 48, 136


def whole(shape, most, g, sign=True):
    x = torch.randint(0, most + 1, shape, generator=g, device="cuda").float()
    return x * (2 * torch.randint(0, 2, shape, generator=g, device="cuda") - 1) if sign else x


def filled(slots, H, D, page, g, positive):
    """(cache, table) of one request: whole numbers, values of one sign from 4 to 7 where asked for."""
    M = -(-slots // page)
    cache = api.spec_cache_alloc(M, H, D, page)
    table = torch.randperm(M, generator=g, device="cuda").int()[None].contiguous()
    k = whole((1, M * page, H, D), 7, g)
    v = whole((1, M * page, H, D), 3, g, False) + 4 if positive else whole((1, M * page, H, D), 7, g)
    k[..., ::32] = 7
    v[..., ::32] = 7
    api.spec_cache_write(cache, k, v, table, ints([0]))
    return cache, table, torch.stack((k[0], v[0]), 2)[:slots].double()  # [slots, H, 2, D]


def expected(q, kv, sees, far, scale, dtype, slopes=None, window=0, sums=None):
    """(out, tol, lse, lse tol) of q [N, Hq, D] against kv [L, H, 2, D], in 64 bits."""
    N, Hq, D = q.shape
    L, H = kv.shape[:2]
    seen = sees & (far < window) if window else sees
    out, tol, lse, ltol = [], [], [], []
    for h in range(Hq):
        k, v = kv[:, h * H // Hq, 0], kv[:, h * H // Hq, 1]
        x = (q[:, h].double() @ k.T) * scale
        b = far * float(slopes[h]) if slopes is not None else torch.zeros_like(x)
        x = (x - b).masked_fill(~seen, -torch.inf)
        m = x.amax(-1, keepdim=True)
        E = 4 * U * (x.abs().nan_to_num(0, 0, 0) + m.abs() + b.abs()) + 2.0 ** -20
        p = x.softmax(-1)
        o = p @ v
        pE = (p * E).sum(-1, keepdim=True)
        add = (L / 16 + 64) * 2 * U if sums is None else sums
        t = (p * (E + 2.0 ** (-22 if dtype == F32 else -11))) @ v.abs() + pE * o.abs()
        many = dtype == BF16 and D <= 128 and N * Hq // H > 16
        t += 2 * add * (p @ v.abs()) + L * 2.0 ** (-32 if many else -39) * v.abs().max()
        out.append(o)
        tol.append(t + plain.HALF_STEP[dtype] * 1.01 * o.abs())
        lse.append(x.logsumexp(-1))
        ltol.append(pE[:, 0] + add + 4 * U * lse[-1].abs())
    return [torch.stack(y, 1) for y in (out, tol, lse, ltol)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("N,Hq,Hkv", SHAPES)
def test_ordinary_and_wide_scores(N, Hq, Hkv, D, dtype):
    """Scores spread by about 1, 6 and 50; chains, trees, windows and biases."""
    g = gen(N * Hq + D)
    for L in (N, N + 70, 900):
        cache, table, kv = filled(L, Hkv, D, 32, g, False)
        q = whole((1, N, Hq, D), 8, g)
        for spread in (1.0, 6.0, 50.0):
            scale = float(torch.tensor(spread / (22 * D ** 0.5), dtype=torch.float32))
            for parent, kw in ((None, {}), (tree(1, N, g), {}), (None, dict(window=61)),
                               (None, dict(slopes=torch.full((Hq,), 2.0 ** -4, device="cuda")))):
                out = api.spec_cache_attention(q.to(dtype), cache, table, ints([L]), scale=scale, lse=True,
                                               parent=parent if N > 1 else None, **kw)
                sees, depth = plain.ancestors(parent[0].cpu() if parent is not None else None, N)
                all_see = torch.ones((N, L), dtype=torch.bool)
                all_see[:, L - N:] = sees
                at = torch.arange(L)
                at[L - N:] = L - N + depth
                far = (at[L - N:, None] - at).double().cuda()
                o, tol, lse, ltol = expected(q[0], kv, all_see.cuda(), far, scale, dtype, **kw)
                # (half of the elements are held to 0.2 %, 3 % in bf16, those near 0 among them)
                assert float((tol / (o.abs() + 0.01)).median()) < (2.0 ** -9 if dtype == F32 else 2.0 ** -5)
                assert bool(((out.out[0].double() - o).abs() <= tol).all())
                assert bool(((out.lse[0].double() - lse).abs() <= ltol).all())


@pytest.mark.parametrize("D,Hq", [(64, 1), (128, 4), (256, 2), (128, 24)])
def test_long_sums_of_fp32(D, Hq):
    """131072 slots of one CTA each, values of one sign. A lane adds 4096 weights; ordinary additions are off
    by up to u in either direction, so that n of them come to sqrt(n) u or so: 8 times that, and 2^-17 for
    the 256 products of the tensor cores between two ordinary additions of the values."""
    g = gen(D + Hq)
    L, page, B = 131072, 256, 640
    cache, table, kv = filled(L, 1, D, page, g, True)
    q = whole((1, 1, Hq, D), 8, g)
    scale = float(torch.tensor(0.5 / (22 * D ** 0.5), dtype=torch.float32))
    out = api.spec_cache_attention(q.expand(B, 1, Hq, D), cache, table.expand(B, -1).contiguous(),
                                   ints([L] * B), scale=scale, lse=True)
    far = torch.arange(L - 1, -1, -1, device="cuda")[None].double()
    o, tol, lse, ltol = expected(q[0], kv, far >= 0, far, scale, F32, sums=8 * 4096 ** 0.5 * U + 2.0 ** -17)
    assert float((tol / o.abs()).median()) < 2.0 ** -13
    assert bool(((out.out.double() - o).abs() <= tol).all())
    assert bool(((out.lse.double() - lse).abs() <= ltol).all())


@pytest.mark.parametrize("Hq,dtype", [(4, BF16), (24, BF16), (64, BF16), (2, F32)])
def test_longest_context_of_one_sign(Hq, dtype):
    """2^27 slots, which all lie in one page, and values of 4 to 7. A block adds the weighted values of 2^27 / 152
    slots at most, 16 at a time, each time off by up to 2^-23 of the sum: 2^-7.2 of it. In fp32 a lane adds
    2^27 / 152 / 32 weights, the same few over and over, each time off by up to u: 2^-9.2."""
    g = gen(Hq)
    D, page, many = 64, 256, 1 << 19
    cache, _, kv = filled(page, 1, D, page, g, True)
    q = whole((1, 1, Hq, D), 8, g)
    scale = float(torch.tensor(1.0 / (22 * D ** 0.5), dtype=torch.float32))
    out = api.spec_cache_attention(q.to(dtype), cache, torch.zeros((1, many), dtype=torch.int32, device="cuda"),
                                   ints([page * many]), scale=scale, lse=True)
    assert out.status.tolist() == [0]
    far = torch.zeros((1, page), dtype=torch.float64, device="cuda")
    sums = 2.0 ** (-7.2 if dtype == BF16 else -9.2)
    o, tol, lse, ltol = expected(q[0], kv, far >= 0, far, scale, dtype, sums=sums / 2)
    assert float((tol / o.abs()).median()) < 2.0 ** (-6 if dtype == BF16 else -9)
    assert bool(((out.out[0].double() - o).abs() <= tol).all())
    assert bool(((out.lse[0].double() - lse - math.log(many)).abs() <= ltol + sums + 4 * U * math.log(many)).all())
