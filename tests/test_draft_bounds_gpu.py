"""Log-sum-exps and beam scores held to the errors that their arithmetic can
make on inputs where those are few (needs a GPU).

u = 2^-24.  Rows of one value: every weight is 2^0 = 1 and every sum a whole
number, so what is left is the logarithm (2^-24 beside the rounding of its two
parts' sum) and the roundings of m / T and of the result.

Rows within [-0.5, 0.5] of at most 8192 logits, T = 1: an exponent (l - m) c is at
most 1.45 in size and rounds three times (the difference, c, the product), 3 u
of the weight in all (3 * 1.45 ln 2), and the exponential is good to 4 u: 7 u.
A thread adds its 32 weights in eight accumulators and a tree, 7 u (fp32: in
two steps, with a move between them); its sum moves to the warp's max and that
one to the row's, 7 u and a product's u each, and a warp adds with 5 u; the
rest is summed in pairs. At most 7 + 7 + 3 * 8 + 5 + 5 = 48 u of the sum, and so
of its logarithm."""
import math

import pytest
import torch

from token_verification_gb300 import api

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("V", [1, 2, 3, 7, 1000, 46341, 152064, 700001, 1 << 24])
@pytest.mark.parametrize("value,T", [(0.0, 1.0), (3.25, 0.7), (-1.5, 2.0), (-40.0, 1.0)])
def test_constant_rows(V, value, T):
    for rows, dtype in ((1, BF16), (2, F32), (150, BF16)):
        if rows * V > 1 << 26:
            continue
        x = torch.full((rows, 1, V), value, dtype=dtype, device="cuda")
        out = api.spec_top_logits(x, 2, T)
        t = float(torch.tensor(T, dtype=F32))
        want = value / t + math.log(V)
        tol = U * (abs(value / t) + 2 * math.log(V) + abs(want)) + 2.0 ** -24
        assert float((out.lse.double() - want).abs().max()) <= tol


@pytest.mark.parametrize("rows", [3, 200])
@pytest.mark.parametrize("V", [500, 4097, 8192])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_short_rows_of_small_logits(rows, V, dtype):
    x = (torch.rand((rows, 1, V), generator=gen(V), device="cuda") - 0.5).to(dtype)
    out = api.spec_top_logits(x, 4)
    want = torch.logsumexp(x.double(), -1)
    assert bool(((out.lse.double() - want).abs() <= (48 + 2) * U + 2 * U * want.abs()).all())


@pytest.mark.parametrize("B,W,V", [(1, 4, 8192), (2, 8, 5000), (3, 32, 4097), (40, 16, 8192)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_beams_of_small_logits(B, W, V, dtype):
    """Scores within 50 u and their own rounding; candidates change places only where they are
    closer than twice that, which equal rows are not."""
    g = gen(B * W + V)
    x = (torch.rand((B, W, V), generator=g, device="cuda") - 0.5).to(dtype)
    s = -torch.rand((B, W), generator=g, device="cuda")
    n = 48
    out = api.spec_beam_select(x, s, n)
    every = (s.double()[..., None] + torch.log_softmax(x.double(), -1)).flatten(1)
    best = every.sort(dim=-1, descending=True, stable=True)
    mine = every.gather(1, out.parents.long() * V + out.tokens)
    off = 50 * U
    assert bool(((mine - best.values[:, :n]).abs() <= 2 * off).all())
    assert bool(((out.scores.double() - mine).abs() <= off + U * mine.abs()).all())
    sure = torch.ones_like(mine, dtype=torch.bool)  # further than that from both neighbours
    gap = best.values[:, :n] - best.values[:, 1:n + 1] > 2 * off
    sure &= gap
    sure[:, 1:] &= gap[:, :-1]
    assert bool(sure.any()) or dtype == BF16
    got = out.parents.long() * V + out.tokens
    assert torch.equal(got[sure], best.indices[:, :n][sure])


@pytest.mark.parametrize("V", [3, 1000, 50001])
def test_beams_of_constant_rows(V):
    x = torch.full((2, 6, V), 0.75, dtype=BF16, device="cuda")
    s = torch.arange(12, device="cuda").view(2, 6) * -0.25
    out = api.spec_beam_select(x, s, 5)
    want = (s[:, :1].double() - math.log(V)).expand(2, 5)
    if V >= 5:
        assert bool(((out.scores.double() - want).abs() <= U * want.abs() + 1.5 * 2.0 ** -24).all())
        assert out.tokens.tolist() == [[0, 1, 2, 3, 4]] * 2
