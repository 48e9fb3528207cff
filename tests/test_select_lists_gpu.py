"""Selections whose lists of candidates hold several hundred entries, which are
cut to their n-th largest key before they are ranked (needs a GPU).

The inputs fix the list's length.  `marks` logits of a row lie in [5, 5 + 2^-6),
all others below 4: in bf16, to which the bound of the unit maxes is rounded
down, every mark is 5.0 (the next value is 5 + 2^-5).  The marks are spread so
evenly that at least n units hold one, so the bound is 5.0 and the list is the
marks: 385 to 1024 of them."""
import pytest
import torch

import plain_draft as plain
from token_verification_gb300 import api

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
TURNS = 60


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def marked(rows, V, marks, dtype, seed, above=0):
    """[rows, V] logits with `marks` of them near 5 at even steps, in random order of size
    (bf16: all equal), `above` of those at 6."""
    g = gen(seed)
    x = torch.rand((rows, V), generator=g, device="cuda") * 8 - 4
    at = (torch.arange(marks, device="cuda") * V) // marks
    if dtype == F32:
        order = torch.rand((rows, marks), generator=g, device="cuda").argsort(-1)
        x[:, at] = 5 + order.float() * (2.0 ** -6 / marks)
    else:
        x[:, at] = 5.0
    if above:
        x[:, at[::marks // above][:above]] = 6.0
    return x.to(dtype).contiguous()


def again(call, names, first):
    """The same call over and over beside a busy stream: the same answer each time."""
    noise, side = torch.empty(1 << 27, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for i in range(TURNS):
        with torch.cuda.stream(side):
            noise.add_(1)
        got.append(call())
    torch.cuda.synchronize()
    for out in got:
        for f in names:
            assert torch.equal(getattr(out, f), getattr(first, f)), f


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,V,marks,k", [
    (6, 70000, 900, 128), (6, 70000, 400, 64), (3, 64001, 1024, 100),  # a cluster a row
    (200, 8000, 900, 128), (200, 8000, 500, 100), (40, 7001, 386, 64)])  # the row kernel
def test_long_lists_of_a_record(rows, V, marks, k, dtype):
    for above in (0, k // 2):
        x = marked(rows, V, marks, dtype, V + k + above, above).view(rows, 1, V)
        out = api.spec_top_logits(x, k)
        torch.cuda.synchronize()
        plain.check_top(x, k, 1.0, out)
        again(lambda: api.spec_top_logits(x, k), ("ids", "logits", "lse", "status"), out)


@pytest.mark.parametrize("V,k", [(385, 64), (400, 128), (700, 64), (1000, 64), (1024, 128)])
@pytest.mark.parametrize("rows", [2, 150])
def test_rows_listed_whole(rows, V, k):
    """Too few units for a bound: all V logits are on the list."""
    for dtype in (BF16, F32):
        x = (torch.randn((rows, 1, V), generator=gen(V), device="cuda") * 3).to(dtype)
        out = api.spec_top_logits(x, k)
        torch.cuda.synchronize()
        plain.check_top(x, k, 1.0, out)
        again(lambda: api.spec_top_logits(x, k), ("ids", "logits", "lse", "status"), out)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("W,V,marks,n", [
    (4, 20000, 225, 128), (2, 9000, 300, 100),   # a cluster a request
    (32, 9000, 22, 128), (64, 5001, 12, 100)])   # a list of W * marks in the merge
def test_long_lists_of_beams(W, V, marks, n, dtype):
    """Equal rows of equal scores: W * marks candidates share the bound's bf16 value."""
    one = marked(1, V, marks, dtype, W + V)
    x = one.expand(3, W, V).contiguous()
    s = torch.full((3, W), -1.0, device="cuda")
    out = api.spec_beam_select(x, s, n)
    torch.cuda.synchronize()
    assert not bool(out.status.any())
    assert plain.check_beam(x, s, n, out) == 0
    again(lambda: api.spec_beam_select(x, s, n), ("tokens", "parents", "scores"), out)


@pytest.mark.parametrize("spread", [1.5, 3.0])
@pytest.mark.parametrize("rows,V,k", [(4, 152064, 128), (120, 152064, 64), (120, 50000, 100)])
def test_vocabularies_ordered_by_frequency(rows, V, k, spread):
    """Logits that fall with the token's id, as real vocabularies' do: the candidates crowd at
    the low ids and the lists are several times longer than over a shuffled vocabulary."""
    g = gen(V + k)
    prior = -1.1 * torch.log1p(torch.arange(V, device="cuda", dtype=F32))
    for dtype in (BF16, F32):
        x = (torch.randn((rows, 1, V), generator=g, device="cuda") * spread + prior).to(dtype)
        out = api.spec_top_logits(x, k)
        torch.cuda.synchronize()
        few = slice(0, 24)
        plain.check_top(x[few], k, 1.0, api.TopLogits(out.ids[few], out.logits[few], out.lse[few],
                                                      out.status[few]))
        again(lambda: api.spec_top_logits(x, k), ("ids", "logits", "lse"), out)
