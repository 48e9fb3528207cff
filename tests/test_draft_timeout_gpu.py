"""The bounded waits of the top-logits and beam kernels (needs a GPU).

A limit of 0 makes every wait give up without polling: no fault, no hang (the
kernels still let what is on its way to them land before they leave). Every
row or request whose wait ran out says so in its status, and in its
log-sum-exp where no status is asked for; the next call is correct."""
import math

import pytest
import torch

import plain_draft as plain
from token_verification_gb300 import api

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


@pytest.fixture
def no_wait():
    old = api.wait_limit_ns()
    def run(call):
        try:
            api.set_wait_limit_ns(0)
            out = call()
            torch.cuda.synchronize()
        finally:
            api.set_wait_limit_ns(old)
        return out
    return run


# a cluster a row; the row kernel with fewer, with more and with many more rows than it has CTAs
@pytest.mark.parametrize("B,P,V,dtype", [(2, 3, 64000, BF16), (1, 1, 152064, F32),
                                         (25, 4, 8000, BF16), (300, 2, 3001, F32),
                                         (600, 6, 1000, BF16)])
def test_records(no_wait, B, P, V, dtype):
    x = torch.randn((B, P, V), generator=gen(V), device="cuda").to(dtype)
    lens = (torch.arange(B, device="cuda") % (P + 1)).to(torch.int32)
    lens[B - 1] = P + 1 if B > 1 else P
    for d in (None, lens):
        out = no_wait(lambda: api.spec_top_logits(x, 20, lens=d))
        quiet = no_wait(lambda: api.spec_top_logits(x, 20, lens=d, status=False))
        need = torch.ones((B, P), dtype=torch.bool, device="cuda")
        want = torch.full((B, P), api.REQ_TIMEOUT, device="cuda")
        if d is not None:
            need = torch.arange(P, device="cuda")[None] < d[:, None]
            need &= (d <= P)[:, None]
            want = torch.where(need, want, 0)
            want[d > P] = api.REQ_BAD_DRAFT_LEN
        assert torch.equal(out.status.long(), want.long())
        for o in (out, quiet):
            assert torch.equal(torch.isnan(o.lse), need)
            assert bool((o.ids == -1).all()) and bool((o.logits == -math.inf).all())
        good = api.spec_top_logits(x, 20, lens=d)
        few = slice(0, 10)
        plain.check_top(x[few], 20, 1.0, api.TopLogits(good.ids[few], good.logits[few],
                                                       good.lse[few], good.status[few]),
                        None if d is None else d[few].tolist())
        assert not bool((good.status == api.REQ_TIMEOUT).any())


@pytest.mark.parametrize("B,W,V", [(2, 4, 32000), (1, 1, 5000), (3, 16, 9001), (200, 12, 1500),
                                   (64, 8, 128256)])
def test_beams(no_wait, B, W, V):
    x = torch.randn((B, W, V), generator=gen(V), device="cuda").to(BF16)
    s = -torch.rand((B, W), generator=gen(1), device="cuda")
    s[:, 0] = -math.inf if W > 1 else 0.0
    out = no_wait(lambda: api.spec_beam_select(x, s, 12))
    assert bool((out.status == api.REQ_TIMEOUT).all()), out.status.unique()
    assert bool((out.tokens == -1).all()) and bool((out.parents == -1).all())
    assert bool((out.scores == -math.inf).all())
    good = api.spec_beam_select(x, s, 12)
    assert not bool(good.status.any())
    plain.check_beam(x[:2], s[:2], 12, api.BeamOutputs(good.tokens[:2], good.parents[:2],
                                                       good.scores[:2]))


def test_finished_requests_wait_for_nothing(no_wait):
    """A request of finished beams only, beside others, in the row kernel."""
    x = torch.randn((6, 16, 3000), generator=gen(2), device="cuda")
    s = torch.zeros((6, 16), device="cuda")
    s[::2] = -math.inf
    out = no_wait(lambda: api.spec_beam_select(x, s, 5))
    assert out.status.tolist() == [0, api.REQ_TIMEOUT] * 3
    assert bool((out.tokens == -1).all())
