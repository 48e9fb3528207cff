"""Gradients of spec_distill where they are differences of nearly equal masses,
against the definition in float64 (needs a GPU).

Bounds, u = 2^-24.  A weight is 2^a, a = (l - m) c: the difference, c and the
product each round, 3 |a| ln 2 u in all, and the exponential is good to 4 u.
Moving a sum to a larger max costs the same once more over all moves (their
exponents add up to at most |a|) and 5 u a move, at most 12 moves; its
additions are at most 32 in a row.  So a weight over a sum of weights is off by
at most
    R(A) = (9 A ln 2 + 4 + 60 + 32 + 4) u < (7 A + 100) u
of itself when every exponent that matters is at least -A (weights below 2^-30
of the sum are 0 to it: A <= 30 whatever the row).  A teacher probability is off
by (2 |t - t_max| / T + |log p| + 4) u < (3 B + 4) u, |log p| <= B."""
import math

import pytest
import torch

from token_verification_gb300 import api

pytestmark = pytest.mark.gpu
F32 = torch.float32
U = 2.0 ** -24


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def ratio(A):
    return (7 * A + 100) * U


def case(B, P, V, k, dtype, T, seed):
    g = gen(seed)
    teacher = (torch.randn((B, P, V), generator=g, device="cuda") * 3.0).to(dtype)
    rec = api.spec_top_logits(teacher, k, T)
    s = teacher.float() * 0.9 + 0.7 * torch.randn((B, P, V), generator=g, device="cuda")
    gl = torch.rand((B, P), generator=g, device="cuda") + 0.5
    return s.to(dtype), rec.ids, rec.logits, rec.lse, gl


def definition(s, ids, t, lse, T):
    """Loss [B, P] in float64 as a function of s (float64, for autograd), and its parts."""
    logq = torch.log_softmax(s / T, -1)
    at = ids.long()
    p = (t.double() / T - lse.double()[..., None]).exp()
    loss = torch.special.xlogy(p, p).sum(-1) - (p * logq.gather(-1, at)).sum(-1)
    outside = torch.ones_like(logq).scatter(-1, at, 0.0).bool()
    p_rest = torch.zeros_like(loss)
    share = torch.zeros_like(logq)
    if ids.shape[-1] < s.shape[-1]:
        p_rest = (1.0 - p.sum(-1)).clamp(min=0.0)
        log_rest = torch.logsumexp(logq.masked_fill(~outside, -math.inf), -1)
        loss = loss + torch.special.xlogy(p_rest, p_rest) - p_rest * log_rest
        share = (logq.masked_fill(~outside, -math.inf) - log_rest[..., None]).exp().detach()
    pv = torch.zeros_like(share).scatter(-1, at, p)
    return loss, logq.exp().detach(), pv, p_rest, share


def both_ways(s, ids, t, lse, T, gl):
    """Losses and gradients: fused, and apart."""
    one = api.spec_distill(s, ids, t, T, top_lse=lse, grad_loss=gl)
    two = api.spec_distill(s, ids, t, T, top_lse=lse)
    grad = api.spec_distill_grad(s, ids, t, T, two.stats, gl, top_lse=lse)
    torch.cuda.synchronize()
    assert not bool(one.status.any()) and not bool(two.status.any())
    return (one.loss, one.grad), (two.loss, grad)


@pytest.mark.parametrize("V,k,T", [(100000, 4, 8.0), (128256, 32, 4.0), (4099, 2, 16.0)])
def test_small_differences_of_large_remainders(V, k, T):
    """Soft rows: nearly all mass lies outside the record on both sides. The gradient there is
    share_i (q_rest - p_rest) = share_i (p_sum - q_sum), and is held to the error of those two
    small sums, not to that of the remainders near 1."""
    s, ids, t, lse, gl = case(4, 6, V, k, F32, T, V)
    x = s.double()
    assert float((x.amax(-1) - x.amin(-1)).max()) / T * math.log2(math.e) < 16
    _, q, pv, p_rest, share = definition(x, ids, t, lse, T)
    outside = torch.ones_like(q).scatter(-1, ids.long(), 0.0)
    p_sum, q_sum = pv.sum(-1), 1.0 - (q * outside).sum(-1)
    assert float((p_sum + q_sum).max()) < 0.2
    scale = (gl.double() / T)[..., None]
    want = scale * share * ((q * outside).sum(-1) - p_rest)[..., None]
    # two sums of ratios (and the p_j: B = 14), then a ratio and a few roundings
    tol = scale * share * (2 * ratio(16) * (p_sum + q_sum))[..., None] + 2 * ratio(16) * want.abs()
    for _, grad in both_ways(s, ids, t, lse, T, gl):
        off = (grad.double() - want).abs() * outside
        assert bool((off <= tol).all()), float((off / tol.clamp(min=1e-300)).max())
