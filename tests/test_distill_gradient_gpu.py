"""Gradients and losses of spec_distill where they are differences of nearly
equal masses, where the record's mass is not 1, and where teacher and student
are masked alike, against the definition in float64 (needs a GPU).

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
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
HALF_STEP = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


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


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V,k,shift", [(1000, 32, -0.4), (1000, 128, -0.05), (50001, 64, -1.0),
                                       (100, 100, -0.3), (100, 100, 0.3), (64, 64, -0.01)])
def test_records_of_another_mass(V, k, shift, dtype):
    """A log-sum-exp that does not fit the record (taken at another temperature, or rounded far
    from zero): sum p is not 1, and the gradient is still the derivative of the loss."""
    T = 1.0
    s, ids, t, lse, gl = case(2, 3, V, k, dtype, T, V + k)
    if k < V:  # from the record's own log-sum-exp: sum p = e^-shift > 1
        lse = torch.logsumexp(t.double() / T, -1).float()
    lse = lse + shift
    x = s.double().requires_grad_()
    loss, q, pv, p_rest, share = definition(x, ids, t, lse, T)
    (gl.double() * loss).sum().backward()
    want = x.grad
    mass = (pv.sum(-1) + p_rest)[..., None]
    assert float((mass - 1).abs().min()) > 0.005
    scale = (gl.double() / T)[..., None]
    tol = scale * (2 * ratio(30) * (mass * q + p_rest[..., None] * share) + 100 * U * pv)
    tol = 1.01 * (tol + HALF_STEP[dtype] * want.abs()) + 1e-37
    size = (pv * (pv.clamp(min=1e-300).log().abs() + q.log().abs())).sum(-1)
    for got, grad in both_ways(s, ids, t, lse, T, gl):
        off = (grad.double() - want).abs()
        assert bool((off <= tol).all()), float((off / tol).max())
        assert bool(((got.double() - loss).abs() <= 2 * ratio(30) * (1 + size)).all())


def test_differences_of_a_loss_of_another_mass():
    """Central differences of the loss itself, sum p = e^0.5: as for records of mass 1, the third
    derivative along a direction of entries at most 1 is at most 8 for each log-sum-exp, times
    the mass."""
    T, h = 1.0, 0.05
    s, ids, t, _, gl = case(2, 3, 1001, 16, F32, T, 9)
    lse = torch.logsumexp(t.double(), -1).float() - 0.5
    one = torch.ones_like(gl)
    grad = api.spec_distill(s, ids, t, T, top_lse=lse, grad_loss=one).grad
    d = torch.rand(s.shape, generator=gen(10), device="cuda") * 2 - 1
    up = api.spec_distill(s + h * d, ids, t, T, top_lse=lse).loss.double()
    down = api.spec_distill(s - h * d, ids, t, T, top_lse=lse).loss.double()
    want = (up - down) / (2 * h)
    got = (grad.double() * d.double()).sum(-1)
    mass = math.exp(0.5)
    tol = h * h / 6 * 8 * mass + 2 * 2 * ratio(30) * 48 * mass / (2 * h)
    assert bool(((got - want).abs() <= tol).all()), (got, want, tol)


@pytest.mark.parametrize("T,at", [(1.0, 0.0), (0.7, 0.0), (1.0, 150.0), (2.0, -900.0)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_teacher_and_student_masked_alike(dtype, T, at):
    """A grammar leaves fewer tokens than the record keeps, on both sides: the record holds all
    of the teacher's mass, and what the rounding of its log-sum-exp leaves of 1 - sum p is no
    mass on tokens that the student rules out."""
    B, P, V, k = 16, 8, 3001, 24
    g = gen(5)
    allow = torch.arange(B * P, device="cuda").view(B, P) % 23 + 1  # 1 to 23 tokens
    order = torch.rand((B, P, V), generator=g, device="cuda").argsort(-1).argsort(-1)
    mask = order >= allow[..., None]
    def rows(noise):
        x = torch.randn((B, P, V), generator=g, device="cuda") * noise + at
        return x.to(dtype).masked_fill(mask, -math.inf)
    rec = api.spec_top_logits(rows(3.0), k, T)
    s = rows(2.0)
    gl = torch.ones((B, P), device="cuda")
    assert torch.equal((rec.ids >= 0).sum(-1), allow)
    use = rec.ids >= 0
    ids = rec.ids.long().clamp(min=0)
    logp = (rec.logits.double() / T - rec.lse.double()[..., None]).masked_fill(~use, -math.inf)
    p = logp.exp()
    assert bool((p.sum(-1) < 1).any()) and bool((p.sum(-1) > 1).any())  # the roundings
    logq = torch.log_softmax(s.double() / T, -1).gather(-1, ids).masked_fill(~use, 0.0)
    terms = torch.where(use, p * (logp - logq), 0.0)
    grads = torch.zeros(s.shape, dtype=torch.float64, device="cuda")
    grads.scatter_add_(-1, ids, torch.where(use, (logq.exp() * p.sum(-1, keepdim=True) - p) / T, 0.0))
    tol = 2 * ratio(30) * (1 + terms.abs().sum(-1))
    for loss, grad in both_ways(s, rec.ids, rec.logits, rec.lse, T, gl):
        assert bool(torch.isfinite(loss).all()), int((~torch.isfinite(loss)).sum())
        assert bool(((loss.double() - terms.sum(-1)).abs() <= tol).all())
        # each p and q at most 1 and 2 ratios off; what is left of 1 - sum p is up to 2^-20 + 2^-23 |lse|
        room = 4 * ratio(30) + 2.0 ** -20 + 2.0 ** -23 * rec.lse.abs().double()[..., None]
        off = (grad.double() - grads).abs()
        assert bool((off <= room / T + HALF_STEP[dtype] * grads.abs() * 1.01).all())
    # a remainder that is more than rounding stays what it is
    far = api.spec_distill(s, rec.ids, rec.logits, T, top_lse=rec.lse + 0.01 + rec.lse.abs() * 1e-4)
    assert bool((far.loss == math.inf).all())


def test_mass_past_the_range():
    """A log-sum-exp so far below its record that a probability is no fp32 number: a data error."""
    s, ids, t, lse, gl = case(1, 3, 1000, 8, F32, 1.0, 11)
    lse[0, 1] -= 200.0
    out = api.spec_distill(s, ids, t, top_lse=lse, grad_loss=gl)
    fwd = api.spec_distill(s, ids, t, top_lse=lse)
    grad = api.spec_distill_grad(s, ids, t, 1.0, fwd.stats, gl, top_lse=lse)
    for o in (out, fwd):
        assert o.status.tolist() == [[0, api.REQ_BAD_LOGITS, 0]]
        assert torch.isnan(o.loss).tolist() == [[False, True, False]]
    for g in (out.grad, grad):
        assert not bool(g[0, 1].any()) and bool(g[0, 0].any())


@pytest.mark.parametrize("T", [1.0, 64.0, 1e6])
def test_ruled_out_token_of_the_least_mass(T):
    """A recorded token of a probability near fp32's least, which the student rules out: the
    loss is +inf, as for any p > 0."""
    s, ids, t, _, gl = case(1, 2, 1000, 4, F32, T, 12)
    t[:, :, 0] = 0.0
    t[:, :, 1:] = torch.tensor([-101.0, -102.0, -400.0], device="cuda") * T  # p: 1e-44, 6e-45, 0
    s[0, 0, ids[0, 0, 1].long()] = -math.inf
    s[0, 1, ids[0, 1, 3].long()] = -math.inf  # (no mass there: a term of 0)
    out = api.spec_distill(s, ids, t, T, grad_loss=gl)
    assert not bool(out.status.any())
    assert float(out.loss[0, 0]) == math.inf and math.isfinite(float(out.loss[0, 1]))
    assert bool(torch.isfinite(out.grad).all())
