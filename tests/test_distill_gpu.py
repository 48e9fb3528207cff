"""spec_distill and spec_distill_grad against the plain 64-bit form
(tests/plain_draft.py), against differences of the loss, on degenerate
records and rows, in place, and in a draft head's training step (needs a GPU)."""
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


def case(B, P, V, k, dtype, T, tail, seed, noise=0.7):
    g = gen(seed)
    teacher = (torch.randn((B, P, V), generator=g, device="cuda") * 3.0).to(dtype)
    rec = api.spec_top_logits(teacher, k, T)
    s = (teacher.float() * 0.9 + noise * torch.randn((B, P, V), generator=g, device="cuda"))
    gl = torch.rand((B, P), generator=g, device="cuda") + 0.5
    return s.to(dtype), rec.ids, rec.logits, (rec.lse if tail else None), gl


def check(s, ids, t, lse, T, gl, lens=None):
    """Fused, apart and in place, all against the plain form."""
    d = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    kw = dict(top_lse=lse, lens=d)
    both = api.spec_distill(s, ids, t, T, grad_loss=gl, **kw)
    fwd = api.spec_distill(s, ids, t, T, **kw)
    assert fwd.grad is None
    grad = api.spec_distill_grad(s, ids, t, T, fwd.stats, gl, **kw)
    torch.cuda.synchronize()
    plain.check_distill(s, ids, t, lse, T, gl, lens, both.loss, both.grad, both.status)
    plain.check_distill(s, ids, t, lse, T, gl, lens, fwd.loss, grad, fwd.status)
    own = s.clone()
    inside = api.DistillOutputs(torch.empty_like(fwd.loss), None, own)
    api.spec_distill(own, ids, t, T, out=inside, grad_loss=gl, **kw)
    assert torch.equal(inside.loss, both.loss) and torch.equal(own, both.grad)
    own = s.clone()
    api.spec_distill_grad(own, ids, t, T, fwd.stats, gl, grad=own, **kw)
    assert torch.equal(own, grad)
    return both


@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 129, 1000, 1001, 4096, 8193])
@pytest.mark.parametrize("k,dtype,T,tail", [(1, BF16, 1.0, True), (16, F32, 0.7, True),
                                            (100, BF16, 2.0, False), (128, F32, 1.0, True)])
def test_sizes(V, k, dtype, T, tail):
    check(*_swap(case(2, 3, V, k, dtype, T, tail, V + k), T))


def _swap(c, T):
    s, ids, t, lse, gl = c
    return s, ids, t, lse, T, gl


@pytest.mark.parametrize("B,P,V,k,dtype,T,tail", [
    (2, 2, 152064, 64, BF16, 1.0, True), (1, 1, 152064, 100, F32, 1.0, True),
    (1, 3, 50001, 32, BF16, 2.0, True), (3, 2, 50001, 128, F32, 0.5, False),
    (400, 1, 1003, 8, BF16, 1.0, True), (1, 1, 393216, 8, F32, 1.0, True),
    (1, 1, 786432, 8, BF16, 1.0, True)])
def test_large(B, P, V, k, dtype, T, tail):
    check(*_swap(case(B, P, V, k, dtype, T, tail, B + V), T))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shift", [1, 3, 4, 6])
def test_unaligned_base(dtype, shift):
    """Student and gradient at different alignments."""
    s, ids, t, lse, gl = case(2, 3, 2056, 20, dtype, 1.0, True, shift)
    buf = torch.empty(s.numel() + 16, dtype=dtype, device="cuda")
    x = buf[shift:shift + s.numel()].view(s.shape)
    x.copy_(s)
    grad = torch.full((s.numel() + 16,), 7.0, dtype=dtype, device="cuda")
    at = 2 * shift % 8
    out = api.DistillOutputs(torch.empty_like(gl), None, grad[at:at + s.numel()].view(s.shape))
    api.spec_distill(x, ids, t, 1.0, out=out, top_lse=lse, grad_loss=gl)
    torch.cuda.synchronize()
    plain.check_distill(s, ids, t, lse, 1.0, gl, None, out.loss, out.grad)
    assert bool((grad[:at] == 7).all()) and bool((grad[at + s.numel():] == 7).all())


def test_padded_batch():
    s, ids, t, lse, gl = case(5, 4, 3001, 12, BF16, 1.0, True, 3)
    s[1, 2:] = math.nan  # not read
    ids[3, 1] = -1       # an empty record
    ids[4, 0, 5:] = -1
    both = check(s, ids, t, lse, 1.0, gl, lens=[4, 2, 0, 3, 1])
    assert float(both.loss[3, 1]) == 0.0


def test_whole_vocabulary_record():
    """k = V: there is no rest; the loss is the full divergence."""
    for dtype in (BF16, F32):
        s, ids, t, lse, gl = case(1, 4, 100, 100, dtype, 1.0, True, 5)
        both = check(s, ids, t, lse, 1.0, gl)
        q = torch.log_softmax(s.double(), -1).gather(-1, ids.long())
        lp = torch.log_softmax(t.double(), -1)
        want = (lp.exp() * (lp - q)).sum(-1)
        assert torch.allclose(both.loss.double(), want, atol=1e-4)


def test_degenerate_students():
    """A student that agrees, one that is certain, one masked at recorded tokens, one
    masked everywhere else, one whose remainder is far below fp32's range."""
    s, ids, t, lse, gl = case(1, 6, 3001, 10, F32, 1.0, True, 6)
    s[0, 1] = -40.0
    s[0, 1, ids[0, 1, 0].long()] = 60.0
    s[0, 2, ids[0, 2, 3].long()] = -math.inf
    keep = s[0, 3, ids[0, 3].long()].clone()
    s[0, 3] = -math.inf
    s[0, 3, ids[0, 3].long()] = keep
    keep = s[0, 4, ids[0, 4].long()].clone()
    s[0, 4] = -300.0
    s[0, 4, ids[0, 4].long()] = keep
    t[0, 5, 4:] = -math.inf  # recorded tokens without teacher mass
    for l in (lse, None):
        both = check(s, ids, t, l, 1.0, gl)
        assert math.isinf(float(both.loss[0, 2]))
        assert bool(torch.isfinite(both.grad).all())
        assert math.isinf(float(both.loss[0, 3])) == (l is not None)


def test_data_errors():
    s, ids, t, lse, gl = case(2, 6, 2000, 10, F32, 1.0, True, 7)
    s[0, 0, 1999] = math.nan
    s[0, 1, ids[0, 1, 2].long()] = math.inf
    s[0, 2] = -math.inf
    t[0, 3, 1] = math.nan
    ids[0, 4, 9] = 2000
    ids[0, 5, 9] = ids[0, 5, 3]
    ids[1, 0, 0] = -2
    lse[1, 1] = math.nan
    lse[1, 2] = math.nan
    ids[1, 2] = -1
    want = [[2, 2, 2, 2, 1, 1], [1, 2, 0, 0, 0, 0]]
    good = torch.tensor(want, device="cuda") == 0
    out = api.spec_distill(s, ids, t, top_lse=lse, grad_loss=gl)
    back = api.spec_distill_grad(s, ids, t, 1.0, out.stats, gl, top_lse=lse)
    assert out.status.tolist() == want
    assert torch.equal(torch.isnan(out.loss), ~good)
    for grad in (out.grad, back):
        assert bool((grad[~good] == 0).all())
        assert bool((grad[1, 3:] != 0).any())
    lens = torch.tensor([7, -1], dtype=torch.int32, device="cuda")
    out = api.spec_distill(s, ids, t, top_lse=lse, grad_loss=gl, lens=lens)
    assert bool((out.status == 4).all()) and bool((out.grad == 0).all())
    assert bool(torch.isnan(out.loss).all())


@pytest.mark.parametrize("tail", [True, False])
def test_gradient_against_differences(tail):
    """The loss along a direction d, |d| <= 1: a central difference of step h is off by at
    most h^2 / 6 times the third derivative (of log-sum-exps along d: at most 8 each, two of
    them) and by the two losses' own errors over 2 h."""
    T, h = 1.0, 0.05
    s, ids, t, lse, gl = case(2, 3, 1001, 16, F32, T, tail, 9)
    one = torch.ones_like(gl)
    grad = api.spec_distill(s, ids, t, T, top_lse=lse, grad_loss=one).grad
    d = torch.rand(s.shape, generator=gen(10), device="cuda") * 2 - 1
    d.scatter_(-1, ids.long(), torch.sign(d.gather(-1, ids.long())))
    up = api.spec_distill(s + h * d, ids, t, T, top_lse=lse).loss.double()
    down = api.spec_distill(s - h * d, ids, t, T, top_lse=lse).loss.double()
    want = (up - down) / (2 * h)
    got = (grad.double() * d.double()).sum(-1)
    tol = h * h / 6 * 16 + 2 * (2 * plain.SUM + 2.0 ** -20 * 48) / (2 * h) + 4 * plain.SUM
    assert bool(((got - want).abs() <= tol).all()), (got, want, tol)
    assert bool((want.abs() > 2 * tol).any())  # the test sees the gradient


def test_grad_loss_scales_and_zero():
    s, ids, t, lse, gl = case(2, 3, 1000, 8, F32, 1.0, True, 11)
    gl[0, 1] = 0.0
    gl[1, 2] = -3.0
    check(s, ids, t, lse, 1.0, gl)


def test_refusals():
    s, ids, t, lse, gl = case(1, 2, 100, 4, BF16, 1.0, True, 12)
    with pytest.raises(ValueError):
        api.spec_distill(s, ids, t[:, :1], top_lse=lse)
    with pytest.raises(TypeError):
        api.spec_distill(s, ids.long(), t, top_lse=lse)
    with pytest.raises(TypeError):
        api.spec_distill(s, ids, t.to(BF16), top_lse=lse)
    with pytest.raises(TypeError):
        api.spec_distill_grad(s, ids, t, 1.0, torch.zeros(1, 2, 4, device="cuda"), gl,
                              grad=s.float())
    buf = torch.zeros(s.numel() + 8, dtype=BF16, device="cuda")
    x = buf[:s.numel()].view(s.shape)
    with pytest.raises(api.VerifyError):
        api.spec_distill(x, ids, t, top_lse=lse, grad_loss=gl, out=api.DistillOutputs(
            torch.empty_like(gl), None, buf[8:].view(s.shape)))
    with pytest.raises(api.VerifyError):
        api.spec_distill(s, ids, t, float("nan"), top_lse=lse)
    with pytest.raises(api.VerifyError):  # a gradient asked for without a place for it
        api.spec_distill(s, ids, t, grad_loss=gl, out=api.DistillOutputs(torch.empty_like(gl)))


def test_graph_replays_over_new_inputs():
    s, ids, t, lse, gl = case(8, 4, 32000, 32, BF16, 1.0, True, 13)
    api.spec_distill(s, ids, t, top_lse=lse, grad_loss=gl)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fwd = api.spec_distill(s, ids, t, top_lse=lse)
        grad = api.spec_distill_grad(s, ids, t, 1.0, fwd.stats, gl, top_lse=lse)
    for seed in (14, 15):
        new = case(8, 4, 32000, 32, BF16, 1.0, True, seed)
        for a, b in zip((s, ids, t, lse, gl), new):
            a.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        want = api.spec_distill(s, ids, t, top_lse=lse, grad_loss=gl)
        assert torch.equal(want.loss, fwd.loss)
        plain.check_distill(s[:1], ids[:1], t[:1], lse[:1], 1.0, gl[:1], None, fwd.loss[:1],
                            grad[:1])


def test_verify_record_distill_a_draft_head():
    """The loop these operators are for: a verify call's target logits and accept lengths give
    the record, the record trains a draft head; its weight gradient equals float64 autograd's."""
    B, K, V, H = 6, 3, 2000, 32
    g = gen(16)
    target = (torch.randn((B, K + 1, V), generator=g, device="cuda") * 3).to(BF16)
    drafts = target[:, :K].argmax(-1).to(torch.int32)
    drafts[2, 1] = (drafts[2, 1] + 1) % V
    u = torch.rand((B, K + 1), generator=g, device="cuda")
    out = api.spec_verify_sample(target, None, drafts, u, 1.0)
    rec = api.spec_top_logits(target, 24, 1.0, lens=out.accept_len)
    hid = torch.randn((B, K + 1, H), generator=g, device="cuda")
    head = (torch.randn((H, V), generator=g, device="cuda") * 0.1).requires_grad_()
    gl = torch.full((B, K + 1), 1.0 / int(out.accept_len.sum()), device="cuda")
    logits = hid @ head
    res = api.spec_distill(logits.detach(), rec.ids, rec.logits, top_lse=rec.lse,
                           lens=out.accept_len, grad_loss=gl)
    logits.backward(res.grad)
    h64 = head.detach().double().requires_grad_()
    q = torch.log_softmax(hid.double() @ h64, -1)
    need = torch.arange(K + 1, device="cuda")[None] < out.accept_len[:, None]
    ids = rec.ids.long().clamp(min=0)
    p = torch.where(need[..., None], (rec.logits.double() - rec.lse.double()[..., None]).exp(), 0)
    p = torch.nan_to_num(p)
    rest = (1 - p.sum(-1)).clamp(min=0)
    outside = torch.ones_like(q).scatter(-1, ids, 0.0)
    q_rest = torch.log((q.exp() * outside).sum(-1))
    loss = -(p * q.gather(-1, ids)).sum(-1) - rest * q_rest
    torch.where(need, loss, 0.0).mul(gl.double()).sum().backward()
    # each row's gradient is within 3 SUM of |grad_loss|, the head sums B (K+1) rows of |hid| <= 5
    tol = 5 * float(gl.sum()) * 3 * plain.SUM + 1e-5 * float(h64.grad.abs().max())
    assert float((head.grad.double() - h64.grad).abs().max()) <= tol


def test_wait_limit_runs_out():
    s, ids, t, lse, gl = case(2, 3, 5001, 8, BF16, 1.0, True, 20)
    fwd = api.spec_distill(s, ids, t, top_lse=lse)
    old = api.wait_limit_ns()
    try:
        api.set_wait_limit_ns(0)
        out = api.spec_distill(s, ids, t, top_lse=lse, grad_loss=gl)
        grad = api.spec_distill_grad(s, ids, t, 1.0, fwd.stats, gl, top_lse=lse)
        torch.cuda.synchronize()
    finally:
        api.set_wait_limit_ns(old)
    assert bool((out.status == api.REQ_TIMEOUT).all()) and bool(torch.isnan(out.loss).all())
    assert not bool(out.grad.any()) and bool(torch.isnan(grad).all())
    check(s, ids, t, lse, 1.0, gl)


def test_offsets_past_32_bits():
    """More than 2^31 student logits: the last rows, and the gradient in place."""
    B, V = 14200, 152064
    s = torch.zeros((B, 1, V), dtype=BF16, device="cuda")
    tail, ids, t, lse, gl = case(2, 1, V, 8, BF16, 1.0, True, 30)
    s[-2:] = tail
    ids = torch.cat([torch.full((B - 2, 1, 8), -1, dtype=torch.int32, device="cuda"), ids])
    t = torch.cat([torch.zeros((B - 2, 1, 8), device="cuda"), t])
    lse = torch.cat([torch.zeros((B - 2, 1), device="cuda"), lse])
    gl = torch.cat([torch.ones((B - 2, 1), device="cuda"), gl])
    out = api.DistillOutputs(torch.empty((B, 1), device="cuda"), None, s)
    api.spec_distill(s, ids, t, top_lse=lse, grad_loss=gl, out=out)
    plain.check_distill(tail, ids[-2:], t[-2:], lse[-2:], 1.0, gl[-2:], None, out.loss[-2:],
                        s[-2:])
    assert not bool(out.loss[:-2].any()) and not bool(s[:-2].any())


def test_two_streams_at_once():
    """Calls on different streams share nothing."""
    cases = [case(64, 4, 32000, 32, BF16, 1.0, True, 40 + i) for i in range(2)]
    want = [api.spec_distill(s, ids, t, top_lse=lse, grad_loss=gl)
            for s, ids, t, lse, gl in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i, ((s, ids, t, lse, gl), st) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(st):
                got[i] = api.spec_distill(s, ids, t, top_lse=lse, grad_loss=gl)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.loss, b.loss) and torch.equal(a.grad, b.grad)


@pytest.mark.parametrize("tail", [True, False])
@pytest.mark.parametrize("shift", [0.0, 2.0 ** 10, -(2.0 ** 20)])
def test_shifted_rows(tail, shift):
    """Student and teacher far from zero and from each other: the loss is of the differences
    (on a grid that the shifted rows hold exactly)."""
    T = 2.0 ** -7 if shift else 1.0
    s, ids, t, lse, gl = case(2, 3, 1500, 24, F32, 1.0, tail, 13)
    s, t = (s * 8).round() / 8, (t * 8).round() / 8
    if tail:  # some log-sum-exp above the record's own
        lse = (t.double().amax(-1) / T + math.log(24)).ceil().float()
    one = check(s, ids, t, lse, T, gl)
    far = check(s + shift, ids, t, lse, T, gl)
    assert torch.equal(one.loss, far.loss) and torch.equal(one.grad, far.grad)
    if not tail:
        far = check(s, ids, t - shift, None, T, gl)
        assert torch.equal(one.loss, far.loss) and torch.equal(one.grad, far.grad)


@pytest.mark.parametrize("tail", [True, False])
@pytest.mark.parametrize("T", [1.0, 0.5])
def test_lowest_value_students(T, tail):
    """Masks of the type's lowest value: in a whole row, at a recorded token and its like
    outside the record, and everywhere outside the record."""
    low = torch.finfo(F32).min
    s, ids, t, lse, gl = case(1, 3, 2000, 10, F32, T, tail, 14)
    s[0, 0] = low
    s[0, 1, 500:] = torch.where(s[0, 1, 500:] > 0, s[0, 1, 500:], torch.full_like(s[0, 1, 500:], low))
    s[0, 1, ids[0, 1, 3].long()] = low
    keep = s[0, 2, ids[0, 2].long()].clone()
    s[0, 2] = low
    s[0, 2, ids[0, 2].long()] = keep
    out = api.spec_distill(s, ids, t, T, top_lse=lse, grad_loss=gl)
    back = api.spec_distill_grad(s, ids, t, T, out.stats, gl, top_lse=lse)
    x, d, r = plain.f64(s), ids.cpu(), plain.f64(t)
    plain.check_distill(s, ids, t, lse, T, gl, None, None, out.grad, out.status)
    plain.check_distill(s, ids, t, lse, T, gl, None, None, back)
    for i in range(3):
        L, size = plain.distill_row(x[0, i], d[0, i], r[0, i],
                                    float(lse[0, i]) if tail else None, T)[:2]
        # each p and the remainder of them within 2^-20, times the largest |log q|
        worst = -low / T if size > 1e30 else 0.0
        tol = 2.0 ** -20 * (size + 32 + worst) + 2 * plain.SUM
        assert abs(float(out.loss[0, i]) - L) <= tol, (i, out.loss, L, tol)
    assert float(out.loss[0, 0]) < 40 and float(out.loss[0, 1]) > 1e30
    assert (float(out.loss[0, 2]) > 1e30) == tail


@pytest.mark.parametrize("T", [1e-40, 1e-38, 1e-20, 1e30])
def test_extreme_temperatures(T):
    """The largest and smallest: both sides certain of the same token, or both uniform."""
    T = float(torch.tensor(T, dtype=F32))  # as the kernel gets it
    s, ids, t, _, gl = case(1, 2, 1000, 6, F32, 1.0, False, 15)
    best = ids[0, :, 0].long()
    s[0, torch.arange(2), best] = 50.0
    both = check(s, ids, t, None, T, gl)
    assert bool(torch.isfinite(both.loss).all()) and bool(torch.isfinite(both.grad).all())
