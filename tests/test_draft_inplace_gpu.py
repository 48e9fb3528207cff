"""Outputs that the caller gives are written in place, and autograd is told so
(needs a GPU)."""
import pytest
import torch

from token_verification_gb300 import api

pytestmark = pytest.mark.gpu


def distill_inputs():
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    leaf = torch.randn((2, 3, 500), generator=g, device="cuda", requires_grad=True)
    rec = api.spec_top_logits(torch.randn((2, 3, 500), generator=g, device="cuda"), 8)
    return leaf, rec, torch.ones((2, 3), device="cuda")


def test_gradient_over_logits_that_autograd_saved():
    """exp keeps its result for its own backward pass: a gradient written over it is noticed."""
    leaf, rec, gl = distill_inputs()
    y = leaf.exp()
    loss = y.square().sum()
    out = api.DistillOutputs(torch.empty_like(gl), torch.empty((2, 3, 4), device="cuda"), y.detach())
    api.spec_distill(y.detach(), rec.ids, rec.logits, top_lse=rec.lse, grad_loss=gl, out=out)
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()
    leaf, rec, gl = distill_inputs()
    y = leaf.exp()
    loss = y.square().sum()
    fwd = api.spec_distill(y.detach(), rec.ids, rec.logits, top_lse=rec.lse)
    api.spec_distill_grad(y.detach(), rec.ids, rec.logits, 1.0, fwd.stats, gl, grad=y.detach(),
                          top_lse=rec.lse)
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()


@pytest.mark.parametrize("with_status", [False, True])  # the compiled binding, the long way
def test_states_that_autograd_saved(with_status):
    leaf = torch.randn((1, 2, 3, 1, 1, 8), device="cuda", requires_grad=True)
    y = leaf.exp()
    loss = y.square().sum()
    state = torch.randn((1, 2, 3, 1, 1, 8), device="cuda")
    p = torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    status = torch.empty(2, dtype=torch.int32, device="cuda") if with_status else None
    api.spec_beam_reorder(state, p, y.detach(), status=status)
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()


def test_versions_of_given_outputs():
    x = torch.randn((2, 3, 1000), device="cuda")
    out = api.spec_top_logits(x, 9)
    was = [t._version for t in (out.ids, out.logits, out.lse, out.status)]
    api.spec_top_logits(x, 9, out=out)
    assert [t._version for t in (out.ids, out.logits, out.lse, out.status)] == [v + 1 for v in was]
    sel = api.spec_beam_select(x, torch.zeros((2, 3), device="cuda"), 4)
    was = [t._version for t in (sel.tokens, sel.parents, sel.scores, sel.status)]
    api.spec_beam_select(x, torch.zeros((2, 3), device="cuda"), 4, out=sel)
    assert [t._version for t in (sel.tokens, sel.parents, sel.scores, sel.status)] == [
        v + 1 for v in was]
    assert x._version == 0


def test_inference_tensors_are_taken():
    """They have no version; a call that writes into them is as good as any."""
    with torch.inference_mode():
        state = torch.randn((1, 2, 3, 1, 1, 8), device="cuda")
        p = torch.tensor([[2, 1, 0], [0, 0, 1]], dtype=torch.int32, device="cuda")
        status = torch.empty(2, dtype=torch.int32, device="cuda")
        for st in (None, status):
            out = torch.zeros_like(state)
            api.spec_beam_reorder(state, p, out, status=st)
            assert torch.equal(out[0, 0], state[0, 0, p[0].long()])
        x = torch.randn((2, 3, 1000), device="cuda")
        a = api.spec_top_logits(x, 9)
        b = api.spec_top_logits(x, 9, out=api.TopLogits(*(torch.empty_like(t) for t in (
            a.ids, a.logits, a.lse, a.status))))
        assert torch.equal(a.ids, b.ids)
