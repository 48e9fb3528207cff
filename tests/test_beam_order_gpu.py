"""The order of beam candidates whose scores in 64 bits are equal although
their logits are not: by beam, then by logit, then by token, whichever kernel
takes the call (needs a GPU).

With a score of -1e30 (a masked beam) or 1e9, score + log-probability is one
64-bit number for many tokens."""
import numpy as np
import pytest
import torch

from token_verification_gb300 import api

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
LOWEST = torch.finfo(F32).min


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def by_logit(row, n):
    return np.argsort(-row.double().cpu().numpy(), kind="stable")[:n]


# lists of candidates, lists that overflow, the row kernel (many bytes, or W > 8 below)
@pytest.mark.parametrize("B,V", [(1, 300), (2, 1000), (2, 2000), (1, 60000), (400, 40000)])
@pytest.mark.parametrize("score", [-1e30, LOWEST, 1e9, 3e7, -7.0])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_one_beam_keeps_its_largest_logits(B, V, score, dtype):
    """A single beam: whatever its score, the order of the logits, equal ones by token."""
    x = torch.randn((B, 1, V), generator=gen(V), device="cuda") * 3
    # close logits: neighbours in fp32, far below the resolution of 1e9 in 64 bits
    x[0, 0, ::7] = 1.0 + torch.arange(len(x[0, 0, ::7]), device="cuda") % 50 * 2.0 ** -23
    x = x.to(dtype)
    s = torch.full((B, 1), score, device="cuda")
    for n in (8, 128):
        out = api.spec_beam_select(x, s, n)
        assert not bool(out.status.any())
        for b in range(min(B, 3)):
            assert out.tokens[b].tolist() == by_logit(x[b, 0], n).tolist(), (b, n)
            assert out.parents[b].tolist() == [0] * n
        assert bool((out.scores[:, 1:] <= out.scores[:, :-1]).all())


@pytest.mark.parametrize("W", [2, 3, 8, 16, 64])
@pytest.mark.parametrize("V", [40, 500, 6000])
def test_masked_beams_tie_by_beam(W, V):
    """Beams of one far score are equal in every candidate: the first beam's come first, each
    beam's in the order of its logits; a beam of a better score comes before them."""
    x = torch.randn((3, W, V), generator=gen(W + V), device="cuda")
    s = torch.full((3, W), -1e30, device="cuda")
    s[1] *= torch.arange(1, W + 1, device="cuda")
    s[2, W - 1] = -2.0
    for n in (16, 128):
        out = api.spec_beam_select(x, s, n)
        assert not bool(out.status.any())
        for b, beams in enumerate([range(W), range(W), [W - 1, *range(W - 1)]]):
            want = [(w, t) for w in beams for t in by_logit(x[b, w], n).tolist()][:n]
            got = list(zip(out.parents[b].tolist(), out.tokens[b].tolist()))[:len(want)]
            assert got == want, (b, n)
