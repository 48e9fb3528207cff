"""Attention steps of no tokens: nothing to compute, but every request has a status."""
import pytest
import torch

from test_cache_abi import FAKE, NULL, attend, lib  # noqa: F401
from token_verification_gb300 import api

OK, BAD_LEN, BAD_PAGE = 0, api.REQ_BAD_DRAFT_LEN, api.REQ_BAD_PAGE


def test_lengths_are_needed_for_statuses(lib):  # noqa: F811
    assert attend(lib, N=0, q=None, lens=None) == OK
    assert attend(lib, N=0, q=None, lens=None, st=FAKE) == NULL


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,Hq", [(64, 2), (128, 48), (256, 4)])
def test_statuses(D, Hq, dtype):
    cache = api.spec_cache_alloc(3, 2, D, 16)
    table = ints([[0, 1], [2, 7], [-1, 0], [9, 9], [1, 1], [0, 0]])
    lens = ints([32, 16, 1, 0, 33, -1])
    want = [OK, OK, BAD_PAGE, OK, BAD_LEN, BAD_LEN]
    q = torch.empty((6, 0, Hq, D), dtype=dtype, device="cuda")
    for junk in (77, -1):
        hold = [torch.full((6,), junk, dtype=torch.int32, device="cuda") for _ in range(50)]
        del hold
        res = api.spec_cache_attention(q, cache, table, lens, lse=True)
        assert res.out.shape == q.shape and res.status.tolist() == want
        out = api.AttentionOutputs(q.clone(), None, ints([junk] * 6))
        api.spec_cache_attention(q, cache, table, lens, out)
        assert out.status.tolist() == want
        api.spec_cache_attention(q, cache, table, lens, out, q_lens=ints([0, 1, 0, -1, 0, 0]))
        assert out.status.tolist() == [OK, BAD_LEN, BAD_PAGE, BAD_LEN, BAD_LEN, BAD_LEN]
    # pages behind a window are not looked at
    table = ints([[7, 0]] * 3000)
    res = api.spec_cache_attention(q[:1].expand(3000, 0, Hq, D), cache, table, ints([32] * 3000), window=10)
    assert not bool(res.status.any())
