"""Arguments of the 4-bit cache's operators that have more than 32 bits: what means something
keeps its meaning, the rest is refused."""
import pytest
import torch

from token_verification_gb300 import api, build

WIDE = 1 << 32


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("page,D", [(WIDE + 64, 64), (64, WIDE + 64), (WIDE + 64, WIDE + 128)])
def test_pages_of_no_such_size(page, D):
    with pytest.raises(api.VerifyError):
        api.spec_cache_alloc(1, 1, D, page, device="cpu")


@pytest.mark.gpu
def test_windows():
    """A window past every slot is none; a negative one is refused, of whatever size."""
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    cache = api.spec_cache_alloc(2, 1, 64, 16)
    table = ints([[1, 0]])
    kv = torch.randn((2, 1, 32, 1, 64), generator=g, device="cuda")
    api.spec_cache_write(cache, kv[0], kv[1], table, ints([0]))
    for N in (1, 24):
        q = torch.randn((1, N, 1, 64), generator=g, device="cuda").bfloat16()
        want = api.spec_cache_attention(q, cache, table, ints([32])).out
        for window in (32, (1 << 31) - 1, 1 << 31, WIDE, WIDE + 3, (1 << 63) - 1, 1 << 70):
            assert torch.equal(api.spec_cache_attention(q, cache, table, ints([32]), window=window).out, want)
        for window in (-1, -(1 << 31), 3 - WIDE, -(1 << 70)):
            with pytest.raises(api.VerifyError):
                api.spec_cache_attention(q, cache, table, ints([32]), window=window)


@pytest.mark.gpu
def test_steps_of_no_such_length():
    cache = api.spec_cache_alloc(1, 1, 64, 16)
    before = cache.clone()
    for N in (1 << 31, WIDE + 3):  # (one token's values at every place)
        k = torch.ones((1, 1, 1, 64), device="cuda").expand(1, N, 1, 64)
        with pytest.raises(api.VerifyError):
            api.spec_cache_write(cache, k, k, ints([[0]]), ints([0]))
        with pytest.raises(api.VerifyError):
            api.spec_cache_attention(k, cache, ints([[0]]), ints([3]))
    assert torch.equal(cache, before)
