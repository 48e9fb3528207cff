"""Sizes past what the 4-bit cache's operators count in 32 bits are refused before any
CUDA call (no GPU)."""
import pytest

from test_cache_abi import lib, read, write  # noqa: F401

SHAPE, SLOTS = 2, 1 << 27
ROW = 64 * 2


@pytest.mark.parametrize("N", [SLOTS + 1, SLOTS + 64, 1 << 30, (1 << 31) - 8, (1 << 31) - 1])
def test_steps_longer_than_any_request(lib, N):  # noqa: F811
    """A request holds SV_MAX_SLOTS slots at most: slot numbers near a longer step's end wrapped."""
    kw = dict(B=1, H=1, D=64, N=N, ks=(0, ROW, 0), vs=(0, ROW, 0))
    assert read(lib, **kw) == SHAPE
    assert write(lib, **kw) == SHAPE
    kw.update(ks=(0, 0, 0), vs=(0, 0, 0))  # (one token's keys and values for every slot)
    assert write(lib, **kw) == SHAPE
