"""spec_distill refuses outputs over the rows' weights, which its CTAs read until
the end (host-side checks, no GPU)."""
import ctypes

import pytest

from token_verification_gb300 import _native, build

FAKE = 0x100000  # never dereferenced: every call below fails validation
ALIAS = 9
ROWS = 6  # 24 bytes of weights, losses and statuses, 96 of statistics


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _native.lib()


@pytest.mark.parametrize("over", ["loss", "stats", "status"])
@pytest.mark.parametrize("at", ["same", "first", "last"])
def test_outputs_over_the_weights(lib, over, at):
    weights = FAKE + 4096
    size = 16 * ROWS if over == "stats" else 4 * ROWS
    step = 16 if over == "stats" else 4
    place = {"same": weights, "first": weights - size + step, "last": weights + 4 * ROWS - 4}[at]
    if over == "stats":
        place -= place % 16
    outs = dict(loss=FAKE + 8192, stats=FAKE + 12288, status=FAKE + 16384)
    outs[over] = place
    code = lib.spec_distill(FAKE + 65536, FAKE, FAKE, None, None, weights, ctypes.c_float(1.0),
                            outs["loss"], outs["stats"], FAKE + 131072, outs["status"], 1, 2, 3,
                            100, 8, None)
    assert code == ALIAS
