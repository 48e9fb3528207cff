"""spec_top_logits against the plain 64-bit form (tests/plain_draft.py):
sizes from one token to whole vocabularies, odd rows and bases, ties, masked
and degenerate rows, padded batches, streams and graphs (needs a GPU)."""
import math

import pytest
import torch

import plain_draft as plain
from token_verification_gb300 import api

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def rows(shape, dtype, seed, scale=3.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def check(x, k, T=1.0, lens=None):
    d = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = api.spec_top_logits(x, k, T, lens=d)
    torch.cuda.synchronize()
    plain.check_top(x, k, T, out, lens)
    return out


@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 127, 255, 256, 257, 1000, 4095, 8191, 8192, 8193,
                               32000])
@pytest.mark.parametrize("k,dtype", [(1, BF16), (8, F32), (64, BF16), (128, F32)])
def test_sizes(V, k, dtype):
    check(rows((3, 2, V), dtype, V + k), k, T=0.7 if k == 8 else 1.0)


@pytest.mark.parametrize("B,P,V,k,dtype,T", [
    (2, 3, 152064, 64, BF16, 1.0), (1, 1, 152064, 128, F32, 2.0), (1, 1, 50001, 100, BF16, 1.0),
    (40, 4, 50001, 33, F32, 0.5), (330, 1, 5003, 5, BF16, 1.0), (1, 2, 700001, 50, BF16, 1.0)])
def test_large(B, P, V, k, dtype, T):
    check(rows((B, P, V), dtype, B + V), k, T)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shift", [1, 2, 3, 5, 7])
def test_unaligned_base(dtype, shift):
    buf = rows((3 * 2 * 2056 + shift,), dtype, shift)
    check(buf[shift:].view(3, 2, 2056), 20)


@pytest.mark.parametrize("V", [300, 20000])
def test_ties(V):
    """Constant rows, two values, coarse values, both zeros: the lowest tokens win."""
    x = rows((1, 6, V), F32, 1)
    x[0, 0] = 2.5
    x[0, 1] = (x[0, 1] > 0).float()
    x[0, 2] = x[0, 2].round()
    x[0, 3] = torch.where(x[0, 3] > 0, 0.0, -0.0)
    x[0, 4] = -7.25
    x[0, 5] = x[0, 5].mul(0.01).round().mul(100)
    for dtype in (BF16, F32):
        for k in (1, 64, 128):
            check(x.to(dtype), k)


def test_sorted_rows():
    x = rows((2, 2, 30000), F32, 2).sort(dim=-1).values
    x[1] = x[1].flip(-1)
    for dtype in (BF16, F32):
        for k in (5, 128):
            check(x.to(dtype), k)


def test_masked_rows():
    """Masked to few, to none, to a strided set (few threads hold all of it), to the
    type's lowest value; the record ends after the last finite logit."""
    x = rows((1, 7, 40000), F32, 3)
    n = -math.inf
    x[0, 0] = n
    x[0, 1, 1:] = n
    x[0, 2, :39990] = n
    keep = torch.zeros(40000, dtype=torch.bool, device="cuda")
    keep.view(-1, 8)[::250] = True
    x[0, 3][~keep] = n
    x[0, 4] = torch.finfo(BF16).min
    x[0, 5, 100:] = torch.finfo(BF16).min
    x[0, 6, ::2] = n
    for dtype in (BF16, F32):
        for k in (1, 100):
            check(x.to(dtype), k)


def test_bad_rows():
    x = rows((2, 4, 9000), F32, 4)
    x[0, 0, 8999] = math.nan
    x[0, 2, 17] = math.inf
    x[1, 3, 4000] = -math.nan
    for dtype in (BF16, F32):
        out = check(x.to(dtype), 30)
        assert int((out.status != 0).sum()) == 3


def test_lens():
    x = rows((6, 4, 3001), BF16, 5)
    x[1, 2:] = math.nan  # not read
    check(x, 12, lens=[4, 2, 0, 1, 5, -1])


def test_magnitudes():
    x = rows((1, 4, 5000), F32, 6)
    x[0, 0] *= 1e-30
    x[0, 1] *= 1e4
    x[0, 2] = x[0, 2] * 0.01 + 3e4
    x[0, 3, 7] = 80.0
    check(x, 50)
    check(x.to(BF16), 50)


def test_equal_rows_give_equal_sums():
    """Odd rows start at every alignment; their sums follow from their contents."""
    x = rows((1, 1, 5003), BF16, 7).expand(4, 9, 5003).contiguous()
    out = api.spec_top_logits(x, 3)
    assert int((out.lse != out.lse[0, 0]).sum()) == 0


def test_given_outputs_and_no_status():
    x = rows((2, 3, 1000), BF16, 8)
    a = api.spec_top_logits(x, 9, status=False)
    assert a.status is None
    out = api.TopLogits(torch.empty_like(a.ids), torch.empty_like(a.logits),
                        torch.empty_like(a.lse))
    assert api.spec_top_logits(x, 9, out=out) is out
    assert torch.equal(a.ids, out.ids) and torch.equal(a.lse, out.lse)
    with pytest.raises(ValueError):
        api.spec_top_logits(x, 8, out=out)
    with pytest.raises(ValueError):
        api.spec_top_logits(x.transpose(0, 1), 9)
    with pytest.raises(TypeError):
        api.spec_top_logits(x.half(), 9)
    for k in (0, 129, (1 << 32) + 5):
        with pytest.raises(api.VerifyError):
            api.spec_top_logits(x, k)
    with pytest.raises(api.VerifyError):
        api.spec_top_logits(x, 9, 0.0)
    empty = api.spec_top_logits(x[:0], 9)
    assert empty.ids.shape == (0, 3, 9)


def test_two_graphs_on_two_streams():
    """Captured calls hold nothing between them: two graphs replay at once, over new inputs."""
    xs = [rows((64, 6, 32000), BF16, 10 + i) for i in range(2)]
    outs, graphs, streams = [], [], []
    for x in xs:
        api.spec_top_logits(x, 40)
        g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=st):
            outs.append(api.spec_top_logits(x, 40))
        graphs.append(g)
        streams.append(st)
    for i, x in enumerate(xs):
        x.copy_(rows((64, 6, 32000), BF16, 20 + i))
    torch.cuda.synchronize()
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for x, out in zip(xs, outs):
        want = api.spec_top_logits(x, 40)
        assert torch.equal(out.ids, want.ids) and torch.equal(out.lse, want.lse)
        plain.check_top(x[:2], 40, 1.0, api.spec_top_logits(x[:2].contiguous(), 40))


def test_offsets_past_32_bits():
    """More than 2^31 logits: the first and last rows, through both kernels."""
    n = 14200
    x = torch.zeros((1, n, 152064), dtype=BF16, device="cuda")
    for i in (0, n - 1):
        x[0, i] = rows((152064,), BF16, i)
    out = api.spec_top_logits(x, 20)
    pick = torch.tensor([0, n - 1], device="cuda")
    few = api.TopLogits(out.ids[:, pick], out.logits[:, pick], out.lse[:, pick],
                        out.status[:, pick])
    plain.check_top(x[:, pick], 20, 1.0, few)
    assert bool((out.ids[0, 1:-1] == torch.arange(20, device="cuda")).all())
    x = torch.zeros((150, 1, 14500001), dtype=BF16, device="cuda")
    x[149] = rows((1, 14500001), BF16, 3)
    out = api.spec_top_logits(x, 3)
    few = api.TopLogits(out.ids[149:], out.logits[149:], out.lse[149:], out.status[149:])
    plain.check_top(x[149:], 3, 1.0, few)
