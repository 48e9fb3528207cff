"""Attention calls in flight together: kernels of every kind on streams of their own, eager and captured,
with nothing waiting on the host in between (needs a GPU)."""
import pytest
import torch

from test_cache_attention_gpu import BF16, F32, filled, gen, ints, query, run, tree
from token_verification_gb300 import api

pytestmark = pytest.mark.gpu
# (N, q heads, kv heads, D, type, tree): 32, 48 and 24 rows in tensor memory, 56, 136 and 244 in tiles of 128, and
# few rows, whose requests are split over many CTAs
CALLS = [(4, 16, 2, 64, BF16, False), (6, 16, 2, 128, BF16, True), (6, 8, 2, 64, BF16, False),
         (7, 16, 2, 64, BF16, False), (17, 16, 2, 128, BF16, True), (61, 8, 2, 128, BF16, True),
         (1, 8, 2, 128, BF16, False), (3, 4, 2, 256, BF16, True), (3, 8, 2, 128, F32, False)]


def prepared(call, g):
    N, Hq, Hkv, D, dtype, as_tree = call
    B, page = 4, 64
    cache, table = filled(B, 3000, Hkv, D, page, g)
    lens = ints([3000, 1500, 900, N])
    q = query(B, N, Hq, D, dtype, g)
    kw = dict(parent=tree(B, N, g)) if as_tree else {}
    want = run(q, cache, page, table, lens, **kw).out
    return (q, cache, table, lens), kw, want


def captured(args, kw, stream, pool=None):
    out = api.AttentionOutputs(torch.zeros_like(args[0]))
    graph = torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream, pool=pool):
        api.spec_cache_attention(*args, out, **kw)
    return graph, out


def test_all_kinds_at_once():
    g = gen(1)
    sets = []
    for call in CALLS:
        args, kw, want = prepared(call, g)
        s = torch.cuda.Stream()
        graph, out = captured(args, kw, s)
        sets.append((args, kw, want, s, graph, out))
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for i, (args, kw, want, s, graph, out) in enumerate(sets):
            with torch.cuda.stream(s):
                graph.replay()
                got.append((i, out.out.clone()))
                got.append((i, api.spec_cache_attention(*args, **kw).out))
    torch.cuda.synchronize()
    for i, x in got:
        assert torch.equal(x, sets[i][2]), CALLS[i]


@pytest.mark.parametrize("first", [0, 3, 6])
def test_one_kind_on_many_streams(first):
    """The same calls on eight streams: each has scratch of its own."""
    g = gen(first)
    prepared_calls = [prepared(c, g) for c in CALLS[first:first + 3]]
    streams = [torch.cuda.Stream() for _ in range(8)]
    torch.cuda.synchronize()
    got = []
    for turn in range(40):
        for n, s in enumerate(streams):
            i = (turn + n) % 3
            args, kw, _ = prepared_calls[i]
            with torch.cuda.stream(s):
                got.append((i, api.spec_cache_attention(*args, **kw).out))
    torch.cuda.synchronize()
    for i, x in got:
        assert torch.equal(x, prepared_calls[i][2]), CALLS[first + i]


def test_graphs_of_one_pool():
    """Graphs that share a memory pool, replayed one after the other, in another order than captured."""
    g = gen(3)
    s = torch.cuda.Stream()
    sets, pool = [], None
    for call in CALLS:
        args, kw, want = prepared(call, g)
        graph, out = captured(args, kw, s, pool)
        pool = pool or graph.pool()
        sets.append((graph, out, want, args, kw))  # (what a graph reads stays allocated)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for turn in range(5):
            for graph, out, *_ in sets[::-1] if turn % 2 else sets:
                out.out.zero_()
                graph.replay()
    torch.cuda.synchronize()
    for graph, out, want, *_ in sets:
        assert torch.equal(out.out, want)


def test_a_step_behind_another():
    """Write, attention and keep of successive steps on one stream, with no wait between them, give what each
    call gives alone: later calls start before earlier ones have ended."""
    g = gen(4)
    for N, Hq, D in ((6, 16, 128), (4, 16, 64), (17, 16, 128), (2, 4, 128)):
        B, Hkv, page, steps = 3, 2, 16, 12
        cache, table = filled(B, 400, Hkv, D, page, g)
        alone = cache.clone()
        start = ints([100, 3, 50])
        k = torch.randn((steps, B, N, Hkv, D), generator=g, device="cuda").to(BF16)
        q = query(steps * B, N, Hq, D, BF16, g).view(steps, B, N, Hq, D)
        path = ints([[0, N - 1, -1]] * B)
        torch.cuda.synchronize()
        out = []
        for c, wait in ((cache, False), (alone, True)):
            at, outs = start.clone(), []
            for i in range(steps):
                for call in (lambda: api.spec_cache_write(c, k[i], -k[i], table, at),
                             lambda: outs.append(api.spec_cache_attention(q[i], c, table, at + N).out),
                             lambda: api.spec_cache_keep(c, table, at, path, D)):
                    call()
                    if wait:
                        torch.cuda.synchronize()
                at = at + 2
            out.append(outs)
        torch.cuda.synchronize()
        assert torch.equal(cache, alone)
        for a, b in zip(*out):
            assert torch.equal(a, b)
