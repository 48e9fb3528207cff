"""spec_cache_attention against the plain form (tests/plain_cache.py), and a step
through write, attention, verification and the kept path (needs a GPU)."""
import math

import pytest
import torch

import plain_cache as plain
from token_verification_gb300 import api

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def filled(B, slots, H, D, page, g, spare=1, wide=1.0):
    """(cache, table) of random keys and values in every slot of every page, the spare pages'
    bytes all ones."""
    M = -(-slots // page)
    n = B * M + spare
    table = torch.randperm(n - spare, generator=g, device="cuda").int().view(B, M).contiguous()
    cache = api.spec_cache_alloc(n, H, D, page)
    if B * M:
        x = torch.randn((2, B, M * page, H, D), generator=g, device="cuda") * wide
        api.spec_cache_write(cache, x[0], x[1], table, torch.zeros(B, dtype=torch.int32, device="cuda"))
    cache[n - spare:] = 255
    return cache, table


def spoil(cache, table, lens, page, D):
    """Every byte of every slot behind a request's last becomes 255 (never read)."""
    codes = cache[..., :page * D // 2].unflatten(-1, (page, D // 2))
    scales = cache[..., page * D // 2:].unflatten(-1, (page // 16, D // 32, 16))
    for b in range(table.shape[0]):
        for slot in range(int(lens[b]), table.shape[1] * page):
            p, t = int(table[b, slot // page]), slot % page
            if t == 0:
                cache[p] = 255
            codes[p, :, :, t] = 255
            scales[p, :, :, t // 16, :, t % 16] = 255


def tree(B, N, g, chain=False):
    n = torch.arange(1, N, device="cuda")
    if chain:
        return (n - 1).int().expand(B, N - 1).contiguous()
    r = torch.rand((B, N - 1), generator=g, device="cuda")
    return (n - 1 - (r * n.clamp(max=7)).int()).int().contiguous()


def run(q, cache, page, table, lens, **kw):
    out = api.spec_cache_attention(q, cache, table, lens, lse=True, **kw)
    torch.cuda.synchronize()
    assert not bool(out.status.any())
    plain.check_attention(q, cache, page, table, lens, out.out, out.lse, **kw)
    again = api.spec_cache_attention(q, cache, table, lens, lse=True, **kw)
    for x, y in ((again.out, out.out), (again.lse, out.lse)):  # (bit for bit, NaN as well)
        assert torch.equal(x.isnan(), y.isnan()) and torch.equal(x.nan_to_num(), y.nan_to_num())
    return out


def query(B, N, Hq, D, dtype, g, wide=1.5):
    return (torch.randn((B, N, Hq, D), generator=g, device="cuda") * wide).to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("N,Hq,Hkv", [(1, 1, 1), (1, 8, 2), (3, 6, 2), (5, 12, 4), (7, 5, 1),
                                      (6, 32, 4), (40, 16, 2)])
def test_heads(N, Hq, Hkv, D, dtype):
    """Groups of 1 to 8 heads and rows of one tile to many; lengths from the step's own on."""
    g = gen(N * Hq + D)
    page = 16
    lens = ints([N, N + 1, N + 15, 131, 300])
    cache, table = filled(5, 320, Hkv, D, page, g)
    spoil(cache, table, lens, page, D)
    run(query(5, N, Hq, D, dtype, g), cache, page, table, lens)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 31, 33, 64, 127, 128, 129, 255, 257, 511, 1000])
def test_lengths(L, page, dtype):
    g = gen(L + page)
    for N, Hq, Hkv, D in ((1, 4, 2, 128), (min(L, 9), 8, 2, 64), (min(L, 9), 16, 1, 128)):
        lens = ints([L, max(N, L // 2)])
        cache, table = filled(2, L, Hkv, D, page, g)
        spoil(cache, table, lens, page, D)
        run(query(2, N, Hq, D, dtype, g), cache, page, table, lens)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kw", [
    dict(softcap=20.0), dict(softcap=0.5, scale=1.0), dict(window=1), dict(window=33),
    dict(window=100000), dict(slopes=True), dict(softcap=30.0, window=50, slopes=True, scale=0.3),
    dict(scale=0.0), dict(scale=-0.2)])
def test_scores(kw, D, dtype):
    """Caps, windows and biases, on a chain and on a tree."""
    g = gen(D + len(kw))
    for N, Hq, Hkv in ((1, 4, 2), (6, 8, 2), (19, 8, 1)):
        B, page = 2, 32
        kw = dict(kw)
        if kw.get("slopes") is not None:
            kw["slopes"] = torch.exp2(-8 * torch.rand(Hq, generator=g, device="cuda"))
        lens = ints([N + 100, 277])
        cache, table = filled(B, 277, Hkv, D, page, g)
        q = query(B, N, Hq, D, dtype, g)
        run(q, cache, page, table, lens, **kw)
        if N > 1:
            run(q, cache, page, table, lens, parent=tree(B, N, g), **kw)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,N,Hq,Hkv,D,L", [
    (3, 2, 4, 2, 64, 2), (2, 61, 8, 2, 128, 61), (2, 61, 8, 1, 128, 500), (1, 257, 4, 2, 64, 700),
    (2, 257, 2, 1, 128, 257), (2, 33, 3, 3, 256, 200), (2, 128, 8, 2, 128, 1111)])
def test_trees(B, N, Hq, Hkv, D, L, dtype):
    """Nodes see their ancestors; NaN in a node reaches its descendants alone; a chain as a tree;
    one tree for the batch."""
    g = gen(N + L)
    page = 64
    cache, table = filled(B, L, Hkv, D, page, g)
    lens = ints([L - (b * (L - N)) // B for b in range(B)])
    q = query(B, N, Hq, D, dtype, g)
    parent = tree(B, N, g)
    run(q, cache, page, table, lens, parent=parent)
    run(q, cache, page, table, lens, parent=parent[0].contiguous())
    a = run(q, cache, page, table, lens, parent=tree(B, N, g, chain=True))
    b = run(q, cache, page, table, lens)
    assert torch.equal(a.out, b.out)
    node = N // 2
    x = torch.full((B, 1, Hkv, D), math.nan, device="cuda")
    api.spec_cache_write(cache, x, x, table, lens - N + node)
    out = run(q, cache, page, table, lens, parent=parent)
    for i in range(B):
        sees, _ = plain.ancestors(parent[i].cpu(), N)
        assert torch.equal(torch.isnan(out.out[i]).any(-1).any(-1).cpu(), sees[:, node])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_ragged_steps(dtype):
    """Steps of 0 to N tokens: rows behind them as they were, empty requests among them."""
    g = gen(11)
    for N, Hq, Hkv, D in ((6, 8, 2, 128), (30, 8, 1, 128), (6, 4, 4, 256)):
        B, page = 7, 16
        q_lens = ints([N, 0, 1, N - 1, 0, 2, 0])
        lens = ints([200, 0, 1, 77, 55, 2, 0])
        cache, table = filled(B, 208, Hkv, D, page, g)
        spoil(cache, table, lens, page, D)
        q = query(B, N, Hq, D, dtype, g)
        for parent in (None, tree(B, N, g)):
            given = api.AttentionOutputs(torch.full((B, N, Hq, D), 3.0, device="cuda", dtype=dtype),
                                         torch.full((B, N, Hq), 4.0, device="cuda"),
                                         torch.full((B,), 9, dtype=torch.int32, device="cuda"))
            before = given.out.clone()
            out = api.spec_cache_attention(q, cache, table, lens, given, q_lens=q_lens, parent=parent)
            assert out is given and not bool(out.status.any())
            plain.check_attention(q, cache, page, table, lens, out.out, out.lse, q_lens=q_lens,
                                  parent=parent, before=before)
            for b in range(B):
                assert bool((out.lse[b, int(q_lens[b]):] == 4).all())
            fresh = api.spec_cache_attention(q, cache, table, lens, q_lens=q_lens, parent=parent)
            for b in range(B):
                n = int(q_lens[b])
                assert torch.equal(fresh.out[b, :n], out.out[b, :n]) and not bool(fresh.out[b, n:].any())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_data_errors(dtype):
    """Lengths out of range, parents that are no tree: rows 0; pages that are none: NaN; the others
    in place."""
    g = gen(12)
    B, N, Hq, Hkv, D, page = 8, 4, 8, 2, 128, 16
    cache, table = filled(B, 96, Hkv, D, page, g)
    q = query(B, N, Hq, D, dtype, g)
    good = ints([50, 60, 70, 80, 50, 60, 70, 80])
    parent = tree(B, N, g)
    lens = good.clone()
    lens[1], lens[2], lens[3] = 3, 97, -1
    bad_tree = parent.clone()
    bad_tree[4, 1] = 2
    bad_tree[5, 2] = -1
    bad_table = table.clone()
    bad_table[6, 2] = cache.shape[0]
    bad_table[7, 5] = -7  # behind the last slot
    out = api.spec_cache_attention(q, cache, bad_table, lens, parent=bad_tree, lse=True)
    assert out.status.tolist() == [0, 4, 4, 4, 16, 16, 32, 0]
    for b in (0, 7):
        plain.check_attention(q[b:b + 1], cache, page, table[b:b + 1], good[b:b + 1],
                              out.out[b:b + 1], out.lse[b:b + 1], parent=parent[b:b + 1])
    assert not bool(out.out[1:6].any()) and bool((out.lse[1:6] == -math.inf).all())
    assert bool(torch.isnan(out.out[6]).all())
    # behind a window the page is not looked at
    out = api.spec_cache_attention(q, cache, bad_table, good, window=10)
    assert out.status.tolist() == [0] * 8 and bool(torch.isfinite(out.out).all())
    q_lens = ints([4, 5, -1, 4, 4, 4, 4, 4])
    out = api.spec_cache_attention(q, cache, table, good, q_lens=q_lens)
    assert out.status.tolist() == [0, 4, 4, 0, 0, 0, 0, 0]
    assert not bool(out.out[1:3].any())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_magnitudes(dtype):
    """Scores far apart and far from 0, values up to the format's largest and least."""
    g = gen(13)
    for wide, qw in ((30.0, 10.0), (1e-5, 1.0), (2000.0, 1e-3), (900.0, 5.0)):
        for N, Hq, Hkv, D in ((1, 4, 2, 128), (8, 8, 1, 128), (2, 2, 2, 256), (9, 4, 1, 64)):
            cache, table = filled(2, 333, Hkv, D, 16, g, wide=wide)
            run(query(2, N, Hq, D, dtype, g, qw), cache, 16, table, ints([333, 100]))


def test_not_finite_queries():
    """NaN and infinity in a query stay in its row."""
    g = gen(14)
    for dtype in (BF16, F32):
        for N, Hq, Hkv in ((2, 4, 2), (9, 8, 2)):
            cache, table = filled(1, 100, Hkv, 128, 16, g)
            q = query(1, N, Hq, 128, dtype, g)
            q[0, 0, 1, 5] = math.nan
            q[0, 1, 2, 127] = math.inf
            out = api.spec_cache_attention(q, cache, table, ints([100])).out
            nan = torch.isnan(out).any(-1)
            assert nan.nonzero().tolist() == [[0, 0, 1], [0, 1, 2]]
            assert bool(torch.isnan(out[nan]).all())


def test_strided_queries_and_layers():
    g = gen(15)
    for N in (3, 9):
        B, Hq, Hkv, D, page = 2, 8, 2, 128, 16
        cache, table = filled(B, 150, Hkv, D, page, g)
        pool = torch.full((cache.shape[0], 3) + cache.shape[1:], 255, dtype=torch.uint8, device="cuda")
        pool[:, 1] = cache
        qkv = query(B, N, Hq + 2 * Hkv, D, BF16, g)
        q = qkv[:, :, :Hq]
        lens = ints([150, 99])
        a = run(q.contiguous(), cache, page, table, lens)
        b = api.spec_cache_attention(q, pool[:, 1], table, lens)
        heads_first = q.transpose(1, 2).contiguous().transpose(1, 2)
        c = api.spec_cache_attention(heads_first, pool[:, 1], table, lens)
        assert torch.equal(a.out, b.out) and torch.equal(a.out, c.out)


@pytest.mark.parametrize("B,N,Hq,Hkv,D,L,dtype", [
    (1, 1, 8, 1, 128, 70001, BF16), (1, 5, 16, 2, 128, 40000, BF16), (300, 1, 2, 1, 64, 150, BF16),
    (40, 6, 16, 4, 128, 600, BF16), (2, 2, 2, 1, 256, 9000, F32), (1, 70, 8, 1, 128, 9000, BF16)])
def test_split(B, N, Hq, Hkv, D, L, dtype):
    """Requests in many pieces, and more requests than CTAs have threads."""
    g = gen(B + L)
    page = 256
    cache, table = filled(B, L, Hkv, D, page, g)
    lens = ints([max(N, L - (b * 37) % L) for b in range(B)])
    run(query(B, N, Hq, D, dtype, g), cache, page, table, lens)


def test_shared_prefix():
    """Requests whose tables name the same pages."""
    g = gen(16)
    cache, table = filled(4, 256, 2, 128, 64, g)
    table[1:, :2] = table[0, :2]
    run(query(4, 3, 8, 128, BF16, g), cache, 64, table, ints([256, 200, 131, 128]))


def test_streams_and_graphs():
    """Two captured graphs replayed at once on two streams, and eager calls beside them."""
    g = gen(17)
    sets = []
    for N, Hq in ((1, 8), (7, 16)):
        cache, table = filled(4, 2000, 2, 128, 64, g)
        q = query(4, N, Hq, 128, BF16, g)
        lens = ints([2000, 1500, 900, 70])
        want = run(q, cache, 64, table, lens).out
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        out = api.AttentionOutputs(torch.zeros_like(q))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            api.spec_cache_attention(q, cache, table, lens, out)
        sets.append((graph, torch.cuda.Stream(), q, cache, table, lens, out, want))
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, s, q, cache, table, lens, out, want in sets:
            with torch.cuda.stream(s):
                graph.replay()
                eager = api.spec_cache_attention(q, cache, table, lens).out
                assert torch.equal(eager, want)
    torch.cuda.synchronize()
    for graph, s, q, cache, table, lens, out, want in sets:
        assert torch.equal(out.out, want)


def test_a_verification_step():
    """A tree's step: its nodes' keys and values written, attention over them, the tree verified,
    the accepted path kept; the next step's attention equals that over a cache written token by
    token."""
    g = gen(18)
    B, N, Hq, Hkv, D, page, V = 5, 14, 8, 2, 128, 16, 96
    cache, table = filled(B, 160, Hkv, D, page, g)
    start = ints([100, 3, 0, 64, 33])
    kv = torch.randn((2, B, N, Hkv, D), generator=g, device="cuda").to(BF16)
    parent = tree(B, N, g)
    api.spec_cache_write(cache, kv[0], kv[1], table, start)
    q = query(B, N, Hq, D, BF16, g)
    att = run(q, cache, page, table, start + N, parent=parent)
    # logits from the attention's rows; each node proposes the argmax at its parent half of the time
    head = torch.randn((Hq * D, V), generator=g, device="cuda")
    logits = att.out.float().flatten(2) @ head
    tokens = torch.empty((B, N - 1), dtype=torch.int32, device="cuda")
    best = logits.argmax(-1).int()
    for n in range(1, N):
        guess = best.gather(1, parent[:, n - 1:n].long())[:, 0]
        keep = torch.rand(B, generator=g, device="cuda") < 0.6
        tokens[:, n - 1] = torch.where(keep, guess, (guess + n) % V)
    res = api.spec_verify_tree(logits, parent, tokens, N)
    assert int(res.accept_len.max()) > 2
    other = cache.clone()
    status = ints([9] * B)
    api.spec_cache_keep(cache, table, start, res.path, D, status=status)
    assert not bool(status.any())
    # the plain way: the accepted nodes alone, in order
    for b in range(B):
        n = int(res.accept_len[b])
        nodes = res.path[b, :n].long()
        api.spec_cache_write(other, kv[0][b:b + 1, nodes], kv[1][b:b + 1, nodes], table[b:b + 1],
                             start[b:b + 1])
    lens = start + res.accept_len
    ka, va = api.spec_cache_read(cache, table, 160, D, lens=lens)
    kb, vb = api.spec_cache_read(other, table, 160, D, lens=lens)
    assert torch.equal(ka, kb) and torch.equal(va, vb)
    q1 = query(B, 1, Hq, D, BF16, g)
    a, b = run(q1, cache, page, table, lens), run(q1, other, page, table, lens)
    assert torch.equal(a.out, b.out)
