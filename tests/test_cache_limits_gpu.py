"""The 4-bit cache's operators at their limits: offsets past 32 bits, the longest
context, many requests, caches without pages, waits that run out (needs a GPU)."""
import math

import pytest
import torch

import plain_cache as plain
from test_cache_attention_gpu import BF16, F32, filled, gen, ints, query, run, spoil, tree
from token_verification_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,group", [(5, 4), (40, 2), (61, 4)])
def test_wait_limit_runs_out(N, group, D):
    """More rows than 16 wait for the tensor cores; when a wait runs out every row is NaN and every
    request says so, and the next call is right again."""
    g = gen(N + D)
    B, H, page = 7, 2, 16
    lens = ints([N, 300, 2000, N + 1, 77, 5000, 900])
    cache, table = filled(B, 5000, H, D, page, g)
    q = query(B, N, H * group, D, BF16, g)
    parent = tree(B, N, g)
    old = api.wait_limit_ns()
    try:
        api.set_wait_limit_ns(0)
        chain = api.spec_cache_attention(q, cache, table, lens, lse=True)
        nodes = api.spec_cache_attention(q, cache, table, lens, lse=True, parent=parent)
        torch.cuda.synchronize()
    finally:
        api.set_wait_limit_ns(old)
    for out in (chain, nodes):
        assert bool((out.status == api.REQ_TIMEOUT).all())
        assert bool(out.out.isnan().all()) and bool(out.lse.isnan().all())
    run(q, cache, page, table, lens)
    run(q, cache, page, table, lens, parent=parent)


def test_few_rows_wait_for_nothing():
    g = gen(3)
    cache, table = filled(2, 500, 2, 128, 16, g)
    old = api.wait_limit_ns()
    try:
        api.set_wait_limit_ns(0)
        run(query(2, 2, 16, 128, BF16, g), cache, 16, table, ints([500, 60]))
    finally:
        api.set_wait_limit_ns(old)


@pytest.mark.parametrize("pages,apart", [(20000, 278528), (3, 4000000000)])
def test_offsets_past_32_bits(pages, apart):
    """Pages behind 4 GB, close together and far apart, through all four calls."""
    g = gen(pages)
    B, H, D, page, L = 1, 8, 128, 256, 500
    size = api.spec_cache_alloc(1, H, D, page)[0].numel()
    assert size <= apart
    room = torch.empty((pages - 1) * apart + size, dtype=torch.uint8, device="cuda")
    far = room.as_strided((pages, H, 2, size // H // 2), (apart, size // H, size // H // 2, 1))
    near = api.spec_cache_alloc(2, H, D, page)
    here, there = ints([[0, 1]]), ints([[pages - 1, pages - 2]])
    kv = torch.randn((2, B, L, H, D), generator=g, device="cuda").to(BF16)
    zero = ints([0])
    for cache, table in ((near, here), (far, there)):
        api.spec_cache_write(cache, kv[0], kv[1], table, zero)
    assert torch.equal(near[0], far[pages - 1])
    for N, group in ((2, 4), (20, 4)):
        q = query(B, N, H * group, D, BF16, g)
        a = api.spec_cache_attention(q, near, here, ints([L]))
        b = api.spec_cache_attention(q, far, there, ints([L]))
        assert torch.equal(a.out, b.out) and not bool(b.status.any())
        plain.check_attention(q, near, page, here, ints([L]), b.out)
    path = ints([[0, 3, 9, -1]])
    for cache, table in ((near, here), (far, there)):
        api.spec_cache_keep(cache, table, ints([250]), path, D)
    for x, y in zip(api.spec_cache_read(near, here, L, D), api.spec_cache_read(far, there, L, D)):
        assert torch.equal(x, y)


def test_dense_offsets_past_32_bits():
    """Requests, tokens and heads whose rows lie 4 GB apart, in and out."""
    g = gen(1)
    H, D, page = 2, 64, 16
    room = torch.zeros(3 * (1 << 31) + 4096, dtype=BF16, device="cuda")
    x = torch.randn((2, 2, 2, H, D), generator=g, device="cuda").to(BF16)
    for order in ((0, 1, 2), (1, 0, 2), (2, 1, 0)):  # (which dimension is the wide one)
        st = [0] * 3
        for i, s in zip(order, (1 << 31, 256, 128)):
            st[i] = s
        far = [room.as_strided((2, 2, H, D), (*st, 1), o) for o in (0, 1 << 10)]
        cache, table = filled(2, 32, H, D, page, g)
        for f, y in zip(far, x):
            f.copy_(y)
        near = cache.clone()
        api.spec_cache_write(near, x[0], x[1], table, ints([5, 20]))
        api.spec_cache_write(cache, far[0], far[1], table, ints([5, 20]))
        assert torch.equal(near, cache)
        want = api.spec_cache_read(cache, table, 2, D, start=ints([5, 20]))
        for f in far:
            f.zero_()
        api.spec_cache_read(cache, table, 2, D, far[0], far[1], start=ints([5, 20]))
        assert torch.equal(far[0], want[0]) and torch.equal(far[1], want[1])
        q = room.as_strided((2, 2, H, D), (*st, 1))
        q.copy_(x[0])
        a = api.spec_cache_attention(x[0], cache, table, ints([7, 22]))
        b = api.spec_cache_attention(q, cache, table, ints([7, 22]))
        assert torch.equal(a.out, b.out)


@pytest.mark.parametrize("group", [4, 24])
def test_longest_context(group):
    """2^27 slots, which all lie in one page: attention is that over the page's 256 slots, the sum
    of the weights 2^19 times it."""
    g = gen(group)
    D, page, many = 64, 256, 1 << 19
    cache, _ = filled(1, page, 1, D, page, g)
    table = torch.zeros((1, many), dtype=torch.int32, device="cuda")
    q = query(1, 1, group, D, BF16, g)
    out = api.spec_cache_attention(q, cache, table, ints([page * many]), lse=True)
    assert out.status.tolist() == [0]
    sees, depth = plain.ancestors(None, 1)
    dec = plain.decode(cache, page, D)
    kv = plain.slots(dec, ints([0]), page)
    o, lse, tol, ltol = plain.attention(q[0].cpu().double(), kv, page - 1, sees, depth, D ** -0.5, 0.0,
                                        0, None, BF16, 2.0 ** -32)
    # An accumulator takes 2^27 slots, 16 at a time, over 152 CTAs or more: 2^15.8 additions, each
    # off by at most a last place of the sum so far (2^-23 of it): 2^-7 of the sum of the magnitudes
    W = kv[:, 0, 1].abs().max()
    assert bool(((out.out[0].cpu().double() - o).abs() <= tol + 2.0 ** -7 * W).all())
    off = (out.lse[0].cpu().double() - lse - math.log(many)).abs()
    assert bool((off <= ltol + 2.0 ** -7 + 2.0 ** -19).all())


@pytest.mark.parametrize("B,N,group,D,dtype", [(300, 5, 4, 64, BF16), (513, 2, 4, 128, BF16),
                                               (270, 3, 2, 64, F32), (700, 17, 1, 128, BF16)])
def test_many_requests(B, N, group, D, dtype):
    """More requests than threads of a block, some with nothing but their step."""
    g = gen(B)
    page = 16
    lens = torch.randint(N, 150, (B,), generator=g, device="cuda").int()
    lens[::7] = N
    cache, table = filled(B, 150, 1, D, page, g)
    spoil(cache, table, lens, page, D)
    run(query(B, N, group, D, dtype, g), cache, page, table, lens, parent=tree(B, N, g))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", [17, 32, 33, 48, 49, 96, 97, 127, 128, 129, 144, 145, 192, 255, 256, 257])
def test_tiles_of_rows(rows, D):
    """Every tile's last row, on a chain and on a tree; one request of several chunks, one of one."""
    g = gen(rows + D)
    cache, table = filled(2, 400, 2, D, 32, g)
    lens = ints([400, rows])
    spoil(cache, table, lens, 32, D)
    q = query(2, rows, 2, D, BF16, g)
    run(q, cache, 32, table, lens)
    run(q, cache, 32, table, lens, parent=tree(2, rows, g), window=90)


@pytest.mark.parametrize("Hq,Hkv,dtype", [(1024, 1, BF16), (1024, 1024, BF16), (1024, 1, F32),
                                          (1000, 8, BF16)])
def test_many_heads(Hq, Hkv, dtype):
    g = gen(Hq + Hkv)
    cache, table = filled(2, 70, Hkv, 64, 16, g)
    run(query(2, 1, Hq, 64, dtype, g), cache, 16, table, ints([70, 1]))


@pytest.mark.parametrize("N", [1, 30])
def test_no_pages(N):
    """A cache of no pages: rows that would see any are NaN, nothing is touched."""
    g = gen(2)
    cache = api.spec_cache_alloc(0, 2, 64, 16)
    table = torch.zeros((3, 4), dtype=torch.int32, device="cuda")
    q = query(3, N, 4, 64, BF16, g)
    out = api.spec_cache_attention(q, cache, table, ints([N, 60, 64]))
    assert out.status.tolist() == [api.REQ_BAD_PAGE] * 3 and bool(out.out.isnan().all())
    st = ints([0, 0, 0])
    k = torch.zeros((3, N, 2, 64), device="cuda")
    api.spec_cache_write(cache, k, k, table, ints([0, 1, 2]), status=st)
    assert st.tolist() == [api.REQ_BAD_PAGE] * 3
    a, b = api.spec_cache_read(cache, table, 5, 64)
    assert not bool(a.any()) and not bool(b.any())
    path = ints([[0, 1]] * 3)
    api.spec_cache_keep(cache, table, ints([0, 0, 0]), path, 64, status=st)
    assert st.tolist() == [api.REQ_BAD_PAGE] * 3


def test_no_slots_at_all():
    """Tables without columns: steps of no tokens are fine, others are refused by a status."""
    cache = api.spec_cache_alloc(2, 2, 64, 16)
    table = torch.zeros((2, 0), dtype=torch.int32, device="cuda")
    q = torch.ones((2, 3, 4, 64), dtype=BF16, device="cuda")
    out = api.spec_cache_attention(q, cache, table, ints([0, 3]), q_lens=ints([0, 3]), lse=True)
    assert out.status.tolist() == [0, api.REQ_BAD_DRAFT_LEN]
    assert not bool(out.out.any()) and bool((out.lse[1] == -math.inf).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("softcap,scale", [(1e-39, 0.1), (1e-39, 0.0), (1e-30, 5.0), (350.0, 0.1),
                                           (511.0, 0.1), (1e6, 0.1), (1e30, 0.1)])
def test_caps_of_any_size(softcap, scale, dtype):
    g = gen(int(softcap) % 1000 + 1)
    for N, group in ((2, 2), (7, 4)):
        cache, table = filled(2, 300, 2, 64, 16, g)
        q = query(2, N, 2 * group, 64, dtype, g)
        run(q, cache, 16, table, ints([300, 40]), softcap=softcap, scale=scale)


@pytest.mark.parametrize("group", [1, 8])
def test_one_query_for_all(group):
    """A query that is broadcast over requests and tokens."""
    g = gen(group)
    cache, table = filled(4, 400, 2, 128, 32, g)
    lens = ints([400, 30, 129, 5])
    q = query(1, 1, 2 * group, 128, BF16, g).expand(4, 5, 2 * group, 128)
    a = api.spec_cache_attention(q, cache, table, lens)
    b = api.spec_cache_attention(q.contiguous(), cache, table, lens)
    assert torch.equal(a.out, b.out)
    plain.check_attention(q, cache, 32, table, lens, a.out)


def test_versions_and_inference_tensors():
    """Autograd learns of what is written; tensors of inference mode are taken."""
    g = gen(4)
    cache, table = filled(1, 32, 2, 64, 16, g)
    k = torch.randn((1, 2, 2, 64), generator=g, device="cuda")
    v0 = cache._version
    api.spec_cache_write(cache, k, k, table, ints([3]))
    v1 = cache._version
    api.spec_cache_keep(cache, table, ints([3]), ints([[0, 1]]), 64)
    v2 = cache._version
    assert v0 < v1 < v2
    api.spec_cache_read(cache, table, 4, 64)
    out = api.AttentionOutputs(torch.zeros((1, 2, 4, 64), device="cuda"))
    w0 = out.out._version
    api.spec_cache_attention(torch.randn((1, 2, 4, 64), generator=g, device="cuda"), cache, table,
                             ints([5]), out)
    assert cache._version == v2 and out.out._version > w0
    with torch.inference_mode():
        c2 = cache.clone()
        api.spec_cache_write(c2, k, k, table, ints([3]))
        api.spec_cache_keep(c2, table, ints([3]), ints([[0, 1]]), 64)
        got = api.spec_cache_attention(torch.ones((1, 1, 2, 64), device="cuda"), c2, table, ints([5]))
        assert got.status.tolist() == [0]


def test_long_way_agrees():
    """The calls that go by way of Python (a status to write, given outputs) give the same bits."""
    g = gen(6)
    for N, dtype in ((1, BF16), (3, F32), (24, BF16)):
        cache, table = filled(3, 200, 2, 128, 16, g)
        other = cache.clone()
        k = torch.randn((3, N, 2, 128), generator=g, device="cuda").to(dtype)
        st = ints([1, 1, 1])
        start = ints([0, 17, 100])
        api.spec_cache_write(cache, k, k + 1, table, start)
        api.spec_cache_write(other, k, k + 1, table, start, status=st)
        assert torch.equal(cache, other) and not bool(st.any())
        q = query(3, N, 6, 128, dtype, g)
        lens = start + N
        parent = tree(3, N, g) if N > 1 else None
        kw = dict(parent=parent, softcap=9.0, window=20, slopes=torch.ones(6, device="cuda"), scale=0.2)
        a = api.spec_cache_attention(q, cache, table, lens, lse=True, **kw)
        out = api.AttentionOutputs(torch.empty_like(q), torch.empty_like(a.lse), torch.empty_like(st))
        b = api.spec_cache_attention(q, cache, table, lens, out, **kw)
        assert b is out and torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)
        assert torch.equal(a.status, b.status)
        x = api.spec_cache_read(cache, table, 90, 128, dtype=dtype)
        y = api.spec_cache_read(cache, table, 90, 128, dtype=dtype, status=st)
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_refusals_on_the_device():
    g = gen(7)
    cache, table = filled(2, 40, 2, 64, 16, g)
    q = query(2, 3, 4, 64, BF16, g)
    lens, k = ints([10, 20]), torch.zeros((2, 3, 2, 64), device="cuda")
    bad_value = [
        lambda: api.spec_cache_attention(q, cache, table[:1], lens),
        lambda: api.spec_cache_attention(q, cache, table, lens[:1]),
        lambda: api.spec_cache_attention(q, cache, table, None),
        lambda: api.spec_cache_attention(q[:, :, :3], cache, table, lens),
        lambda: api.spec_cache_attention(q.transpose(2, 3), cache, table, lens),
        lambda: api.spec_cache_attention(q, cache, table, lens, parent=ints([0])),
        lambda: api.spec_cache_attention(q, cache, table, lens, slopes=torch.ones(3, device="cuda")),
        lambda: api.spec_cache_attention(q, cache[:, :, :1], table, lens),
        lambda: api.spec_cache_attention(q, cache[..., :-1], table, lens),
        lambda: api.spec_cache_attention(q[..., 1:], cache, table, lens),
        lambda: api.spec_cache_write(cache, k, k[:1], table, lens),
        lambda: api.spec_cache_write(cache, k, k, table, None),
        lambda: api.spec_cache_write(cache, k[:, :, :1], k[:, :, :1], table, lens),
        lambda: api.spec_cache_write(cache, k.cpu(), k, table, lens),
        lambda: api.spec_cache_write(cache, torch.zeros(2 * 3 * 2 * 64 + 1, device="cuda")[1:].view(
            2, 3, 2, 64), k, table, lens),
        lambda: api.spec_cache_read(cache, table, -1, 64),
        lambda: api.spec_cache_read(cache, table, 3, 96),
        lambda: api.spec_cache_read(cache, table, 3, 64, k),
        lambda: api.spec_cache_keep(cache, table, None, ints([[0], [0]]), 64),
        lambda: api.spec_cache_keep(cache, table, lens, ints([0, 0]), 64),
    ]
    bad_type = [
        lambda: api.spec_cache_attention(q.half(), cache, table, lens),
        lambda: api.spec_cache_attention(q, cache.float(), table, lens),
        lambda: api.spec_cache_attention(q, cache, table.long(), lens),
        lambda: api.spec_cache_attention(q, cache, table, lens.long()),
        lambda: api.spec_cache_write(cache, k, k.to(BF16), table, lens),
        lambda: api.spec_cache_write(cache, k, k, table, lens.long()),
        lambda: api.spec_cache_keep(cache, table, lens, ints([[0], [0]]).long(), 64),
    ]
    refused = [
        lambda: api.spec_cache_attention(q, cache, table, lens, scale=math.inf),
        lambda: api.spec_cache_attention(q, cache, table, lens, softcap=-1.0),
        lambda: api.spec_cache_attention(q, cache, table, lens, softcap=math.nan),
        lambda: api.spec_cache_attention(q, cache, table, lens, window=-1),
        lambda: api.spec_cache_attention(q[:, :1].expand(2, 258, 4, 64), cache, table, lens),
        lambda: api.spec_cache_read(cache, table, 3, 64, k[:1].expand(2, 3, 2, 64), k.clone()),
    ]
    for kind, calls in ((ValueError, bad_value), (TypeError, bad_type), (api.VerifyError, refused)):
        for i, call in enumerate(calls):
            with pytest.raises(kind):
                call()
                raise AssertionError((kind, i))
