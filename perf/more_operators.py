"""Cases and plain forms of the operators of a 4-bit key/value cache around the
verification step: writing keys and values into the cache's pages and reading
them back, keeping a verified tree's path, and attention of a step's tokens
(one token, a chain of drafts, a candidate tree) over the cache.

`run` computes an operator in elementary torch operations, or with `own` set
makes the framework's calls.

The cache is bytes [pages, kv heads, 2 (keys, values), page bytes].  A page holds
`page` tokens of a head: D / 2 bytes of codes a token, in words of 8 values
(value i of a word in its nibble i // 2 + 4 (i % 2)), then scale bytes
[page / 16, D / 32, 16], one for each 32 values of a token.  A scale byte c is the scale
s = (1 + c % 8 / 8) 2^(c // 8 - 20), the least with 7 s >= the group's largest magnitude
(c <= 238), and a code q + 8 with q = the value / s to the nearest whole number, ties to
even, kept within -7..7.
"""
import math

import torch

own = False

TORCH_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ESIZE = {"bf16": 2, "f32": 4}
TOP_BYTE = 238  # scale 896


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _attend(name, B, N, Hq, Hkv, D, L, page, dtype="bf16", ragged=True, tree=False, softcap=0.0,
            window=0, bias=False):
    case = dict(op="attend", B=B, N=N, Hq=Hq, Hkv=Hkv, D=D, L=L, page=page, dtype=dtype,
                ragged=ragged, tree=tree, softcap=softcap, window=window, bias=bias)
    return dict(name=name, **case) if name else case


def _store(name, B, N, Hkv, D, page, dtype="bf16", ragged=False, read_only=False):
    case = dict(op="store", B=B, N=N, Hkv=Hkv, D=D, page=page, dtype=dtype, ragged=ragged,
                read_only=read_only)
    return dict(name=name, **case) if name else case


def _keep(name, B, N, P, Hkv, D, page, dtype="bf16"):
    case = dict(op="keep", B=B, N=N, P=P, Hkv=Hkv, D=D, page=page, dtype=dtype)
    return dict(name=name, **case) if name else case


def listed():
    return [
        # one request's single token, a short context: the latency of a drafting step
        _attend("attend_token", 1, 1, 32, 8, 128, 1000, 16, ragged=False),
        # a serving batch of single tokens (a draft layer, or a step without drafts)
        _attend("attend_decode", 256, 1, 32, 8, 128, 4096, 64),
        # the verification step of a serving batch: 5 drafts and the last token
        _attend("attend_chain", 64, 6, 64, 8, 128, 8192, 64),
        # the 60-node candidate tree of a batch of 32, each node seeing its ancestors
        _attend("attend_tree", 32, 61, 32, 8, 128, 4096, 64, tree=True),
        # one request's drafts over a very long context
        _attend("attend_long", 1, 4, 64, 8, 128, 131072, 256, ragged=False),
        # wide heads with capped scores and a sliding window
        _attend("attend_capped", 16, 5, 16, 8, 256, 8192, 32, softcap=50.0, window=4096),
        # fp32, heads in groups of three, scores biased by distance, an odd length
        _attend("attend_odd_f32", 7, 3, 12, 4, 64, 5003, 16, dtype="f32", bias=True),
        # a step's keys and values into the cache, and back
        _store("store_step", 256, 6, 8, 128, 64),
        # the same of whole prompts
        _store("store_prompt", 8, 8192, 8, 128, 64, ragged=True),
        # a cached prefix read back for a dense kernel
        _store("store_prefix", 4, 32768, 8, 128, 256, read_only=True),
        # one request's tree: its nodes written, the accepted path kept and read back
        _keep("keep_one", 1, 61, 6, 8, 128, 16),
        # the same of a serving batch
        _keep("keep_batch", 128, 61, 6, 8, 128, 64),
    ]


MOST_VALUES = 3 << 28           # keys' values of an attention call's cache
MOST_STORED = 1 << 26           # keys' values of a store
MOST_PRODUCTS = 20_000_000_000  # of queries and keys, over the head dimension


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "store", "keep"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    page = rng.choice([16, 32, 64, 128, 256])
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    if op == "store":
        B = _spread(rng, 1, 256)
        most = MOST_STORED // (B * Hkv * D) // (2 if dtype == "f32" else 1)
        N = _spread(rng, 1, max(1, min(16384, most)))
        return _store("", B, N, Hkv, D, page, dtype, rng.random() < 0.5, rng.random() < 0.3)
    if op == "keep":
        N = _spread(rng, 2, 129)
        return _keep("", _spread(rng, 1, 128), N, rng.randint(2, min(N, 9)), Hkv, D, page, dtype)
    B = _spread(rng, 1, 256)
    tree = rng.random() < 0.3
    N = _spread(rng, 2, 128) if tree else rng.choice([1, 1, rng.randint(2, 8)])
    group = rng.choice([1, 2, 4, 4, 5, 8])
    most = min(MOST_VALUES // (B * Hkv * D),
               MOST_PRODUCTS // (B * Hkv * group * N * D) // (4 if dtype == "f32" else 1))
    L = _spread(rng, 1, max(1, min(131072, most)))
    return _attend("", B, N, Hkv * group, Hkv, D, max(L, N), page, dtype, rng.random() < 0.7, tree,
                   rng.choice([0.0, 0.0, 30.0]), rng.choice([0, 0, 0, _spread(rng, 1, L)]),
                   rng.random() < 0.2)


def _lens(case):
    """Tokens of each request, evenly spaced in (L / 2, L], the step's own among them."""
    B, L = case["B"], case["L"]
    if not case["ragged"]:
        return [L] * B
    return [max(case["N"], math.ceil(L * (0.5 + 0.5 * (b + 1) / B))) for b in range(B)]


def _counts(case):
    """Tokens that each request stores: N, or evenly spaced in (0, N]."""
    B, N = case["B"], case["N"]
    return [math.ceil(N * (b + 1) / B) if case["ragged"] else N for b in range(B)]


def work(case):
    D, Hkv, e = case["D"], case["Hkv"], ESIZE[case["dtype"]]
    token = 2 * Hkv * (D // 2 + D // 32)  # a cached token's bytes
    values = 2 * Hkv * D
    if case["op"] == "attend":
        seen = sum(min(n, case["window"] + case["N"] - 1) if case["window"] else n
                   for n in _lens(case))
        rows = case["B"] * case["N"] * case["Hq"]
        return {"bytes": seen * token + 2 * rows * D * e,
                "flops": 4 * seen * case["N"] * case["Hq"] * D}
    if case["op"] == "store":
        n = sum(_counts(case))
        if case["read_only"]:
            return {"bytes": n * (token + values * e), "flops": 0}
        return {"bytes": 2 * n * (token + values * e), "flops": 2 * n * values}
    n, kept = case["B"] * case["N"], case["B"] * case["P"]
    return {"bytes": n * (token + values * e) + kept * (3 * token + values * e),
            "flops": 2 * n * values}


# ---------------------------------------------------------------------------
# the cache's format, in torch
# ---------------------------------------------------------------------------

def _quantised(x):
    """(codes 1..15, scale bytes, values) of fp32 [..., D]."""
    g = x.unflatten(-1, (-1, 32))
    top = g.abs().amax(dim=-1, keepdim=True)
    byte = ((top / 7).view(torch.int32) >> 20) - 856   # the scale's exponent and three bits below
    byte = byte.clamp(min=0, max=TOP_BYTE)
    byte = (byte + (7 * _scale(byte) < top)).clamp(max=TOP_BYTE)
    scale = _scale(byte)
    q = (g / scale).round().clamp(-7, 7)
    return (q + 8).to(torch.uint8).flatten(-2), byte[..., 0].to(torch.uint8), (q * scale).flatten(-2)


def _scale(byte):
    return ((byte.int() + 856) << 20).view(torch.float32)


def _codes_packed(c):
    w = c.unflatten(-1, (-1, 8))
    return (w[..., [0, 4, 1, 5]] | (w[..., [2, 6, 3, 7]] << 4)).flatten(-2)


def _values(codes, scales):
    """fp32 [..., D] of packed codes [..., D / 2] and scale bytes [..., D / 32]."""
    w = codes.unflatten(-1, (-1, 4))
    low, high = (w & 15).float() - 8, (w >> 4).float() - 8
    v = torch.stack([low[..., 0], low[..., 2], high[..., 0], high[..., 2],
                     low[..., 1], low[..., 3], high[..., 1], high[..., 3]], dim=-1)
    v = v.flatten(-2).unflatten(-1, (-1, 32)) * _scale(scales)[..., None]
    return v.flatten(-2)


def _parts(cache, page, D):
    """Views of a cache: codes [pages, heads, 2, page, D / 2] and scale bytes
    [pages, heads, 2, page / 16, D / 32, 16]."""
    n = page * D // 2
    return (cache[..., :n].unflatten(-1, (page, D // 2)),
            cache[..., n:].unflatten(-1, (page // 16, D // 32, 16)))


def _empty_cache(pages, Hkv, page, D):
    size = page * (D // 2 + D // 32)
    return torch.zeros((pages, Hkv, 2, size), dtype=torch.uint8, device="cuda")


def _slots(s, first, count):
    """(page ids, slots in the page) [B, count] of slots first[b].. of each request."""
    at = first.long()[:, None] + torch.arange(count, device=first.device)
    inside = at.clamp(max=s["table"].shape[1] * s["page"] - 1)
    return s["table"].long().gather(1, inside // s["page"]), inside % s["page"]


def _put(s, first, count, x, take):
    """Quantises x [B, count, 2, Hkv, D] into slots first[b].. where take [B, count]."""
    codes, scales = _parts(s["cache"], s["page"], s["D"])
    c, b, _ = _quantised(x)
    page, slot = (i[take] for i in _slots(s, first, count))
    codes[page, :, :, slot] = _codes_packed(c)[take].transpose(1, 2)
    scales[page, :, :, slot // 16, :, slot % 16] = b[take].transpose(1, 2)


def _get(s, first, count):
    """fp32 [B, count, 2, Hkv, D] of slots first[b].. of each request."""
    codes, scales = _parts(s["cache"], s["page"], s["D"])
    page, slot = _slots(s, first, count)
    x = _values(codes[page, :, :, slot], scales[page, :, :, slot // 16, :, slot % 16])
    return x.transpose(2, 3)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(shape, g, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _shuffled(values, g):
    v = torch.tensor(values, dtype=torch.int32, device="cuda")
    return v[torch.randperm(len(values), generator=g, device="cuda")].contiguous()


def _filled(cache, page, D, g):
    """Fills a cache with the quantised keys and values of a trained layer's spread: some
    channels of the keys larger than others."""
    codes, scales = _parts(cache, page, D)
    wide = torch.exp(0.7 * _randn((cache.shape[1], 1, D), g))
    step = max(1, (1 << 26) // (cache.shape[1] * page * D))
    for at in range(0, cache.shape[0], step):
        for part in (0, 1):
            c, b, _ = _quantised(_randn(codes[at:at + step, :, part, :, :1].shape[:-1] + (D,), g)
                                 * (wide if part == 0 else 1.0))
            codes[at:at + step, :, part] = _codes_packed(c)
            scales[at:at + step, :, part] = b.unflatten(2, (-1, 16)).transpose(-1, -2)


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    B, N, Hkv, D, page = (case[x] for x in ("B", "N", "Hkv", "D", "page"))
    t = TORCH_TYPES[case["dtype"]]
    if case["op"] == "attend":
        lens = _lens(case)
        start = [0] * B
    elif case["op"] == "store":
        lens = [0] * B if case["read_only"] else [(37 * b) % 200 for b in range(B)]
        start, lens = lens, [x + N for x in lens]
    else:
        start = [(53 * b) % 1000 for b in range(B)]
        lens = [x + N for x in start]
    width = -(-max(lens) // page)
    pages = B * width + 3
    s["cache"] = _empty_cache(pages, Hkv, page, D)
    order = torch.randperm(pages, generator=g, device="cuda")[:B * width]
    s["table"] = order.to(torch.int32).view(B, width).contiguous()
    if case["op"] == "attend":
        Hq = case["Hq"]
        _filled(s["cache"], page, D, g)
        s["lens"] = _shuffled(lens, g)
        s["q"] = (1.5 * _randn((B, N, Hq, D), g)).to(t)
        s["parent"] = s["slopes"] = None
        if case["tree"]:
            # candidate nodes hang under one of the eleven nodes before them
            r = torch.rand((B, N - 1), generator=g, device="cuda")
            n = torch.arange(1, N, device="cuda")
            back = 1 + (r * n.clamp(max=11)).int()
            s["parent"] = (n - torch.minimum(back, n)).to(torch.int32).contiguous()
        if case["bias"]:
            s["slopes"] = torch.exp2(-8.0 * torch.arange(1, Hq + 1, device="cuda") / Hq)
        return s
    s["start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
    if case["op"] == "store":
        s["counts"] = _shuffled(_counts(case), g)
    else:
        # an accepted path: ascending nodes from the root on, some shorter than P
        ids = torch.rand((B, N - 1), generator=g, device="cuda").argsort(dim=1)
        ids = (ids[:, :case["P"] - 1] + 1).sort(dim=1).values
        path = torch.cat([torch.zeros_like(ids[:, :1]), ids], dim=1).to(torch.int32)
        kept = _shuffled([1 + b % case["P"] if B > 1 else case["P"] for b in range(B)], g)
        path[torch.arange(case["P"], device="cuda") >= kept[:, None]] = -1
        s["path"], s["kept"] = path, kept
    if case["op"] == "store" and case["read_only"]:
        _filled(s["cache"], page, D, g)
        return s
    # keys and values as a layer's projection leaves them: beside each other in a row
    s["kv"] = _randn((B, N, 2, Hkv, D), g, t)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _ancestors(parent):
    """(sees [B, N, N], depth [B, N]) of trees of N - 1 nodes under a root."""
    B, n = parent.shape
    sees = torch.zeros((B, n + 1, n + 1), dtype=torch.bool, device=parent.device)
    depth = torch.zeros((B, n + 1), dtype=torch.int64, device=parent.device)
    sees[:, 0, 0] = True
    at = torch.arange(B, device=parent.device)
    for i in range(1, n + 1):
        up = parent[:, i - 1].long()
        sees[:, i] = sees[at, up]
        sees[:, i, i] = True
        depth[:, i] = depth[at, up] + 1
    return sees, depth


def _plain_attend_part(s, rows, sees, depth):
    """Attention of requests `rows` (a slice)."""
    N, Hq, Hkv, D = s["N"], s["Hq"], s["Hkv"], s["D"]
    part = dict(s, table=s["table"][rows])
    lens = s["lens"][rows].long()
    L = s["L"]
    first = torch.zeros_like(lens)
    x = _get(part, first, L)                                    # [b, L, 2, Hkv, D]
    k, v = x[:, :, 0].permute(0, 2, 3, 1), x[:, :, 1].transpose(1, 2)
    q = s["q"][rows].float().transpose(1, 2).unflatten(1, (Hkv, Hq // Hkv))
    score = (q.flatten(2, 3) @ k).unflatten(2, (Hq // Hkv, N)) * (1.0 / math.sqrt(D))
    if s["softcap"]:
        score = s["softcap"] * torch.tanh(score / s["softcap"])
    slot = torch.arange(L, device=lens.device)
    base = lens - N                                             # the root's slot
    node = slot[None, :] - base[:, None]                        # [b, L], a key's node or < 0
    here = torch.arange(N, device=lens.device)
    if sees is None:
        seen = node[:, None, :] <= here[None, :, None]
        key_at, query_at = slot[None, :].expand_as(node), base[:, None] + here
    else:
        nodes = node.clamp(0, N - 1)
        seen = (node < 0)[:, None, :] | sees[rows].gather(2, nodes[:, None, :].expand(-1, N, -1))
        d = depth[rows]
        key_at = torch.where(node < 0, slot[None, :], base[:, None] + d.gather(1, nodes))
        query_at = base[:, None] + d
    seen = seen & (slot[None, :] < lens[:, None])[:, None, :]
    far = query_at[:, :, None] - key_at[:, None, :]             # [b, N, L]
    if s["window"]:
        seen = seen & (far < s["window"])
    if s["slopes"] is not None:
        slopes = s["slopes"].view(Hkv, Hq // Hkv)
        score = score - slopes[None, :, :, None, None] * far[:, None, None].float()
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(dim=-1, keepdim=True)
    e = torch.exp(score - top)
    o = (e.flatten(2, 3) @ v).unflatten(2, (Hq // Hkv, N)) / e.sum(dim=-1, keepdim=True)
    return o.flatten(1, 2).transpose(1, 2).to(s["q"].dtype)


def _plain_attend(s):
    sees, depth = _ancestors(s["parent"]) if s["parent"] is not None else (None, None)
    out = torch.empty_like(s["q"])
    one = s["L"] * max(s["Hq"] * s["N"], 2 * s["Hkv"] * s["D"])
    step = max(1, (1 << 29) // one)
    for b in range(0, s["B"], step):
        rows = slice(b, b + step)
        out[rows] = _plain_attend_part(s, rows, sees, depth)
    return out


def _plain_store(s):
    t = TORCH_TYPES[s["dtype"]]
    take = torch.arange(s["N"], device="cuda")[None, :] < s["counts"][:, None]
    if not s["read_only"]:
        _put(s, s["start"], s["N"], s["kv"].float(), take)
    x = _get(s, s["start"], s["N"]) * take[:, :, None, None, None]
    return {"k": x[:, :, 0].to(t), "v": x[:, :, 1].to(t)}


def _plain_keep(s):
    t = TORCH_TYPES[s["dtype"]]
    every = torch.ones((s["B"], s["N"]), dtype=torch.bool, device="cuda")
    _put(s, s["start"], s["N"], s["kv"].float(), every)
    codes, scales = _parts(s["cache"], s["page"], s["D"])
    take = s["path"] >= 0
    page, slot = _slots(s, s["start"], s["N"])
    path = s["path"].long().clamp(min=0)
    p, i = page.gather(1, path)[take], slot.gather(1, path)[take]
    c, b = codes[p, :, :, i], scales[p, :, :, i // 16, :, i % 16]
    page, slot = (x[take] for x in _slots(s, s["start"], s["P"]))
    codes[page, :, :, slot] = c
    scales[page, :, :, slot // 16, :, slot % 16] = b
    x = _get(s, s["start"], s["P"]) * take[:, :, None, None, None]
    return {"k": x[:, :, 0].to(t), "v": x[:, :, 1].to(t)}


PLAIN = {"attend": _plain_attend, "store": _plain_store, "keep": _plain_keep}


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _own(s):
    from token_verification_gb300 import api
    cache, table, t = s["cache"], s["table"], TORCH_TYPES[s["dtype"]]
    if s["op"] == "attend":
        return api.spec_cache_attention(s["q"], cache, table, s["lens"], parent=s["parent"],
                                        softcap=s["softcap"], window=s["window"],
                                        slopes=s["slopes"]).out
    if s["op"] == "store":
        if not s["read_only"]:
            api.spec_cache_write(cache, s["kv"][:, :, 0], s["kv"][:, :, 1], table, s["start"],
                                 lens=s["counts"])
        k, v = api.spec_cache_read(cache, table, s["N"], s["D"], start=s["start"],
                                   lens=s["counts"], dtype=t)
    else:
        api.spec_cache_write(cache, s["kv"][:, :, 0], s["kv"][:, :, 1], table, s["start"])
        api.spec_cache_keep(cache, table, s["start"], s["path"], s["D"])
        k, v = api.spec_cache_read(cache, table, s["P"], s["D"], start=s["start"], lens=s["kept"],
                                   dtype=t)
    return {"k": k, "v": v}


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _table64():
    """Every scale, in 64 bits."""
    return torch.tensor([(1 + c % 8 / 8) * 2.0 ** (c // 8 - 20) for c in range(TOP_BYTE + 1)],
                        dtype=torch.float64, device="cuda")


def _exact_values(x):
    """What [..., D] is held as, in 64 bits: the least scale that reaches the group's top."""
    scales = _table64()
    g = x.double().unflatten(-1, (-1, 32))
    top = g.abs().amax(-1)
    at = torch.searchsorted(7 * scales, top).clamp(max=TOP_BYTE)
    s = scales[at][..., None]
    return (torch.round(g / s).clamp(-7, 7) * s).flatten(-2)


def _exact_token(s, b, slots, heads):
    """[len(slots), len(heads), 2, D] in 64 bits, decoded nibble by nibble."""
    page, D = s["page"], s["D"]
    flat, size = s["cache"].flatten(), s["cache"].shape[-1]
    here = s["table"][b].long()[slots // page]
    block = (here[:, None, None] * s["Hkv"] + heads[:, None]) * 2 + torch.arange(2, device="cuda")
    block = (block * size)[..., None]                             # [n, heads, 2, 1]
    at = (slots % page)[:, None, None, None]
    d = torch.arange(D, device="cuda")
    i = d % 8
    nibble = i // 2 + 4 * (i % 2)
    byte = flat[block + at * (D // 2) + d // 8 * 4 + nibble // 2]
    q = ((byte >> (4 * (nibble % 2)).to(torch.uint8)) & 15).double() - 8
    byte = flat[block + page * D // 2 + (at // 16 * (D // 32) + d // 32) * 16 + at % 16]
    return q * _table64()[byte.long()]


def _exact_attend(s):
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lens = s["lens"].tolist()
    parents = s["parent"].tolist() if s["parent"] is not None else None
    N, Hq, Hkv = s["N"], s["Hq"], s["Hkv"]
    for b in range(s["B"]):
        n, base = lens[b], lens[b] - N
        # place[j]: the position of slot j; seen[i, j]: whether query i sees slot j
        place = torch.arange(n, device="cuda", dtype=torch.float64)
        seen = torch.ones((N, n), dtype=torch.bool)
        seen[:, base:] = False
        deep = [0] * N
        for i in range(N):
            at = i
            while True:
                seen[i, base + at] = True
                if at == 0:
                    break
                at = parents[b][at - 1] if parents else at - 1
                deep[i] += 1
        place[base:] = base + torch.tensor(deep, dtype=torch.float64)
        seen = seen.cuda()
        far = place[base:, None] - place
        if s["window"]:
            seen &= far < s["window"]
        for h in range(Hkv):
            kv = _exact_token(s, b, torch.arange(n, device="cuda"),
                              torch.tensor([h], device="cuda"))
            for j in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                x = s["q"][b, :, j].double() @ kv[:, 0, 0].T / math.sqrt(s["D"])
                if s["softcap"]:
                    x = s["softcap"] * torch.tanh(x / s["softcap"])
                if s["slopes"] is not None:
                    x = x - s["slopes"][j].double() * far
                x[~seen] = -math.inf
                out[b, :, j] = torch.softmax(x, dim=-1) @ kv[:, 0, 1]
    return out


def exact(case, seed):
    # (a key head at a time in 64 bits: long where there are many)
    if case["op"] == "attend" and case["B"] * case["L"] * case["Hq"] * case["N"] > 1 << 30:
        return None
    if case["op"] == "attend" and case["B"] * case["Hkv"] * case["Hq"] > 1 << 17:
        return None
    s = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(s)
    counts = (s["counts"] if case["op"] == "store" else s["kept"]).tolist()
    start = s["start"].tolist()
    P = case["N"] if case["op"] == "store" else case["P"]
    out = torch.zeros((case["B"], P, 2, case["Hkv"], case["D"]), dtype=torch.float64,
                      device="cuda")
    for b in range(case["B"]):
        n = counts[b]
        if case["op"] == "keep":
            out[b, :n] = _exact_values(s["kv"][b, s["path"][b, :n].long()])
        elif case["read_only"]:
            slots = start[b] + torch.arange(n, device="cuda")
            for h in range(case["Hkv"]):
                x = _exact_token(s, b, slots, torch.tensor([h], device="cuda"))
                out[b, :n, :, h] = x[:, 0]
        else:
            out[b, :n] = _exact_values(s["kv"][b, :n])
    return {"k": out[:, :, 0], "v": out[:, :, 1]}
