"""Cases and plain forms of the operators around the verification step: the
record of a teacher's top logits, distillation from it (forward and
backward), beam selection over beams and vocabulary, and the reordering of
per-beam states.

`run` computes an operator in elementary torch operations, or with `own` set
makes the framework's calls.
"""
import math

import torch

own = False

TORCH_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ESIZE = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one request's verified rows of a small-vocabulary model: the latency of a record
        dict(name="top_latency", op="top", B=1, P=4, V=32000, k=8, dtype="bf16", T=1.0),
        # the teacher's record of a full serving batch (256 requests, 5 drafts), rows up to
        # each request's accept length
        dict(name="top_serving", op="top", B=256, P=6, V=152064, k=64, dtype="bf16", T=1.0),
        # fp32 logits of an odd vocabulary (unaligned rows), a long record, a temperature
        dict(name="top_odd_f32", op="top", B=24, P=4, V=50001, k=100, dtype="f32", T=0.8),
        # a draft head's online update on one request, the record renormalised over its tokens
        dict(name="distill_online", op="distill", B=1, P=6, V=32000, k=16, dtype="bf16", T=1.0,
             tail=False, split=False),
        # a training batch of 2048 positions, loss and gradient in one call
        dict(name="distill_batch", op="distill", B=64, P=32, V=152064, k=64, dtype="bf16", T=1.0,
             tail=True, split=False),
        # the same with forward and backward apart, padded rows, a softer temperature
        dict(name="distill_split", op="distill", B=96, P=16, V=128256, k=32, dtype="bf16", T=2.0,
             tail=True, split=True),
        # fp32 training of an odd vocabulary
        dict(name="distill_odd_f32", op="distill", B=16, P=13, V=50001, k=100, dtype="f32", T=1.0,
             tail=True, split=True),
        # one request's draft tree, four beams: the latency of a drafting step
        dict(name="beam_latency", op="beam", B=1, W=4, V=32000, n=8, dtype="bf16", dead=0),
        # a serving batch's drafting step
        dict(name="beam_serving", op="beam", B=64, W=8, V=128256, n=16, dtype="bf16", dead=0),
        # wide beams of an odd vocabulary, some of them finished
        dict(name="beam_wide", op="beam", B=24, W=32, V=50001, n=64, dtype="f32", dead=7),
        # the accepted path of a candidate tree of 60 nodes, out of a draft layer's keys and values
        dict(name="reorder_path", op="reorder", G=2, B=32, W=61, Wo=5, H=8, L=1, D=128,
             dtype="bf16", layout="heads_first", ragged=False),
        # a draft layer's keys and values of 8 beams over prompts of up to 2048 tokens
        dict(name="reorder_cache", op="reorder", G=2, B=32, W=8, Wo=8, H=8, L=2048, D=128,
             dtype="bf16", layout="beams_first", ragged=True),
    ]


MAX_VALUES = {"top": 230_000_000, "distill": 300_000_000, "beam": 120_000_000,
              "reorder": 1_000_000_000}


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["top", "distill", "distill", "beam", "reorder"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    most = MAX_VALUES[op] // (2 if dtype == "f32" else 1)
    if op == "reorder":
        B, W = _spread(rng, 1, 32), _spread(rng, 2, 16)
        G, H, D = rng.choice([1, 2, 4]), rng.choice([1, 4, 8]), rng.choice([64, 80, 128, 256])
        L = _spread(rng, 1, max(1, min(4096, most // (G * B * W * H * D))))
        return dict(op=op, G=G, B=B, W=W, Wo=rng.choice([W, _spread(rng, 1, W)]), H=H, L=L, D=D,
                    dtype=dtype, layout=rng.choice(["beams_first", "heads_first"]),
                    ragged=rng.random() < 0.7)
    V = _spread(rng, 1000, 152064)
    if rng.random() < 0.6:
        V -= V % 8
    if op == "beam":
        W = _spread(rng, 1, 32)
        B = _spread(rng, 1, max(1, min(128, most // (W * V))))
        return dict(op=op, B=B, W=W, V=V, n=_spread(rng, 1, 64), dtype=dtype,
                    dead=rng.choice([0, 0, W // 4, W - 1]))
    k = _spread(rng, 1, 128)
    P = rng.randint(1, 32) if op == "distill" else rng.randint(1, 8)
    B = _spread(rng, 1, max(1, min(256, most // (P * V))))
    case = dict(op=op, B=B, P=P, V=V, k=k, dtype=dtype, T=rng.choice([1.0, 1.0, 0.7, 2.0]))
    if op == "distill":
        case.update(tail=rng.random() < 0.7, split=rng.random() < 0.5)
    return case


def _row_lens(case):
    """How many of its P rows each request needs: 1..P in turn, from P down."""
    return [case["P"] - b % case["P"] for b in range(case["B"])]


def _seq_lens(case):
    """How many of the L entries each request holds: evenly spaced in (L / 2, L]."""
    if not case["ragged"]:
        return [case["L"]] * case["B"]
    return [max(1, math.ceil(case["L"] * (0.5 + 0.5 * (b + 1) / case["B"])))
            for b in range(case["B"])]


def work(case):
    if case["op"] == "reorder":
        values = case["G"] * case["Wo"] * case["H"] * case["D"] * sum(_seq_lens(case))
        values = values * _kept(case) // case["Wo"]
        return {"bytes": 2 * values * ESIZE[case["dtype"]], "flops": 0}
    e = ESIZE[case["dtype"]]
    if case["op"] == "beam":
        live = case["B"] * (case["W"] - case["dead"])
        return {"bytes": live * case["V"] * e + case["B"] * (4 * case["W"] + 12 * case["n"]),
                "flops": 4 * live * case["V"]}
    rows, need = case["B"] * case["P"], sum(_row_lens(case))
    if case["op"] == "top":
        return {"bytes": need * case["V"] * e + rows * (8 * case["k"] + 4),
                "flops": 4 * need * case["V"]}
    # the student's needed rows once and the whole gradient once; apart, forward and backward
    # each read the rows
    reads = 2 if case["split"] else 1
    return {"bytes": (reads * need + rows) * case["V"] * e + rows * (8 * case["k"] + 12),
            "flops": 8 * need * case["V"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _logits(shape, dtype, g):
    """3 N(0, 1) plus a log-Zipf prior over a permuted vocabulary."""
    V = shape[-1]
    rank = torch.randperm(V, generator=g, device="cuda").float()
    x = torch.randn(shape, generator=g, device="cuda", dtype=TORCH_TYPES[dtype])
    return x.mul_(3.0).add_((-1.1 * torch.log1p(rank)).to(x.dtype))


def _shuffled(values, g):
    v = torch.tensor(values, dtype=torch.int32, device="cuda")
    return v[torch.randperm(len(values), generator=g, device="cuda")].contiguous()


def _kept(case):
    """Slots of `Wo` that take a state: all of a beam's, or a path that ends before the last."""
    return case["Wo"] if case["L"] > 1 else max(1, case["Wo"] - 1)


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    if case["op"] == "reorder":
        G, B, W, Wo, H, L, D = (case[x] for x in ("G", "B", "W", "Wo", "H", "L", "D"))

        def cache(slots):
            t = TORCH_TYPES[case["dtype"]]
            if case["layout"] == "beams_first":
                return torch.randn((G, B, slots, H, L, D), generator=g, device="cuda", dtype=t)
            x = torch.randn((G, B, H, slots, L, D), generator=g, device="cuda", dtype=t)
            return x.transpose(2, 3)
        s.update(state=cache(W), out=cache(Wo), lens=_shuffled(_seq_lens(case), g))
        parents = torch.randint(0, W, (B, Wo), generator=g, device="cuda", dtype=torch.int32)
        parents[:, _kept(case):] = -1
        s["parents"] = parents
        return s
    if case["op"] == "beam":
        B, W = case["B"], case["W"]
        s["logits"] = _logits((B, W, case["V"]), case["dtype"], g)
        scores = -3.0 * torch.rand((B, W), generator=g, device="cuda")
        order = torch.rand((B, W), generator=g, device="cuda").argsort(dim=1)
        s["scores"] = scores.masked_fill(order < case["dead"], -math.inf)
        return s
    B, P, V = case["B"], case["P"], case["V"]
    s["lens"] = _shuffled(_row_lens(case), g)
    x = _logits((B, P, V), case["dtype"], g)
    if case["op"] == "top":
        s["logits"] = x
        return s
    top = x.topk(min(case["k"], V), dim=-1)
    s["top_ids"] = top.indices.to(torch.int32)
    s["top_logits"] = top.values.float()
    s["top_lse"] = None
    if case["tail"]:
        s["top_lse"] = torch.stack([torch.logsumexp(r.float() / case["T"], dim=-1) for r in x])
    noise = torch.randn(x.shape, generator=g, device="cuda", dtype=x.dtype)
    s["student"] = x.mul_(0.9).add_(noise.mul_(0.7))
    w = torch.rand((B, P), generator=g, device="cuda") + 0.5
    s["grad_loss"] = w / float(sum(_row_lens(case)))
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _needed(lens, P):
    return torch.arange(P, device=lens.device)[None, :] < lens[:, None]


def _top_of_rows(x, k):
    """(values, ids) of the k largest of each row of fp32 values, equal values by the lowest
    id: the largest whole-number keys (value in order, then the id from the end)."""
    V = x.shape[-1]
    bits = (x + 0.0).view(torch.int32)
    key = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).to(torch.int64) * (1 << 24)
    key = key + torch.arange(V - 1, -1, -1, device=x.device)
    ids = V - 1 - (key.topk(min(k, V), dim=-1).values & 0xFFFFFF)
    return x.gather(-1, ids), ids


def _padded(x, k, value):
    return torch.nn.functional.pad(x, (0, k - x.shape[-1]), value=value)


def _plain_top(s):
    x = s["logits"].float()
    m = x.amax(dim=-1, keepdim=True)
    lse = torch.log(torch.exp((x - m) / s["T"]).sum(dim=-1)) + m[..., 0] / s["T"]
    values, ids = _top_of_rows(x, s["k"])
    need = _needed(s["lens"], s["P"])
    gone = ~(need[..., None] & (values > -math.inf))
    return {"ids": _padded(ids.masked_fill(gone, -1), s["k"], -1).to(torch.int32),
            "logits": _padded(values.masked_fill(gone, -math.inf), s["k"], -math.inf),
            "lse": lse.masked_fill(~need, -math.inf)}


def _plain_distill(s):
    T, ids = s["T"], s["top_ids"].long()
    need = _needed(s["lens"], s["P"])
    x = s["student"].float() / T
    t = s["top_logits"].double() / T
    if s["top_lse"] is None:
        logp = t - torch.logsumexp(t, dim=-1, keepdim=True)
        p_tail = torch.zeros_like(logp[..., 0])
    else:
        logp = t - s["top_lse"].double()[..., None]
        p_tail = (1.0 - torch.exp(logp).sum(dim=-1)).clamp(min=0.0)
        if ids.shape[-1] == s["V"]:
            p_tail = torch.zeros_like(p_tail)
    p = torch.exp(logp)
    x = x - x.amax(dim=-1, keepdim=True)
    e = torch.exp(x)
    total = e.sum(dim=-1).double()
    rest = e.scatter(-1, ids, 0.0).sum(dim=-1).double()
    logq = x.gather(-1, ids).double() - torch.log(total)[..., None]
    loss = (p * (logp - logq)).sum(dim=-1)
    with_tail = p_tail > 0
    logs = torch.log(p_tail.clamp(min=1e-300)) - (torch.log(rest) - torch.log(total))
    loss = loss + torch.where(with_tail, p_tail * logs, 0.0)
    share = torch.where(with_tail, 1.0 - p_tail * total / rest, 1.0)
    scale = torch.where(need, s["grad_loss"], 0.0).double() / T
    grad = e * (scale * share / total).float()[..., None]
    at_ids = (scale[..., None] * (torch.exp(logq) - p)).float()
    grad = grad.scatter(-1, ids, at_ids).to(s["student"].dtype)
    return {"loss": torch.where(need, loss, 0.0).float(), "grad": grad}


def _plain_beam(s):
    W, V, n = s["W"], s["V"], s["n"]
    x = s["logits"].double()
    m = x.amax(dim=-1)
    lse = torch.log(torch.exp(x - m[..., None]).sum(dim=-1)) + m
    values, ids = _top_of_rows(s["logits"].float(), n)  # no other candidate can be kept
    score = s["scores"].double()[..., None] - lse[..., None] + values.double()
    flat = ids + V * torch.arange(W, device=x.device)[None, :, None]
    flat, order = flat.flatten(1).sort(dim=1)
    score, by = score.flatten(1).gather(1, order).sort(dim=1, descending=True, stable=True)
    score, flat = score[:, :n], flat.gather(1, by)[:, :n]
    gone = ~(score > -math.inf)
    return {"tokens": _padded((flat % V).masked_fill(gone, -1), n, -1).to(torch.int32),
            "parents": _padded((flat // V).masked_fill(gone, -1), n, -1).to(torch.int32),
            "scores": _padded(score.masked_fill(gone, -math.inf), n, -math.inf).float()}


def _plain_reorder(s):
    state, out, parents = s["state"], s["out"], s["parents"].long()
    at = torch.arange(s["B"], device=out.device)[:, None]
    moved = state[:, at, parents.clamp(min=0)]
    inside = torch.arange(s["L"], device=out.device)[None, :] < s["lens"][:, None]
    take = (parents >= 0)[None, :, :, None, None, None] & inside[None, :, None, None, :, None]
    return out.copy_(torch.where(take, moved, out))


PLAIN = {"top": _plain_top, "distill": _plain_distill, "beam": _plain_beam,
         "reorder": _plain_reorder}


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _own(s):
    from token_verification_gb300 import api
    if s["op"] == "top":
        o = api.spec_top_logits(s["logits"], s["k"], s["T"], lens=s["lens"])
        return {"ids": o.ids, "logits": o.logits, "lse": o.lse}
    if s["op"] == "beam":
        o = api.spec_beam_select(s["logits"], s["scores"], s["n"])
        return {"tokens": o.tokens, "parents": o.parents, "scores": o.scores}
    if s["op"] == "reorder":
        return api.spec_beam_reorder(s["state"], s["parents"], s["out"], lens=s["lens"])
    args = s["student"], s["top_ids"], s["top_logits"], s["T"]
    more = dict(top_lse=s["top_lse"], lens=s["lens"])
    if not s["split"]:
        o = api.spec_distill(*args, grad_loss=s["grad_loss"], **more)
        return {"loss": o.loss, "grad": o.grad}
    o = api.spec_distill(*args, **more)
    grad = api.spec_distill_grad(*args, o.stats, s["grad_loss"], **more)
    return {"loss": o.loss, "grad": grad}


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits, a request at a time
# ---------------------------------------------------------------------------

def _exact_distill(s, b):
    """(loss [P], gradient [P, V]) of request b, the gradient from the definition's derivative
    by each log-probability."""
    P, V, T = s["P"], s["V"], s["T"]
    n = int(s["lens"][b])
    loss = torch.zeros(P, dtype=torch.float64, device="cuda")
    grad = torch.zeros((P, V), dtype=torch.float64, device="cuda")
    logq = torch.log_softmax(s["student"][b, :n].to(torch.float64) / T, dim=-1)
    ids = s["top_ids"][b, :n].long()
    t = s["top_logits"][b, :n].to(torch.float64) / T
    if s["top_lse"] is None:
        logp = torch.log_softmax(t, dim=-1)
    else:
        logp = t - s["top_lse"][b, :n, None].to(torch.float64)
    p = logp.exp()
    loss[:n] = (p * (logp - logq.gather(-1, ids))).sum(-1)
    by_logq = torch.zeros_like(logq).scatter(-1, ids, -p)
    if s["top_lse"] is not None and ids.shape[-1] < V:
        p_rest = torch.clamp(1.0 - p.sum(-1), min=0.0)
        outside = torch.ones_like(logq).scatter(-1, ids, 0.0).bool()
        log_rest = logq.masked_fill(~outside, -math.inf)
        q_rest = torch.logsumexp(log_rest, dim=-1)
        loss[:n] += torch.special.xlogy(p_rest, p_rest) - p_rest * q_rest
        by_logq = by_logq - p_rest[:, None] * (log_rest - q_rest[:, None]).exp()
    g = (s["grad_loss"][b, :n].to(torch.float64) / T)[:, None]
    grad[:n] = g * (by_logq - logq.exp() * by_logq.sum(-1, keepdim=True))
    return loss, grad


def _sorted_rows(x, k):
    v, i = x.sort(dim=-1, descending=True, stable=True)
    return v[..., :k], i[..., :k]


def _exact_top(s, b):
    P, k = s["P"], s["k"]
    n = int(s["lens"][b])
    ids = torch.full((P, k), -1, dtype=torch.int32, device="cuda")
    logits = torch.full((P, k), -math.inf, dtype=torch.float64, device="cuda")
    lse = torch.full((P,), -math.inf, dtype=torch.float64, device="cuda")
    x = s["logits"][b, :n].to(torch.float64)
    v, i = _sorted_rows(x, k)
    ids[:n, :v.shape[-1]], logits[:n, :v.shape[-1]] = i.to(torch.int32), v
    lse[:n] = torch.logsumexp(x / s["T"], dim=-1)
    return ids, logits, lse


def _exact_beam(s, b):
    n = s["n"]
    x = s["scores"][b].double()[:, None] + torch.log_softmax(s["logits"][b].double(), dim=-1)
    v, i = _sorted_rows(x.flatten(), n)
    scores = torch.full((n,), -math.inf, dtype=torch.float64, device="cuda")
    scores[:v.numel()] = v
    tokens = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    parents = tokens.clone()
    tokens[:v.numel()] = (i % s["V"]).int()
    parents[:v.numel()] = (i // s["V"]).int()
    tokens[scores == -math.inf] = -1
    parents[scores == -math.inf] = -1
    return tokens, parents, scores


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "reorder":
        out = s["out"].double() if s["out"].numel() < 100_000_000 else s["out"].clone()
        lens, parents = s["lens"].tolist(), s["parents"].tolist()
        for b in range(case["B"]):
            for w, p in enumerate(parents[b]):
                if p >= 0:
                    out[:, b, w, :, :lens[b]] = s["state"][:, b, p, :, :lens[b]].to(out.dtype)
        return out
    one = {"top": _exact_top, "distill": _exact_distill, "beam": _exact_beam}[case["op"]]
    names = {"top": ("ids", "logits", "lse"), "distill": ("loss", "grad"),
             "beam": ("tokens", "parents", "scores")}[case["op"]]
    if case["op"] == "distill" and case["B"] * case["P"] * case["V"] > 100_000_000:
        rows = [torch.zeros((case["B"], case["P"]), dtype=torch.float64, device="cuda"),
                torch.zeros(s["student"].shape, dtype=torch.float64, device="cuda")]
        for b in range(case["B"]):
            rows[0][b], rows[1][b] = one(s, b)
        return dict(zip(names, rows))
    return dict(zip(names, (torch.stack(x) for x in zip(*(one(s, b) for b in range(case["B"]))))))
