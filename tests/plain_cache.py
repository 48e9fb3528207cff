"""Plain 64-bit forms of the 4-bit key/value cache's operators (spec_cache_write,
spec_cache_read, spec_cache_keep, spec_cache_attention) on the CPU, and the
bounds the attention kernels are held to.

Bounds.  u = 2^-24.  A score's dot product of D exact products is added in 32 bits,
in steps off by at most 2 u of the running sum: within 2 (D + 8) u of the sum A of the
products' magnitudes (scale included).  Scaling, the cap's quotient and product
and the bias are roundings of at most 4 u of their own sizes; the cap's tanh is within
2^-21 of 1 (tanhf in fp32: 2^-22).  A weight 2^(x - m) is an exponential good to 2^-21 of an
exponent rounded by 2 u (|x| + |m|).  So a weight is off by E = the sum of these,
relative; it is rounded to fp16 (2^-11; 2^-22 where a second fp16 takes the rest, in
fp32), or lies where fp16's steps end: weights are scaled by 2^15, so a part is off by at
most half of fp16's least step, 2^-25, which is 2^-40 of the row's largest weight.  Calls of
bf16 with more than 16 rows a key/value head scale by 2^7 against a reference that the
row's max may exceed by up to 2^8: the largest weight is 2^7 or more there, and a weight off by
at most 2^-25 / 2^7 = 2^-32 of it.  The running sums add n terms in steps of 16 or more: (64 + n / 4) u.
With p the exact weights, o their result and W = sum_j p_j |v_j|:
(step = 2^-40 or 2^-32)
    |out - o| <= (round + 2 E + 2 (64 + n / 4) u) W + n step max |v| + half a step of o,
and the log of the sum is within E + (64 + n / 4) u + 2 u |lse|.
"""
import math

import torch

U = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
TOP = 238
SCALES = torch.tensor([(1 + c % 8 / 8) * 2.0 ** (c // 8 - 20) for c in range(TOP + 1)],
                      dtype=torch.float64)


def quantise(x):
    """(q, scale bytes, values) of [..., D] by the definition: the least scale that
    reaches the group's top, multiples to the nearest, ties to even."""
    g = x.detach().cpu().double().unflatten(-1, (-1, 32))
    top = g.abs().amax(-1)
    byte = torch.searchsorted(7 * SCALES, top).clamp(max=TOP)
    s = SCALES[byte][..., None]
    q = torch.round(g / s).clamp(-7, 7)
    return q.flatten(-2).int(), byte, (q * s).flatten(-2)


def held(k, v):
    """What k and v [..., H, D] read back as: NaN in a head with anything not finite."""
    bad = ~(torch.isfinite(k).all(-1) & torch.isfinite(v).all(-1)).cpu()
    out = []
    for x in (k, v):
        y = quantise(torch.where(bad[..., None], 0.0, x.detach().cpu().double()))[2]
        y[bad] = math.nan
        out.append(y)
    return out


def decode(cache, page, D):
    """[pages, H, 2, page, D] float64 of a cache's bytes, nibble by nibble."""
    c = cache.cpu()
    codes = c[..., :page * D // 2].unflatten(-1, (page, D // 2)).int()
    scales = c[..., page * D // 2:].unflatten(-1, (page // 16, D // 32, 16)).int()
    out = torch.empty(codes.shape[:-1] + (D,), dtype=torch.float64)
    for d in range(D):
        nib = d % 8 // 2 + 4 * (d % 8 % 2)
        byte = codes[..., d // 8 * 4 + nib // 2]
        s = scales[..., d // 32, :].flatten(-2)
        out[..., d] = ((byte >> (4 * (nib % 2))) & 15).double() - 8
        out[..., d] *= SCALES[s.clamp(max=TOP)]
    nan = (scales[:, :, 0] == 247).any(-2).flatten(-2)
    out[nan[:, :, None].expand(-1, -1, 2, -1)] = math.nan
    return out


def slots(dec, table, n):
    """[n, H, 2, D] of one request's first n slots (table: its page ids)."""
    page = dec.shape[3]
    at = torch.arange(n)
    return dec[table.cpu().long()[at // page], :, :, at % page]


def ancestors(parent, n):
    """(sees [n, n], depth [n]) of a chain (parent None) or a tree."""
    sees = torch.zeros((n, n), dtype=torch.bool)
    depth = torch.zeros(n, dtype=torch.int64)
    for i in range(n):
        at = i
        while True:
            sees[i, at] = True
            if at == 0:
                break
            at = int(parent[at - 1]) if parent is not None else at - 1
            depth[i] += 1
    return sees, depth


def attention(q, kv, base, sees, depth, scale, softcap, window, slopes, dtype, step=2.0 ** -40):
    """One request: q [n, Hq, D], kv [L, H, 2, D] float64.  (out, lse, tol, lse tol), rows that
    see nothing 0 and -inf."""
    n, Hq, D = q.shape
    L, H = kv.shape[:2]
    group = Hq // H
    exact = dtype == torch.float32
    pos = torch.arange(L)
    pos[base:] = base + depth
    seen = torch.ones((n, L), dtype=torch.bool)
    seen[:, base:] = sees
    far = pos[base:base + n, None] - pos
    if window:
        seen &= far < window
    nan = torch.isnan(kv).flatten(2).any(-1)  # [L, H]: rows that see such a slot are NaN
    kv = kv.nan_to_num(0.0)
    out = torch.zeros((n, Hq, D), dtype=torch.float64)
    lse = torch.full((n, Hq), -math.inf, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    for h in range(Hq):
        k, v = kv[:, h // group, 0], kv[:, h // group, 1]
        x = (q[:, h] @ k.T) * scale
        A = (q[:, h].abs() @ k.abs().T) * abs(scale)
        E = 2 * (D + 8) * U * A + 4 * U * x.abs()
        if softcap:
            x = softcap * torch.tanh(x / softcap)
            # (tanh to a few last places, or by one exponential where that is 2^-12 at most)
            E = E + 8 * U * x.abs() + (0 if exact or softcap > 360 else softcap * 2.0 ** -21)
        if slopes is not None:
            b = float(slopes[h]) * far
            x = x - b
            E = E + 4 * U * (b.abs() + x.abs())
        x = x.masked_fill(~seen, -math.inf)
        some = seen.any(-1)
        if not bool(some.any()):
            continue
        m = x.amax(-1, keepdim=True)
        size = torch.where(seen, x.abs(), 0.0) + m.abs()
        E = torch.where(seen, E + 4 * U * size + 2.0 ** -20, 0.0)
        w = torch.exp(x - m)
        total = w.sum(-1, keepdim=True)
        p = torch.where(seen, w / total, 0.0)
        o = p @ v
        out[some, h] = o[some]
        lse[some, h] = (m + torch.log(total))[some, 0]
        sees_nan = (seen & nan[:, h // group]).any(-1)
        out[sees_nan, h] = math.nan
        lse[sees_nan, h] = math.nan
        steps = (64 + L / 4) * U
        top = E.amax(-1, keepdim=True)
        W = p @ v.abs()
        rounding = 2.0 ** (-22 if exact else -11)
        tol[:, h] = ((rounding + 2 * top + 2 * steps) * W
                     + L * step * v.abs().max()
                     + HALF_STEP[dtype] * o.abs() * 1.01 + 1e-37)
        ltol[:, h] = (top[:, 0] + steps + 2 * U * lse[:, h].abs().nan_to_num(0.0, 0.0, 0.0))
    return out, lse, tol, ltol


def check_attention(q, cache, page, table, lens, got, lse=None, q_lens=None, parent=None,
                    scale=None, softcap=0.0, window=0, slopes=None, before=None):
    """Every row of a spec_cache_attention result on valid inputs."""
    B, N, Hq, D = q.shape
    dec = decode(cache, page, D)
    lens = lens.cpu()
    many = q.dtype == torch.bfloat16 and D <= 128 and N * Hq // cache.shape[1] > 16
    step = 2.0 ** (-32 if many else -40)
    got64 = got.cpu().double()
    for b in range(B):
        n = N if q_lens is None else int(q_lens[b])
        if before is not None:
            assert torch.equal(got[b, n:].cpu(), before[b, n:].cpu()), b
        if n == 0:
            continue
        par = None if parent is None else (parent if parent.dim() == 1 else parent[b]).cpu()
        sees, depth = ancestors(par, n)
        L = int(lens[b])
        o, l, tol, ltol = attention(
            q[b, :n].cpu().double(), slots(dec, table[b], L), L - n, sees, depth,
            D ** -0.5 if scale is None else scale, softcap, window,
            None if slopes is None else slopes.cpu().double(), q.dtype, step)
        off = (got64[b, :n] - o).abs()
        bad = ~(off <= tol)
        bad &= ~(torch.isnan(o) & torch.isnan(got64[b, :n]))
        if bool(bad.any()):
            i = tuple(int(x) for x in bad.nonzero()[0])
            raise AssertionError((b, i, float(got64[b][i]), float(o[i]), float(tol[i]),
                                  int(bad.sum())))
        if lse is not None:
            mine = lse[b, :n].cpu().double()
            fine = ((mine - l).abs() <= ltol) | (mine == l) | (torch.isnan(mine) & torch.isnan(l))
            assert bool(fine.all()), (b, mine[~fine][:4], l[~fine][:4], ltol[~fine][:4])
