"""Plain 64-bit forms of the operators that train drafts and grow candidate
trees (spec_top_logits, spec_distill, spec_beam_select, spec_beam_reorder),
one row at a time in float64 on the CPU, and the bounds their kernels are
held to.

Bounds.  u = 2^-24 is half a step of fp32.  A kernel's weight 2^(l c - o) is
one rounded fma, |a| u for the exponent a, and an exponential good to 2^-22;
a thread adds at most 2^8 of them to a partial sum before the partial sums
are joined, each addition off by u.  Weights of exponent a < -40 do not
matter at this level, so a row sum is off by at most
    2^-22 + 40 ln 2 u + 2^8 u < 2e-5
of itself, and its logarithm by 2e-5: SUM.  A value written in fp32 adds u of
its size, one written in bf16 2^-8.
"""
import math

import numpy as np
import torch

SUM = 2e-5
U32 = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def f64(t):
    return t.detach().cpu().to(torch.float64)


def lse64(x):
    m = x.max()
    if m == -math.inf:
        return -math.inf
    return float(m + torch.log(torch.exp(x - m).sum()))


def top_row(row, k, T):
    """(ids, logits, lse) of one float64 row; ids and logits of its finite part."""
    v = row.numpy() + 0.0  # -0.0 -> +0.0
    order = np.argsort(-v, kind="stable")[:k]
    order = order[v[order] > -np.inf]
    return order, v[order], lse64(row / T)


def check_top(logits, k, T, out, lens=None):
    """Every row of a spec_top_logits result against the plain form."""
    x = f64(logits)
    B, P, V = x.shape
    ids, val, lse = out.ids.cpu().numpy(), out.logits.cpu().numpy(), out.lse.cpu().numpy()
    st = out.status.cpu().numpy()
    for b in range(B):
        n = P if lens is None else int(lens[b])
        for i in range(P):
            where = (b, i)
            row = x[b, i]
            ok_len = 0 <= n <= P
            bad = bool(torch.isnan(row).any() or (row == math.inf).any())
            if not ok_len or i >= n or bad:
                assert (ids[b, i] == -1).all() and (val[b, i] == -np.inf).all(), where
                if ok_len and i < n:
                    assert np.isnan(lse[b, i]) and st[b, i] == 2, where
                else:
                    assert lse[b, i] == -np.inf and st[b, i] == (0 if ok_len else 4), where
                continue
            want, wv, wl = top_row(row, k, T)
            c = len(want)
            assert (ids[b, i, :c] == want).all(), where
            assert (val[b, i, :c] == wv).all(), where
            assert (ids[b, i, c:] == -1).all() and (val[b, i, c:] == -np.inf).all(), where
            assert st[b, i] == 0, where
            if wl == -math.inf:
                assert lse[b, i] == -np.inf, where
            else:
                assert abs(lse[b, i] - wl) <= SUM + U32 * abs(wl), (where, lse[b, i], wl)


def distill_row(s, ids, t, lse, T):
    """(loss, size of its terms, gradient by s, q, p by token, share, p_rest) of one row
    in float64: `share` is each token's part of the student's mass outside the record."""
    V = s.numel()
    use = ids >= 0
    ids, t = ids[use].long(), t[use]
    x = (s - s.max()) / T  # differences first: rows of any magnitude
    L = lse64(x)
    top = max(float(t.max()), -torch.finfo(torch.float32).max)
    t = (t - top) / T
    logp = t - (lse64(t) if lse is None else lse - top / T)
    p = torch.exp(logp)
    p_rest = 0.0 if lse is None or len(ids) >= V else max(0.0, 1.0 - float(p.sum()))
    logq = x - L
    outside = torch.ones(V, dtype=torch.bool)
    outside[ids] = False
    terms = torch.where(p > 0, p * (logp - logq[ids]), torch.zeros_like(p))
    loss, size = float(terms.sum()), float(terms.abs().sum())
    share = torch.zeros(V, dtype=torch.float64)
    rest = float(x[outside].max()) if bool(outside.any()) else -math.inf
    if rest > -math.inf:
        d = x[outside] - rest
        share[outside] = torch.exp(d - lse64(d))
        rest += lse64(d) - L
    if p_rest > 0:
        d = p_rest * (math.log(p_rest) - rest)
        loss, size = loss + d, size + abs(d)
    q = torch.exp(logq)
    pv = torch.zeros(V, dtype=torch.float64)
    pv[ids] = p
    grad = (q - pv - p_rest * share) / T
    return loss, size, grad, q, pv, share, p_rest


def check_distill(student, ids, t, lse, T, grad_loss, lens, loss, grad, status=None):
    """loss and grad (either may be None) of valid inputs against the plain form."""
    s, ids, t = f64(student), ids.cpu(), f64(t)
    B, P, V = s.shape
    step = HALF_STEP[student.dtype]
    for b in range(B):
        n = P if lens is None else int(lens[b])
        for i in range(P):
            where = (b, i)
            if status is not None:
                assert int(status[b, i]) == 0, where
            if i >= n or not bool((ids[b, i] >= 0).any()):
                assert loss is None or float(loss[b, i]) == 0.0, where
                assert grad is None or not bool(grad[b, i].any()), where
                continue
            L, size, dg, q, p, share, p_rest = distill_row(
                s[b, i], ids[b, i], t[b, i], None if lse is None else float(lse[b, i]), T)
            if loss is not None:
                # each log q within SUM, each log p within 2 u |t / T| and p within
                # 2^-22: the terms' own sizes count once more for p's error
                got = float(loss[b, i])
                if math.isinf(L):
                    assert got == L, (where, got, L)
                else:
                    tol = 2 * SUM + 2.0 ** -20 * (size + 32)
                    assert abs(got - L) <= tol + U32 * abs(L), (where, got, L, tol)
            if grad is not None:
                g = float(grad_loss[b, i])
                got = f64(grad[b, i])
                want = g * dg
                # q within 2 SUM, p within 2^-20, p_rest = 1 - sum p within 2^-20 in all;
                # share is a weight over a sum of weights as q is: it is within 2 SUM too,
                # far below the max as well (2^-126: 126 ln 2 u = 5e-6), and p_rest takes that
                # into p_rest * share
                tol = abs(g) / T * (2 * SUM * (q + p_rest * share) + 2.0 ** -20 * (p + share))
                tol = tol * 1.01 + step * want.abs() * 1.01 + 1e-37
                off = (got - want).abs()
                j = int((off - tol).argmax())
                assert bool((off <= tol).all()), (where, j, float(got[j]), float(want[j]),
                                                  float(tol[j]))


def beam_scores(logits, scores):
    """[B, W, V] float64 scores of every continuation (-inf: none)."""
    x = f64(logits)
    s = f64(scores)
    out = torch.full_like(x, -math.inf)
    for b in range(x.shape[0]):
        for w in range(x.shape[1]):
            if s[b, w] > -math.inf:
                m = x[b, w].max()  # differences first: rows of any magnitude
                if m > -math.inf:
                    d = x[b, w] - m
                    out[b, w] = (s[b, w] - torch.log(torch.exp(d).sum())) + d
    return out


def check_beam(logits, scores, n, out):
    """A spec_beam_select result on valid inputs: wherever neighbouring scores
    are further apart than two errors the choice is exact; closer ones may
    change places, between beams only (within a beam the order of the logits
    decides, ties by the lower token)."""
    all_scores = beam_scores(logits, scores)
    B, W, V = all_scores.shape
    tok, par, sc = out.tokens.cpu().numpy(), out.parents.cpu().numpy(), out.scores.cpu().numpy()
    moved = 0
    for b in range(B):
        flat = all_scores[b].flatten().numpy()
        order = np.argsort(-flat, kind="stable")[:n]
        order = order[flat[order] > -np.inf]
        c = len(order)
        assert (tok[b, c:] == -1).all() and (par[b, c:] == -1).all(), b
        assert (sc[b, c:] == -np.inf).all(), b
        got = par[b, :c].astype(np.int64) * V + tok[b, :c]
        assert ((par[b, :c] >= 0) & (par[b, :c] < W) & (tok[b, :c] >= 0) & (tok[b, :c] < V)).all()
        assert len(set(got.tolist())) == c, b
        want = flat[order]
        tol = 2 * SUM + U32 * np.abs(want)
        mine = flat[got]
        assert (np.abs(mine - want) <= 2 * tol).all(), b
        assert (np.abs(sc[b, :c] - mine) <= tol).all(), (b, np.abs(sc[b, :c] - mine).max())
        for w in range(W):  # within a beam: the same tokens in the same order
            a = got[par[b, :c] == w]
            ref = np.argsort(-flat[w * V:(w + 1) * V], kind="stable")[:len(a)] + w * V
            assert (a == ref).all(), (b, w)
        moved += int((got != order).sum())
    return moved


def reorder(state, parents, out, lens):
    """The plain gather, slot by slot (CPU tensors)."""
    out = out.clone()
    L = state.shape[4]
    for b in range(parents.shape[0]):
        n = L if lens is None else int(lens[b])
        if not 0 <= n <= L:
            continue
        for w in range(parents.shape[1]):
            p = int(parents[b, w])
            if 0 <= p < state.shape[2]:
                out[:, b, w, :, :n] = state[:, b, p, :, :n]
    return out
