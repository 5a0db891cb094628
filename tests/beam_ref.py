"""Plain forms of beam search's selection and reordering, for the tests."""
from __future__ import annotations

import numpy as np


def scores64(x, cum):
    """64-bit scores [W][V] of logits x [W][V] and the beams' scores cum [W]; -inf for what is no candidate."""
    x = np.asarray(x, np.float64)
    out = np.full(x.shape, -np.inf)
    for w in range(x.shape[0]):
        if np.isneginf(cum[w]) or np.isnan(cum[w]) or cum[w] == np.inf or np.isnan(x[w]).any() or np.isposinf(x[w]).any():
            continue
        m = x[w].max()
        if np.isneginf(m):
            continue
        with np.errstate(over="ignore", under="ignore"):
            out[w] = ((x[w] - m) - np.log(np.exp(x[w] - m).sum())) + np.float64(cum[w])   # (m may be the lowest number)
    return out


def best(s, K):
    """tokens, parents, scores of the K best, -1, -1, -inf behind the last."""
    flat = s.reshape(-1)
    at = np.argsort(-flat, kind="stable")[:K]
    at = at[flat[at] > -np.inf]
    t, p, v = np.full(K, -1), np.full(K, -1), np.full(K, -np.inf)
    t[:len(at)], p[:len(at)], v[:len(at)] = at % s.shape[1], at // s.shape[1], flat[at]
    return t, p, v


def lse_error(V):
    """Bound on the kernel's error of a row's log of the sum of exponentials: a term exp(x - m) is off by its argument's two
    roundings, 2^-23 |x - m| (2^-24 more where m nears 2^24), and by exp2's 2^-22; the terms' share-weighted mean of |x - m| is at most log V (the entropy of
    the shares); 64 terms to a lane and five steps over lanes, half a step of 2^-23 each.  Then one term for each 4 KiB (at
    least 1024 tokens): an exponential of a rounded difference (2^-24 of it, again log V in the mean; the exponential 2^-22),
    a product, a 32nd of the terms to a lane and five steps over lanes.  The logarithm of the sum is off by 2^-22 at most."""
    terms = -(-V // 1024)
    return np.log(V + 1) * 1.5 * 2.0 ** -23 + 3 * 2.0 ** -22 + (1 + 69 + 1 + -(-terms // 32) + 5) * 2.0 ** -24


def check_best(x, cum, K, tokens, parents, scores):
    """The kernel's K best of one request: right but where scores of different beams lie closer than their errors."""
    s = scores64(x, cum)
    W, V = s.shape
    n = min(K, int((s > -np.inf).sum()))
    assert np.all(tokens[n:] == -1) and np.all(parents[n:] == -1) and np.all(np.isneginf(scores[n:]))
    t, p = tokens[:n], parents[:n]
    assert np.all((p >= 0) & (p < W) & (t >= 0) & (t < V))
    assert len(set(zip(p.tolist(), t.tolist()))) == n
    exact = s[p, t]
    d = lse_error(V)
    far = exact <= -(2.0 ** 128 - 2.0 ** 103)      # rounds to -infinity in fp32 (half a step behind the largest number)
    assert np.all(np.isneginf(scores[:n][far]))
    assert np.all(np.abs(scores[:n] - exact)[~far] <= d + np.abs(exact[~far]) * 2.0 ** -24)
    # of each beam the first ones by logit, then token, in that order
    for w in set(p.tolist()):
        mine = t[p == w]
        assert np.array_equal(mine, np.argsort(-np.asarray(x[w], np.float64), kind="stable")[:len(mine)]), w
    assert np.all(np.diff(exact) <= 2 * d)
    if n:
        left = s.copy()
        left[p, t] = -np.inf
        assert left.max() <= exact.min() + 2 * d


def reorder(parents, table, seq_len):
    """New table [B W][np_max], the copies [(request, from page, to page)]."""
    B, W = parents.shape
    new = table.copy()
    copies = []
    for b in range(B):
        par, rows, L = parents[b], range(b * W, b * W + W), int(seq_len[b * W])
        full = L // 64
        for w in range(W):
            if par[w] >= 0:
                new[rows[w], :full] = table[rows[par[w]], :full]
        if L % 64 == 0:
            continue
        free = [p for p in range(W) if p not in par]
        for w in range(W):
            p = par[w]
            if p >= 0 and w == (p if par[p] == p else list(par).index(p)):
                new[rows[w], full] = table[rows[p], full]
                continue
            to = table[rows[free.pop(0)], full]
            new[rows[w], full] = to
            if p >= 0:
                copies.append((b, int(table[rows[p], full]), int(to)))
        assert not free
    return new, copies
