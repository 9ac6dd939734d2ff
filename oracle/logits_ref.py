"""Host definitions, in 64 bits, of the operators on rows of logits beside the verify (the best ids of a row, distillation from a
record of them, a beam step's selection) and of the fork of paged requests (TEST INFRASTRUCTURE ONLY). Plain numpy, row by
row."""
from __future__ import annotations

import math

import numpy as np


def log_sum(z):
    """ln(sum exp(z)); -inf for none."""
    z = np.asarray(z, dtype=np.float64)
    if z.size == 0 or np.all(z == -np.inf):
        return -np.inf
    m = z.max()
    return m + math.log(np.exp(z - m).sum())


def allowed(words, V):
    """Truth value of every id, from the packed words of one row."""
    return np.unpackbits(np.ascontiguousarray(words).view(np.uint8), bitorder="little")[:V].astype(bool)


def top_logits(z, n, temperature=1.0, mask=None):
    """One row: ids, log-probabilities, ln of the sum."""
    z = np.array(z, dtype=np.float64)
    if mask is not None:
        z[~mask] = -np.inf
    lse = np.nan if np.isnan(z).any() or (z == np.inf).any() else log_sum(z / temperature)
    ids, logprobs = np.full(n, -1, dtype=np.int64), np.full(n, -np.inf)
    order = [i for i in np.argsort(-z, kind="stable") if z[i] > -np.inf][:n]        # (NaN is not)
    ids[: len(order)] = order
    logprobs[: len(order)] = z[order] / temperature - lse
    return ids, logprobs, lse


def entries(ids, logprobs, V, rest=True):
    """The entries of a list that count: (ids, log-probabilities, whether any is at fault). Where the list is not renormalised, a
    log-probability above 0.5 is none."""
    got, lps, fault = [], [], False
    for j, (i, lp) in enumerate(zip(ids, logprobs)):
        if i == -1:
            continue
        if not 0 <= i < V or i in list(ids[:j]) or not lp < np.inf or (rest and lp > 0.5):
            fault = True
            continue
        got.append(int(i))
        lps.append(float(lp))
    return np.array(got, dtype=np.int64), np.array(lps), fault


def distill(z, ids, logprobs, temperature=1.0, rest=True, weight=1.0):
    """One row: loss, (ln of the sum of all, of the ids not listed), gradient, r / rho."""
    z = np.array(z, dtype=np.float64) / temperature
    V = z.shape[0]
    if weight == 0:
        return 0.0, (0.0, 0.0), np.zeros(V), 0.0
    ids, lps, _ = entries(ids, logprobs, V, rest)
    outside = np.ones(V, dtype=bool)
    outside[ids] = False
    every, others = log_sum(z), log_sum(z[outside])
    if not rest and lps.size and lps.max() > -np.inf:
        lps = lps - log_sum(lps)
    t = np.exp(lps)
    r = max(0.0, 1.0 - t.sum()) if rest else 0.0
    asks = t.sum() + r > 0
    if others == -np.inf:
        r = 0.0
    if every == -np.inf:
        return (math.inf if asks else 0.0) * weight, (every, others), np.zeros(V), 0.0
    if not asks:
        return 0.0, (every, others), np.zeros(V), 0.0
    mass = t.sum() + r
    some = t > 0
    with np.errstate(divide="ignore"):
        loss = float((t[some] * (lps[some] - (z[ids][some] - every))).sum())
    if r > 0:
        loss += r * (math.log(r) - (others - every))
    d = mass * np.exp(z - every)
    d[ids] -= t
    ratio = 0.0
    if r > 0:
        d[outside] -= r * np.exp(z[outside] - others)
        ratio = r / math.exp(others - every)
    return weight * loss, (every, others), d * weight / temperature, ratio


def beam_select(z, scores, n, mask=None, finished=None, end_token=-1):
    """One request: z [beams, V], scores [beams]. (beams, tokens, scores, finished) of the n best, -1 behind them, and the
    score of the best that is left out."""
    found = []
    for w, s in enumerate(scores):
        if not np.isfinite(s):
            continue
        if finished is not None and finished[w]:
            found.append((float(s), w, end_token, 1))
            continue
        ids, lps, lse = top_logits(z[w], min(n + 1, z.shape[1]), mask=None if mask is None else mask[w])
        if np.isnan(lse):
            continue
        found += [(float(s) + lp, w, int(i), int(i == end_token and end_token >= 0)) for i, lp in zip(ids, lps) if i >= 0]
    found.sort(key=lambda f: (-f[0], f[1], f[2]))
    best = found[:n] + [(-np.inf, -1, -1, 0)] * max(0, n - len(found))
    return ([f[1] for f in best], [f[2] for f in best], [f[0] for f in best], [f[3] for f in best], found)


def kv_fork(held, table, lengths, parent, fresh, page, out_table, out_lengths):
    """Copies the parents' begun pages in `held` (a list of [pages, heads, page, ...] arrays, changed in place) and fills
    out_table, out_lengths."""
    before = [x.copy() for x in held]
    for i, p in enumerate(parent):
        out_table[i] = -1
        out_lengths[i] = 0
        if p < 0:
            continue
        n = int(lengths[p])
        full, begun = n // page, n % page
        out_lengths[i] = n
        out_table[i, :full] = table[p, :full]
        if begun:
            out_table[i, full] = table[p, full]
        if fresh is not None and fresh[i] >= 0 and full < table.shape[1]:
            out_table[i, full] = fresh[i]
            for x, old in zip(held, before):
                x[fresh[i], :, :begun] = old[table[p, full], :, :begun]
