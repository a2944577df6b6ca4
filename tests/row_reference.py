"""Plain 64-bit references of the whole-row operators (truncated sampling,
truncated rows, top logits, the distillation loss), row by row in numpy."""
import math

import numpy as np


def kept_tokens(x, T, k=0, p=1.0, m=0.0):
    """The kept tokens of one row, in descending order; settings as the fp32
    numbers the library takes."""
    x = np.asarray(x, dtype=np.float64)
    T, p, m = float(np.float32(T)), float(np.float32(p)), float(np.float32(m))
    order = np.lexsort((np.arange(x.size), -x))
    order = order[np.isfinite(x[order])]
    if T == 0.0:
        return order[:1]
    z = (x[order] - x[order[0]]) / T
    w = np.exp(z)
    n = order.size if k == 0 else min(k, order.size)
    if p < 1.0:
        c = np.cumsum(w[:n])
        n_p = int((c < p * c[-1]).sum()) + 1
    else:
        n_p = n
    n_m = int((z >= math.log(m)).sum()) if m > 0.0 else order.size
    return order[:max(1, min(n, n_p, n_m))]


def draw(x, kept, T, u):
    """The first token in index order whose running sum of kept weights
    exceeds u times their sum, and how near u lies to a boundary."""
    x = np.asarray(x, dtype=np.float64)
    T = float(np.float32(T))
    w = np.zeros(x.size)
    w[kept] = 1.0 if T == 0.0 else np.exp((x[kept] - x[kept].max()) / T)
    c = np.cumsum(w)
    return int(np.searchsorted(c, float(u) * c[-1], side="right"))


def top(x, k, T):
    """(values, index, rest) of one row."""
    x = np.asarray(x, dtype=np.float64)
    order = np.lexsort((np.arange(x.size), -x))
    order = order[np.isfinite(x[order])]
    values, index = np.full(k, -np.inf), np.full(k, -1)
    n = min(k, order.size)
    values[:n], index[:n] = x[order[:n]], order[:n]
    others = x[order[n:]] / float(np.float32(T))
    rest = -np.inf if others.size == 0 else others.max() + math.log(np.exp(others - others.max()).sum())
    return values, index, rest


def distill(s, values, index, rest, T, weight=1.0):
    """(loss, gradient) of one row: the derivative through the softmax over
    all tokens, written out outcome by outcome."""
    s = np.asarray(s, dtype=np.float64)
    T, weight = float(np.float32(T)), float(np.float32(weight))
    grad = np.zeros(s.size)
    if weight == 0.0:
        return 0.0, grad
    here = np.asarray(index) >= 0
    index, values = np.asarray(index)[here], np.asarray(values, dtype=np.float64)[here]
    outcome = np.append(values / T, rest)
    if not (outcome > -np.inf).any():
        return 0.0, grad
    e = np.exp(outcome - outcome.max())
    p = e / e.sum()
    z = s / T
    q = np.exp(z - z.max())
    q /= q.sum()
    other = np.ones(s.size, dtype=bool)
    other[index] = False
    q_r = q[other].sum()
    with np.errstate(divide="ignore", invalid="ignore"):
        # ln q from the logits: a q that underflows keeps its logarithm
        lse = z.max() + math.log(np.exp(z - z.max()).sum())
        lo = z[other]
        l_r = lo.max() + math.log(np.exp(lo - lo.max()).sum()) - lse if lo.size and lo.max() > -np.inf else -np.inf
        lq = np.append(z[index] - lse, l_r)
        terms = np.where(p > 0, p * (np.log(p) - lq), 0.0)
    grad[:] = q
    grad[index] -= p[:-1]
    if q_r > 0 or p[-1] > 0:
        with np.errstate(invalid="ignore"):
            share = np.exp(lo - lo.max())
        if lo.size and lo.max() > -np.inf:
            grad[other] -= p[-1] * share / share.sum()
    return weight * terms.sum(), weight / T * grad
