"""Logits operators around a round (oracle side).  TEST INFRASTRUCTURE.

"11.1 核心原理" section 11.1.2 takes p_i and q_i after each model's
constraints, and the tutorial's section 4.2 names distilling the draft model
toward the target; neither page fixes formulas.  Readings fixed here, numpy
float64, one row at a time:

* adjust_row: repetition (z / r or z * r by the sign of z, on every token seen
  in the prompt or generated), then frequency and presence (generated tokens
  only), then biases, then the mask;
* top_logits: order by value descending, equal values by token ascending; the
  log-sum-exps of z / T over the row and over the tokens outside the record;
* distill: sum_j p_j (log p_j - log q_j) over the record's tokens, with the
  rest of the vocabulary as one more outcome ("bucket") or with the teacher
  renormalised over the record ("renorm"), and its gradient.

Pins: ``tests/test_oracle_logits.py`` (worked values, a full sort, central
differences of the loss, and torch's KL divergence of full softmaxes).
"""

import numpy as np


def adjust_row(z, counts=None, prompt=(), drafts=(), repetition=1.0, presence=0.0, frequency=0.0, bias=(),
               allowed=None):
    """One adjusted row.  counts {token: occurrences among the generated
    tokens}, prompt tokens, drafts before this position, bias (token, value)
    pairs, allowed truth values."""
    x = np.array(z, dtype=np.float64)
    V = len(x)
    c = {t: n for t, n in (counts or {}).items()}
    for d in drafts:
        if 0 <= d < V:
            c[d] = c.get(d, 0) + 1
    for v in set(c) | set(prompt):
        x[v] = x[v] / repetition if x[v] > 0 else x[v] * repetition
        if c.get(v, 0) > 0:
            x[v] = x[v] - frequency * c[v] - presence
    for t, value in bias:
        if 0 <= t < V:
            x[t] += value
    if allowed is not None:
        x[~np.asarray(allowed, bool)] = -np.inf
    return x


def log_sum_exp(x):
    x = np.asarray(x, np.float64)
    m = x.max() if x.size else -np.inf
    if m == -np.inf:
        return -np.inf
    with np.errstate(invalid="ignore"):
        return m + np.log(np.exp(x - m).sum())


def usable(z):
    z = np.asarray(z, np.float64)
    return not (np.isnan(z).any() or np.isposinf(z).any() or not np.isfinite(z).any())


def top_logits(z, K, T):
    """(tokens [K], logits [K], lse, rest lse) of one row."""
    z = np.asarray(z, np.float64)
    tokens, logits = np.full(K, -1, np.int32), np.full(K, -np.inf)
    if not usable(z):
        return tokens, logits, np.nan, np.nan
    order = np.argsort(-z, kind="stable")[:K]
    tokens[:len(order)], logits[:len(order)] = order, z[order]
    rest = np.delete(z, order)
    return tokens, logits, log_sum_exp(z / T), log_sum_exp(rest / T)


def teacher_probs(tokens, logits, lse, V, T, tail):
    """(probabilities of the record's entries, probability of the rest) or
    None when the record has none."""
    tokens, t = np.asarray(tokens), np.asarray(logits, np.float64) / T
    live = (tokens >= 0) & (tokens < V)
    if np.isnan(t[live]).any() or np.isposinf(t[live]).any():
        return None
    t = np.where(live, t, -np.inf)
    if tail == "bucket":
        if not np.isfinite(lse[0]):
            return None
        p, p_rest = np.exp(t - lse[0]), np.exp(lse[1] - lse[0])
    else:
        if not (t > -np.inf).any():
            return None
        p, p_rest = np.exp(t - log_sum_exp(t)), 0.0
    return (p, p_rest) if p.sum() + p_rest > 0 else None


def distill(z, tokens, logits, lse, T, tail, w=1.0):
    """(loss, gradient [V], (student lse, rest lse), ok) of one student row."""
    z = np.asarray(z, np.float64)
    V = len(z)
    tokens = np.asarray(tokens)
    x = z / T
    S = sorted({int(t) for t in tokens if 0 <= t < V})
    inside = np.zeros(V, bool)
    inside[S] = True
    good = usable(z)
    L = log_sum_exp(x) if good else np.nan
    Lo = log_sum_exp(x[~inside]) if good else np.nan
    pr = teacher_probs(tokens, logits, lse, V, T, tail)
    if pr is None or w == 0:
        return 0.0, np.zeros(V), (L, Lo), pr is not None and good
    p, p_rest = pr
    if not good:
        return np.nan, np.full(V, np.nan), (L, Lo), False
    loss = 0.0
    grad = np.exp(x - L) * (p.sum() + p_rest)
    for t, pj in zip(tokens, p):
        if pj > 0:
            loss += pj * (np.log(pj) - (x[t] - L))
            grad[t] -= pj
    if p_rest > 0:
        loss += p_rest * (np.log(p_rest) - (Lo - L))
        if Lo > -np.inf:
            grad[~inside] -= p_rest * np.exp(x[~inside] - Lo)
    return w * loss, w / T * grad, (L, Lo), True
