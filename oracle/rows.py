"""Operators on rows of vocabulary logits, one row at a time in float64: the
filters and the draw of a serving request, and distillation from a teacher's
top logits with its gradient.

The pages leave a request's filters to the serving engine (P2 "A 2B Drafter
Made a 27B Model 3.4x Faster. Same Exact Output.", section "Running it") and
the drafter's training to its authors (section "Caveats before you rebuild
your serving stack": drafters are trained per target model), so these
definitions are this project's own.  Pinned by tests/test_oracle_rows.py
against closed forms, the filters' one-by-one definitions and differences.
"""

import numpy as np


def order(z):
    """Unmasked tokens of a row by value descending, then index ascending."""
    z = np.asarray(z, dtype=np.float64)
    live = np.flatnonzero(z > -np.inf)  # NaN compares false: masked
    return live[np.argsort(-z[live], kind="stable")]


def keep(z, T=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(kept tokens in order, their weights exp((z - max) / T))."""
    z = np.asarray(z, dtype=np.float64)
    o = order(z)
    if o.size == 0:
        return o, np.zeros(0)
    if not T > 0:
        return o[:1], np.ones(1)
    v = z[o]
    w = np.where(v == v[0], 1.0, np.exp((v - v[0]) / T)) if np.isfinite(T) else np.ones(o.size)
    n = o.size
    if top_k > 0:
        n = min(n, int(top_k))
    if top_p < 1:
        run = np.cumsum(w[:n])
        n = min(n, 1 + int(np.count_nonzero(run < max(float(top_p), 0.0) * run[-1])))
    if min_p > 0:
        n = min(n, int(np.count_nonzero(w >= min(float(min_p), 1.0))))
    return o[:n], w[:n]


def sample(z, u, **filters):
    """(token, its probability among the kept, how many were kept)."""
    o, w = keep(z, **filters)
    if o.size == 0:
        return -1, 0.0, 0
    u = float(u)
    u = min(u, 1.0 - 2.0 ** -53) if u > 0 else 0.0
    run = np.cumsum(w)
    i = min(int(np.count_nonzero(run <= u * run[-1])), o.size - 1)
    return int(o[i]), float(w[i] / run[-1]), int(o.size)


def filtered(z, fill, **filters):
    z = np.asarray(z, dtype=np.float64)
    out = np.full(z.shape, float(fill))
    o, _ = keep(z, **filters)
    out[o] = z[o]
    return out


RANGE = 2.0 ** 40 * np.log(2.0)  # beyond it float64 does not hold a log-sum-exp beside its largest term


def log_sum_exp(x):
    x = np.asarray(x, dtype=np.float64)
    if x.size == 0:
        return -np.inf
    m = x.max()
    if m <= -RANGE:
        return -np.inf
    if m >= RANGE:
        return np.nan
    if not np.isfinite(m):
        return -np.inf if m == -np.inf else np.nan
    return float(m + np.log(np.exp(x - m).sum()))


def distill(s, t_idx, t_logit, tau=1.0, t_lse=None):
    """The divergence of one student row and its gradient.

    Returns a dict: loss, lse, lse_rest (unlisted tokens; None without
    ``t_lse``), grad [V] = d loss / d s, and what a tolerance needs: p_sum.
    """
    s = np.asarray(s, dtype=np.float64)
    V = s.size
    x = s / tau
    ok = (t_idx >= 0) & (t_idx < V)
    idx, t = np.asarray(t_idx)[ok].astype(np.int64), np.asarray(t_logit, dtype=np.float64)[ok] / tau
    t = np.where(t == np.inf, np.nan, t)  # no logit: the row has no result
    lse = log_sum_exp(x)
    out = dict(lse=lse, lse_rest=None, grad=np.zeros(V), loss=0.0, p=np.zeros(V), A=0.0, p_rest=0.0)
    unlisted = np.ones(V, dtype=bool)
    unlisted[idx] = False
    rest = None
    if t_lse is not None:
        rest = log_sum_exp(x[unlisted])
        out["lse_rest"] = rest
    c = float(t_lse) if t_lse is not None else log_sum_exp(t)
    if lse == -np.inf or c in (np.inf, -np.inf):
        return out
    p = np.exp(t - c)
    pv = np.zeros(V)
    np.add.at(pv, idx, p)
    on = p != 0
    with np.errstate(invalid="ignore"):
        loss = float(np.sum(p[on] * (t[on] - c - x[idx[on]] + lse)))
    p_rest = 0.0
    if rest is not None and rest > -np.inf:
        p_rest = max(0.0, 1.0 - float(p.sum()))
        if p_rest > 0:
            loss += p_rest * (np.log(p_rest) - rest + lse)
    A = float(p.sum()) + p_rest
    g = A * np.exp(x - lse) - pv
    if p_rest > 0:
        g = g - np.where(unlisted, p_rest * np.exp(x - rest), 0.0)
    out.update(grad=g / tau, loss=loss, p=pv, A=A, p_rest=p_rest)
    return out
