"""Plain fp64 definitions of the operators on tokens and rows of logits, and of distillation
(test infrastructure only).

Values are computed from the exact inputs the GPU reads.  Where a result is a choice at a border
of a sum, the distance to the nearest border stands beside it.
"""
from __future__ import annotations

import numpy as np

from .train_oracle import MASK_LEVEL


def order(z):
    """Token ids by falling logit, equal ones by rising id, -infinity and NaN left out."""
    z = np.asarray(z, np.float64)
    with np.errstate(invalid="ignore"):
        ids = np.nonzero(z > -np.inf)[0]
    return ids[np.argsort(-z[ids], kind="stable")]


def sample_row(z, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """Token, log-probability, and how near (relative to the mass) a border was."""
    z = np.asarray(z, np.float64)
    ids = order(z)
    if len(ids) == 0:
        return -1, -np.inf, np.inf
    if not temperature > 0:
        return int(ids[0]), 0.0, np.inf
    top = z[ids[0]]
    with np.errstate(invalid="ignore", over="ignore"):
        d = np.where(z[ids] == top, 0.0, (z[ids] - top) / temperature)
    w = np.exp(d)
    n, near = len(ids), np.inf
    if 0 < top_k < n:
        n = int(top_k)
    exact = bool(np.all(w[:n] == 1.0))       # whole numbers: every border is exact
    if top_p < 1:
        mass = w[:n].sum()
        before = np.cumsum(w[:n]) - w[:n]
        want = max(0.0, float(top_p)) * mass
        if n > 1:
            near = min(near, np.min(np.abs(before[1:] - want)) / mass)
        n = max(1, int(np.sum(before < want)))
    if min_p > 0:
        level = min(1.0, float(min_p))
        near = min(near, np.min(np.abs(w[:n] - level) + np.where(w[:n] == 1.0, 1.0, 0.0)))
        n = int(np.sum(w[:n] >= level))
    kept = np.sort(ids[:n])
    by_id = np.zeros(len(z))
    by_id[ids[:n]] = w[:n]
    cum = np.cumsum(by_id[kept])
    u = min(max(float(u), 0.0), 1.0) if u == u else 0.0
    last = int(np.searchsorted(cum, cum[-1]))        # the last with a weight
    at = min(int(np.searchsorted(cum, u * cum[-1], side="right")), last)
    if u > 0 and last > 0:
        near = min(near, np.min(np.abs(cum[:last] - u * cum[-1])) / cum[-1])
    if exact:
        near = np.inf
    return int(kept[at]), float(np.log(by_id[kept[at]] / cum[-1])), near


def top_row(z, k):
    """The k largest: ids, values (-1 and -infinity where none is left), log-sum-exp."""
    z = np.asarray(z, np.float64)
    ids = order(z)
    top = ids[:k]
    out_ids = np.full(k, -1, np.int64)
    out = np.full(k, -np.inf)
    out_ids[:len(top)], out[:len(top)] = top, z[top]
    if len(ids) == 0:
        return out_ids, out, -np.inf
    m = z[ids[0]]
    with np.errstate(invalid="ignore"):
        s = np.exp(np.where(z[ids] == m, 0.0, z[ids] - m)).sum()
    return out_ids, out, m + np.log(s)


def embed(table, ids, scale):
    table = np.asarray(table, np.float64)
    out = np.zeros((len(ids), table.shape[1]))
    on = (ids >= 0) & (ids < len(table))
    out[on] = scale * table[ids[on]]
    return out


def embed_backward(ids, d_out, V, scale, add=None):
    """The gradient, and the sums of its terms' magnitudes."""
    d_out = np.asarray(d_out, np.float64)
    g, mag = np.zeros((V, d_out.shape[1])), np.zeros((V, d_out.shape[1]))
    on = (ids >= 0) & (ids < V)
    np.add.at(g, ids[on], scale * d_out[on])
    np.add.at(mag, ids[on], np.abs(scale * d_out[on]))
    if add is not None:
        g += np.asarray(add, np.float64)
    return g, mag


def distill_loss(hidden, lm_head, ids, logits, lse=None, t_scale=1.0, prev=None, w1=None, w2=None,
                 lm_bias=None, d2t=None, weights=None, reduction="mean", loss_scale=1.0, V=None):
    """As train_oracle.head_loss, for a teacher's listed tokens."""
    h, W = np.asarray(hidden, np.float64), np.asarray(lm_head, np.float64)
    T, Vh = h.shape[0], W.shape[0]
    V = Vh if V is None else V
    k = ids.shape[1]
    where = {int(v): j for j, v in enumerate(range(V) if d2t is None else d2t)}
    col = np.full((T, k), -1)
    dropped = 0
    s = np.asarray(logits, np.float64)
    for t in range(T):
        listed = [int(v) for v, x in zip(ids[t], s[t]) if v >= 0 and not x == -np.inf]
        if any(v >= V for v in listed) or len(set(listed)) < len(listed):
            dropped += 1
            continue
        for j in range(k):
            if ids[t, j] >= 0 and not s[t, j] == -np.inf:
                c = where.get(int(ids[t, j]), -1)
                if c >= 0 and lm_bias is not None and not lm_bias[c] > MASK_LEVEL:
                    c = -1
                col[t, j] = c
        if (col[t] >= 0).any() and w1 is not None and not 0 <= prev[t] < V:
            dropped += 1
            col[t] = -1
    tok = np.nonzero((col >= 0).any(1))[0]
    live = np.ones(Vh, bool) if lm_bias is None else np.asarray(lm_bias) > MASK_LEVEL
    place = np.cumsum(live) - 1
    w = np.ones(T) if weights is None else np.asarray(weights, np.float64)
    out = {"loss": np.zeros(T), "total": 0.0, "n_rows": len(tok), "dropped": dropped,
           "d_hidden": np.zeros_like(h), "d_lm_head": np.zeros_like(W)}
    mag = {"d_hidden": np.zeros_like(h), "d_lm_head": np.zeros_like(W), "z": 0.0,
           "loss": np.zeros(T), "q": 0.0}
    if w1 is not None:
        w1, w2 = np.asarray(w1, np.float64), np.asarray(w2, np.float64)
        out["d_markov_w1"], out["d_markov_w2"] = np.zeros_like(w1), np.zeros_like(w2)
        mag["d_markov_w1"], mag["d_markov_w2"] = np.zeros_like(w1), np.zeros_like(w2)
    out["mag"] = mag
    if len(tok) == 0:
        return out
    x, Wl = h[tok], W[live]
    z, zm = x @ Wl.T, np.abs(x) @ np.abs(Wl).T
    if w1 is not None:
        e, w2l = w1[np.asarray(prev)[tok]], w2[:, live]
        z, zm = z + e @ w2l, zm + np.abs(e) @ np.abs(w2l)
    if lm_bias is not None:
        b = np.asarray(lm_bias, np.float64)[live]
        z, zm = z + b, zm + np.abs(b)
    mag["z"] = float(zm.max())
    m = z.max(1, keepdims=True)
    logp = z - m - np.log(np.exp(z - m).sum(1, keepdims=True))
    q = np.zeros_like(z)
    for i, t in enumerate(tok):
        on = col[t] >= 0
        a = t_scale * s[t, on]
        if lse is None:
            top = a.max()
            lq = a - top - np.log(np.exp(a - top).sum())
        else:
            lq = a - float(lse[t])
        at = place[col[t, on]]
        q[i, at] = np.exp(lq)
        term = np.where(np.exp(lq) > 0, np.exp(lq) * (lq - logp[i, at]), 0.0)
        out["loss"][t] = term.sum()
        mag["loss"][t] = np.sum(np.exp(lq) * (np.abs(a) + np.abs(lq) + np.abs(logp[i, at])))
    Q = q.sum(1, keepdims=True)
    mag["q"] = float(Q.max())
    wt = w[tok]
    D = wt.sum() if reduction == "mean" else 1.0
    f = loss_scale * wt / D if D > 0 else np.zeros_like(wt)
    out["total"] = float((f * out["loss"][tok]).sum())
    mag["total"] = float((np.abs(f) * mag["loss"][tok]).sum())
    p = np.exp(logp)
    dz, dm = f[:, None] * (Q * p - q), np.abs(f)[:, None] * (Q * p + q)
    out["d_hidden"][tok], mag["d_hidden"][tok] = dz @ Wl, dm @ np.abs(Wl)
    out["d_lm_head"][live], mag["d_lm_head"][live] = dz.T @ x, dm.T @ np.abs(x)
    if w1 is not None:
        np.add.at(out["d_markov_w1"], np.asarray(prev)[tok], dz @ w2l.T)
        np.add.at(mag["d_markov_w1"], np.asarray(prev)[tok], dm @ np.abs(w2l).T)
        out["d_markov_w2"][:, live], mag["d_markov_w2"][:, live] = e.T @ dz, np.abs(e).T @ dm
    return out
