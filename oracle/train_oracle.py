"""Plain fp64 definitions of the head's training operators (test infrastructure only).

Values are computed from the exact inputs the GPU reads.  Beside each gradient stands the
sum of the magnitudes of its terms, from which the tests derive rounding bounds.
"""
from __future__ import annotations

import numpy as np

MASK_LEVEL = -1.0e8


def label_rows(labels, V, V_head, d2t=None, lm_bias=None):
    """Head row of every label, -1 for a row that carries no loss."""
    out = []
    where = None if d2t is None else {int(v): j for j, v in enumerate(d2t)}
    for t in labels:
        t = int(t)
        j = -1
        if 0 <= t < V:
            j = t if where is None else where.get(t, -1)
        if j >= 0 and lm_bias is not None and not lm_bias[j] > MASK_LEVEL:
            j = -1
        out.append(j)
    return np.array(out, dtype=np.int64)


def head_loss(hidden, lm_head, labels, prev=None, w1=None, w2=None, lm_bias=None, d2t=None,
              weights=None, reduction="mean", loss_scale=1.0, V=None):
    """Losses, total, and the gradients of the total, as a dict; ``mag`` holds, under the
    gradients' names, the sums of their terms' magnitudes, and ``mag["z"]`` the largest such
    sum of a logit."""
    h, W = np.asarray(hidden, np.float64), np.asarray(lm_head, np.float64)
    T, Vh = h.shape[0], W.shape[0]
    V = Vh if V is None else V
    rows = label_rows(labels, V, Vh, d2t, lm_bias)
    live = np.ones(Vh, bool) if lm_bias is None else np.asarray(lm_bias) > MASK_LEVEL
    tok = np.nonzero(rows >= 0)[0]
    if w1 is not None:
        w1, w2 = np.asarray(w1, np.float64), np.asarray(w2, np.float64)
        p = np.asarray(prev)[tok]
    w = np.ones(T) if weights is None else np.asarray(weights, np.float64)
    out = {"loss": np.zeros(T), "total": 0.0, "n_rows": len(tok),
           "d_hidden": np.zeros_like(h), "d_lm_head": np.zeros_like(W)}
    mag = {"d_hidden": np.zeros_like(h), "d_lm_head": np.zeros_like(W), "z": 0.0}
    if w1 is not None:
        out["d_markov_w1"], out["d_markov_w2"] = np.zeros_like(w1), np.zeros_like(w2)
        mag["d_markov_w1"], mag["d_markov_w2"] = np.zeros_like(w1), np.zeros_like(w2)
    out["mag"] = mag
    if len(tok) == 0:
        return out
    x, Wl = h[tok], W[live]
    z = x @ Wl.T
    zm = np.abs(x) @ np.abs(Wl).T
    if w1 is not None:
        e, w2l = w1[p], w2[:, live]
        z = z + e @ w2l
        zm = zm + np.abs(e) @ np.abs(w2l)
    if lm_bias is not None:
        z = z + np.asarray(lm_bias, np.float64)[live]
        zm = zm + np.abs(np.asarray(lm_bias, np.float64)[live])
    mag["z"] = zm.max()
    m = z.max(axis=1, keepdims=True)
    lse = m[:, 0] + np.log(np.exp(z - m).sum(axis=1))
    at = np.cumsum(live)[rows[tok]] - 1
    nll = lse - z[np.arange(len(tok)), at]
    out["loss"][tok] = nll
    D = w[tok].sum() if reduction == "mean" else 1.0
    k = loss_scale / D if D != 0 else 0.0
    out["total"] = k * (w[tok] * nll).sum()
    q = np.exp(z - lse[:, None])
    q[np.arange(len(tok)), at] -= 1.0
    q *= w[tok][:, None]
    aq = np.abs(q)
    out["d_hidden"][tok] = k * (q @ Wl)
    mag["d_hidden"][tok] = abs(k) * (aq @ np.abs(Wl))
    out["d_lm_head"][live] = k * (q.T @ x)
    mag["d_lm_head"][live] = abs(k) * (aq.T @ np.abs(x))
    if w1 is not None:
        np.add.at(out["d_markov_w1"], p, k * (q @ w2l.T))
        np.add.at(mag["d_markov_w1"], p, abs(k) * (aq @ np.abs(w2l).T))
        out["d_markov_w2"][:, live] = k * (e.T @ q)
        mag["d_markov_w2"][:, live] = abs(k) * (np.abs(e).T @ aq)
    return out


def block_norm(x, y, w_pre, gate=None, w_post=None, eps=1e-6, scale=1.0, offset=0.0, span=1):
    """(x_out, h)."""
    x = np.asarray(x, np.float64)
    xo = x
    if y is not None:
        u = np.asarray(y, np.float64)
        if w_post is not None:
            u = u / np.sqrt((u * u).mean(1, keepdims=True) + eps) * (offset + w_post)
        if gate is not None:
            u = u * np.asarray(gate, np.float64)[np.arange(x.shape[0]) // span]
        xo = x + scale * u
    return xo, xo / np.sqrt((xo * xo).mean(1, keepdims=True) + eps) * (offset + w_pre)


def block_norm_backward(x, y, w_pre, d_h, d_x_out=None, gate=None, w_post=None, eps=1e-6,
                        scale=1.0, offset=0.0, span=1):
    """Gradients as a dict, with ``mag`` as in :func:`head_loss`."""
    x, dh = np.asarray(x, np.float64), np.asarray(d_h, np.float64)
    T = x.shape[0]
    up = np.zeros_like(x) if d_x_out is None else np.asarray(d_x_out, np.float64)
    xo, _ = block_norm(x, y, w_pre, gate, w_post, eps, scale, offset, span)
    rx = 1.0 / np.sqrt((xo * xo).mean(1, keepdims=True) + eps)
    xn = xo * rx
    xm = (np.abs(x) + np.abs(xo - x)) * rx        # the terms of xn: x' may cancel
    a = dh * (offset + w_pre)
    dx = up + rx * (a - xn * (a * xn).mean(1, keepdims=True))
    mx = np.abs(up) + rx * (np.abs(a) + xm * (np.abs(a) * xm).mean(1, keepdims=True))
    d = {"d_x": dx, "d_w_pre": (dh * xn).sum(0)}
    mag = {"d_x": mx, "d_w_pre": (np.abs(dh) * xm).sum(0)}
    if y is not None:
        y = np.asarray(y, np.float64)
        ry = 1.0 / np.sqrt((y * y).mean(1, keepdims=True) + eps) if w_post is not None else 1.0
        ow = offset + w_post if w_post is not None else 1.0
        yn = y * ry
        g = 1.0
        if gate is not None:
            rows = np.arange(T) // span
            g = np.asarray(gate, np.float64)[rows]
            d["d_gate"], mag["d_gate"] = np.zeros_like(gate, np.float64), np.zeros_like(
                gate, np.float64)
            np.add.at(d["d_gate"], rows, scale * dx * yn * ow)
            np.add.at(mag["d_gate"], rows, np.abs(scale * mx * yn * ow))
        du, mu = scale * g * dx, np.abs(scale * g) * mx
        if w_post is None:
            d["d_y"], mag["d_y"] = du, mu
        else:
            d["d_w_post"], mag["d_w_post"] = (du * yn).sum(0), np.abs(mu * yn).sum(0)
            b, mb = du * ow, mu * np.abs(ow)
            d["d_y"] = ry * (b - yn * (b * yn).mean(1, keepdims=True))
            mag["d_y"] = ry * (mb + np.abs(yn) * np.abs(mb * yn).mean(1, keepdims=True))
    d["mag"] = mag
    return d


def clip_grads(grads, max_norm):
    """(norm, clipped gradients)."""
    norm = np.sqrt(sum(float((np.asarray(g, np.float64) ** 2).sum()) for g in grads))
    k = min(1.0, max_norm / (norm + 1e-6)) if np.isfinite(norm) else 1.0
    return norm, [np.asarray(g, np.float64) * k for g in grads]
