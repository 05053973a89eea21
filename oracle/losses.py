"""Losses of a packed batch in 64 bits: the plain statement of what the CUDA
loss kernels compute.

TEST INFRASTRUCTURE ONLY, like the rest of this package.  NumPy float64 row by
row, from the formulas; masked rows are never touched, so nothing they hold can
reach a result.
"""

from __future__ import annotations

import numpy as np

from .thd_oracle import zigzag_partition

TOKEN_MEAN, DOC_MEAN, TOKEN_SUM = 0, 1, 2


def row_documents(cu, cp=1):
    """Document of each row in the zigzag layout of cp ranks (cp = 1: contiguous)."""
    doc_of_row = [i for i in range(len(cu) - 1) for _ in range(cu[i], cu[i + 1])]
    if cp == 1:
        return np.array(doc_of_row, dtype=np.int64)
    return np.array([doc_of_row[g] for rank in zigzag_partition(list(cu), cp) for g in rank], dtype=np.int64)


def loss_weights(mask, cu, cp=1, reduction=TOKEN_MEAN):
    mask = np.asarray(mask)
    docs = row_documents(cu, cp)
    n = [int((mask[docs == i] != 0).sum()) for i in range(len(cu) - 1)]
    w = np.zeros(len(mask))
    for t in range(len(mask)):
        if mask[t]:
            if reduction == TOKEN_SUM:
                w[t] = 1.0
            elif reduction == TOKEN_MEAN:
                w[t] = 1.0 / sum(n)
            else:
                w[t] = 1.0 / (n[docs[t]] * sum(1 for k in n if k > 0))
    return w, docs


def log_softmax(z, tau):
    """(log-probabilities, log-sum-exp) of one row.  A row of which nothing is
    above -inf has log-probabilities and log-sum-exp -inf."""
    x = np.asarray(z, dtype=np.float64) / tau
    if np.all(x == -np.inf):
        return x, -np.inf
    top = x.max()
    if not np.isfinite(top):
        top = 0.0
    log_sum = np.log(np.exp(x - top).sum())
    return (x - top) - log_sum, top + log_sum


def token_logprobs(z, labels, mask=None, tau=1.0):
    T = len(labels)
    lp, lse = np.zeros(T), np.zeros(T)
    for t in range(T):
        if mask is None or mask[t]:
            logp, lse[t] = log_softmax(z[t], tau)
            lp[t] = logp[labels[t]]
    return lp, lse


def token_logprobs_backward(z, labels, g, tau=1.0):
    d = np.zeros(np.shape(z))
    for t in range(len(labels)):
        if g[t] != 0:
            logp, lse = log_softmax(z[t], tau)
            if lse == -np.inf:
                continue
            d[t] = -g[t] * np.exp(logp) / tau
            d[t, labels[t]] = g[t] * -np.expm1(logp[labels[t]]) / tau
    return d


def policy_loss(z, labels, w, old, advantages, ref=None, docs=None, clip_low=0.2, clip_high=0.2, kl_coef=0.0,
                tau=1.0):
    """dict(loss, kl, clip_fraction, logprobs, dlogits)."""
    T = len(labels)
    lp = np.zeros(T)
    g = np.zeros(T)
    loss = kl_sum = clipped = 0.0
    for t in range(T):
        if w[t] == 0:
            continue
        logp, _ = log_softmax(z[t], tau)
        lp[t] = logp[labels[t]]
        A = float(advantages[docs[t]] if docs is not None else advantages[t])
        r = np.exp(lp[t] - float(old[t]))
        bounded = min(max(r, 1 - clip_low), 1 + clip_high)
        cut = r * A > bounded * A
        kl = slope = 0.0
        if ref is not None:
            d = float(ref[t]) - lp[t]
            kl = np.expm1(d) - d
            slope = -kl_coef * np.expm1(d)
        loss += w[t] * (-(bounded if cut else r) * A + kl_coef * kl)
        kl_sum += w[t] * kl
        clipped += w[t] * cut
        g[t] = w[t] * (slope - (0.0 if cut else r * A))
    return dict(loss=loss, kl=kl_sum, clip_fraction=clipped, logprobs=lp, dlogits=token_logprobs_backward(z, labels, g, tau))


def preference_loss(lp, mask, cu, chosen, rejected, ref=None, cp=1, beta=0.1, label_smoothing=0.0, margin=0.0,
                    length_normalized=False):
    """dict(loss, margins, doc_logprobs, dlogprobs)."""
    docs = row_documents(cu, cp)
    N = len(cu) - 1
    rows = [[t for t in range(len(mask)) if mask[t] and docs[t] == i] for i in range(N)]
    per = [len(r) if length_normalized and r else 1 for r in rows]
    s = np.array([sum(float(lp[t]) for t in rows[i]) / per[i] for i in range(N)])
    u = np.array([sum(float(lp[t]) - (float(ref[t]) if ref is not None else 0.0) for t in rows[i]) / per[i]
                  for i in range(N)])
    P = len(chosen)
    h = np.array([beta * (u[c] - u[r]) for c, r in zip(chosen, rejected)])
    loss = 0.0
    ds = np.zeros(N)
    for c, r, m in zip(chosen, rejected, h):
        x = m - margin
        loss += ((1 - label_smoothing) * np.logaddexp(0.0, -x) + label_smoothing * np.logaddexp(0.0, x)) / P
        dh = (label_smoothing * np.exp(-np.logaddexp(0.0, -x)) - (1 - label_smoothing) * np.exp(-np.logaddexp(0.0, x))) / P
        ds[c] += beta * dh
        ds[r] -= beta * dh
    g = np.zeros(len(mask))
    for i in range(N):
        for t in rows[i]:
            g[t] = ds[i] / per[i]
    return dict(loss=loss, margins=h, doc_logprobs=s, dlogprobs=g)


def distill_topk_loss(z, ids, scores, w, tau=1.0, normalize=True):
    """dict(loss, token_losses, dlogits)."""
    T, V = np.shape(z)
    losses = np.zeros(T)
    d = np.zeros((T, V))
    for t in range(T):
        if w[t] == 0:
            continue
        logp, lse = log_softmax(z[t], tau)
        here = [(int(i), float(s)) for i, s in zip(ids[t], scores[t]) if 0 <= i < V]
        here = [(i, s) for i, s in here if s != -np.inf]
        if not here:
            continue
        s = np.array([v for _, v in here])
        lq = log_softmax(s, tau)[0] if normalize else s
        q = np.exp(lq)
        losses[t] = tau * tau * sum(q[k] * (lq[k] - logp[i]) for k, (i, _) in enumerate(here) if q[k] != 0)
        if lse == -np.inf:
            continue
        d[t] = q.sum() * np.exp(logp)
        for k, (i, _) in enumerate(here):
            d[t, i] -= q[k]
        d[t] *= w[t] * tau
    return dict(loss=float((np.asarray(w) * losses)[np.asarray(w) != 0].sum()), token_losses=losses, dlogits=d)
