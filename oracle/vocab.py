"""Float64 oracle of the vocabulary operators: softmax cross entropy and log
probabilities over an output head, embedding lookup, and their gradients,
straight from the definitions (numpy, whole logits, no blocking)."""

from __future__ import annotations

import numpy as np


def cross_entropy(x, w, targets, weights=None, mean=True, logit_scale=1.0, grad_scale=1.0):
    """x (n, d), w (v, d), targets (n,), below zero: not counted.  Returns loss,
    lse (n), total, dx, dw, and dz (the gradient of the logits x w^T)."""
    targets = np.asarray(targets)
    counted = targets >= 0
    # A row that is not counted has no part in anything, whatever it holds.
    x = np.where(counted[:, None], np.asarray(x, np.float64), 0.0)
    w = np.asarray(w, np.float64)
    a = np.where(counted, 1.0 if weights is None else np.asarray(weights, np.float64), 0.0)
    z = logit_scale * (x @ w.T)
    top = z.max(axis=1, keepdims=True)
    e = np.exp(z - top)
    sums = e.sum(axis=1, keepdims=True)
    lse = (top + np.log(sums))[:, 0]
    rows = np.arange(len(targets))
    at = np.where(counted, targets, 0)
    loss = np.where(counted, lse - z[rows, at], 0.0)
    norm = a.sum() if mean else 1.0
    coef = a / norm if norm != 0 else np.zeros_like(a)
    onehot = np.zeros_like(z)
    onehot[rows, at] = 1.0
    dz = (grad_scale * logit_scale * coef)[:, None] * (e / sums - onehot)
    return {"loss": loss, "lse": np.where(counted, lse, 0.0), "total": float((coef * loss).sum()),
            "dx": dz @ w, "dw": dz.T @ x, "dz": dz}


def embed(ids, table, scale=1.0):
    ids = np.asarray(ids)
    rows = np.asarray(table, np.float64)[np.maximum(ids, 0)] * scale
    return np.where((ids >= 0)[:, None], rows, 0.0)


def embed_grad(ids, dout, vocab, scale=1.0, base=None):
    """The whole table's gradient, added to ``base`` if given."""
    dout = np.asarray(dout, np.float64)
    out = np.zeros((vocab, dout.shape[1])) if base is None else np.array(base, np.float64)
    for i, t in enumerate(np.asarray(ids)):
        if t >= 0:
            out[t] += scale * dout[i]
    return out


def token_logprobs(x, w, tokens=None, logit_scale=1.0, n_top=0, dlogprobs=None, dentropy=None, grad_scale=1.0):
    """Log probabilities of ``tokens`` (below zero: not scored; None: every row
    scored, no token given), lse, entropy, the n_top most likely ids (equal
    logits by ascending id) with theirs, and the gradients of
    sum(dlogprobs * logprobs + dentropy * entropy)."""
    n = len(x)
    given = np.full(n, tokens is not None)
    tokens = np.zeros(n, np.int64) if tokens is None else np.asarray(tokens)
    scored = tokens >= 0
    given &= scored
    x = np.where(scored[:, None], np.asarray(x, np.float64), 0.0)
    w = np.asarray(w, np.float64)
    z = logit_scale * (x @ w.T)
    top = z.max(axis=1, keepdims=True)
    lse = top[:, 0] + np.log(np.exp(z - top).sum(axis=1))
    logp = z - lse[:, None]
    p = np.exp(logp)
    entropy = -(p * logp).sum(axis=1)
    rows = np.arange(n)
    at = np.where(given, tokens, 0)
    order = np.argsort(-z, axis=1, kind="stable")[:, :n_top]
    zero = np.zeros(n)
    g = np.where(given, zero if dlogprobs is None else np.asarray(dlogprobs, np.float64), 0.0)
    h = np.where(scored, zero if dentropy is None else np.asarray(dentropy, np.float64), 0.0)
    dz = -p * (g[:, None] + h[:, None] * (logp + entropy[:, None]))
    dz[rows, at] += g
    dz *= grad_scale * logit_scale
    return {"logprobs": np.where(given, logp[rows, at], 0.0), "lse": np.where(scored, lse, 0.0),
            "entropy": np.where(scored, entropy, 0.0), "top_ids": np.where(scored[:, None], order, -1),
            "top_logprobs": np.where(scored[:, None], np.take_along_axis(logp, order, axis=1), 0.0),
            "dx": dz @ w, "dw": dz.T @ x, "dz": dz, "logp": logp}
