"""Plain fp64 scoring of given tokens (numpy): log-probabilities, entropy, alternatives, gradients.

Written from the definitions; shares no code with the CUDA path or with the loss's oracle.
"""
from __future__ import annotations

import numpy as np

__all__ = ["score", "alternatives", "logits_gradient", "projected", "projected_gradients"]


def _log_softmax(z):
    """log q per row, in fp64; rows whose logits are all -inf give -inf throughout."""
    m = z.max(axis=1, keepdims=True)
    safe = np.where(np.isneginf(m), 0.0, m)
    with np.errstate(divide="ignore", invalid="ignore"):
        log_s = np.log(np.exp(z - safe).sum(axis=1, keepdims=True))
        lq = z - safe - log_s
    return np.where(np.isneginf(m), -np.inf, lq), m[:, 0], np.where(np.isneginf(m), 0.0, log_s)[:, 0]


def score(logits, tokens):
    """(logp [N, T], entropy [N], m [N], log_s [N])."""
    z = np.asarray(logits, dtype=np.float64)
    lq, m, log_s = _log_softmax(z)
    q = np.exp(lq)
    entropy = -np.where(q > 0, q * np.where(q > 0, lq, 0.0), 0.0).sum(axis=1)
    tokens = np.asarray(tokens, dtype=np.int64)
    logp = np.take_along_axis(lq, np.maximum(tokens, 0), axis=1)
    return np.where(tokens < 0, 0.0, logp), entropy, m, log_s


def alternatives(logits, top):
    """(ids [N, top], log-probabilities): largest logits first, equal ones by smaller id."""
    z = np.asarray(logits, dtype=np.float64)
    ids = np.argsort(-z, axis=1, kind="stable")[:, :top]
    return ids, np.take_along_axis(_log_softmax(z)[0], ids, axis=1)


def logits_gradient(logits, tokens, g_logp, g_entropy=None):
    """d/dz of sum g_logp logp + sum g_entropy entropy, [N, V]."""
    z = np.asarray(logits, dtype=np.float64)
    lq, m, _ = _log_softmax(z)
    q = np.exp(lq)
    lq0 = np.where(q > 0, lq, 0.0)
    tokens = np.asarray(tokens, dtype=np.int64)
    g = np.where(tokens < 0, 0.0, np.asarray(g_logp, dtype=np.float64))
    ge = np.zeros(len(z)) if g_entropy is None else np.asarray(g_entropy, dtype=np.float64)
    entropy = -(q * lq0).sum(axis=1)
    dz = -q * (g.sum(axis=1, keepdims=True) + ge[:, None] * (lq0 + entropy[:, None]))
    for n, t in zip(*np.nonzero(tokens >= 0)):
        dz[n, tokens[n, t]] += g[n, t]
    dz[np.isneginf(m)] = 0.0
    return dz


def projected(H, W, tokens):
    """score() of the logits H W^T, with the log-partition: (logp, entropy, lse)."""
    z = np.asarray(H, dtype=np.float64) @ np.asarray(W, dtype=np.float64).T
    logp, entropy, m, log_s = score(z, tokens)
    return logp, entropy, m + log_s


def projected_gradients(H, W, tokens, g_logp, g_entropy=None):
    """(dH, dW) of sum g_logp logp + sum g_entropy entropy."""
    H = np.asarray(H, dtype=np.float64)
    W = np.asarray(W, dtype=np.float64)
    dz = logits_gradient(H @ W.T, tokens, g_logp, g_entropy)
    return dz @ W, dz.T @ H
