"""Plain fp64 forms (numpy) of the tied embedding, the gradients' norm and the logit rules.

Written from the definitions; shares no code with the CUDA path or with the other oracles.
"""
from __future__ import annotations

import numpy as np

__all__ = ["embedding", "embedding_gradient", "norm", "clip", "adjust", "adjust_gradient"]


def embedding(W, tokens, scale=1.0):
    """[*tokens.shape, d]; zeros where the token is -1."""
    W = np.asarray(W, dtype=np.float64)
    out = np.zeros((*tokens.shape, W.shape[1]))
    for at in np.ndindex(tokens.shape):
        if tokens[at] >= 0:
            out[at] = scale * W[tokens[at]]
    return out


def embedding_gradient(g, tokens, V, scale=1.0, old=None):
    """(dW [V, d], sum of |g| per row and column, number of positions per row)."""
    g = np.asarray(g, dtype=np.float64)
    dW, size, count = np.zeros((V, g.shape[-1])), np.zeros((V, g.shape[-1])), np.zeros(V, dtype=np.int64)
    for at in np.ndindex(tokens.shape):
        t = tokens[at]
        if 0 <= t < V:
            dW[t] += g[at]
            size[t] += np.abs(g[at])
            count[t] += 1
    return scale * dW + (0 if old is None else np.asarray(old, dtype=np.float64)), size, count


def norm(tensors):
    return float(np.sqrt(sum(np.square(np.asarray(t, dtype=np.float64)).sum() for t in tensors)))


def clip(tensors, max_norm):
    """(norm, coefficient, scaled tensors)."""
    n = norm(tensors)
    c = min(1.0, max_norm / (n + 1e-6))
    return n, c, [np.asarray(t, dtype=np.float64) * c for t in tensors]


def _history(n, history, lengths, prompt):
    """(tokens seen, {token: times generated}) of row n."""
    if history is None:
        return set(), {}
    L = history.shape[1]
    m = L if lengths is None else min(max(int(lengths[n]), 0), L)
    p = 0 if prompt is None else int(prompt[n])
    seen, made = set(), {}
    for i in range(m):
        t = int(history[n, i])
        if t < 0:
            continue
        seen.add(t)
        if i >= p:
            made[t] = made.get(t, 0) + 1
    return seen, made


def _keep(n, allowed, V):
    if allowed is None:
        return np.ones(V, dtype=bool)
    words = np.asarray(allowed if allowed.ndim == 1 else allowed[n]).astype(np.int64) & 0xffffffff
    return np.array([(int(words[v // 32]) >> (v % 32)) & 1 == 1 for v in range(V)])


def _each(x, n):
    return float(x) if np.ndim(x) == 0 else float(x[n])


def adjust(z, history=None, lengths=None, prompt=None, r=1.0, f=0.0, p=0.0, bias_tokens=None, bias=None, allowed=None):
    """(adjusted logits [N, V], the largest size of any intermediate value [N, V])."""
    z = np.array(z, dtype=np.float64)
    size = np.abs(z)
    for n in range(z.shape[0]):
        seen, made = _history(n, history, lengths, prompt)
        for t in seen:
            z[n, t] = z[n, t] / _each(r, n) if z[n, t] > 0 else z[n, t] * _each(r, n)
            size[n, t] = max(size[n, t], abs(z[n, t]))
        for t, c in made.items():
            z[n, t] -= _each(f, n) * c + _each(p, n)
            size[n, t] += abs(_each(f, n)) * c + abs(_each(p, n))
        if bias is not None:
            for t, b in zip(bias_tokens[n], bias[n]):
                if t >= 0:
                    z[n, t] += float(b)
                    size[n, t] += abs(float(b))
        z[n, ~_keep(n, allowed, z.shape[1])] = -np.inf
    return z, size


def adjust_gradient(g, z, history=None, lengths=None, r=1.0, allowed=None):
    """Gradient [N, V] with respect to the logits."""
    dz = np.array(g, dtype=np.float64)
    for n in range(dz.shape[0]):
        for t in _history(n, history, lengths, None)[0]:
            dz[n, t] *= 1 / _each(r, n) if z[n, t] > 0 else _each(r, n)
        dz[n, ~_keep(n, allowed, dz.shape[1])] = 0.0
    return dz
