"""float64 numpy forms of the dense operators around the routed experts: token
log probabilities, the gated block and adapters, with their gradients.  Each
follows its definition; nothing here is shared with the GPU path."""

from __future__ import annotations

import numpy as np


def token_logprobs(logits: np.ndarray, tokens: np.ndarray, top: int = 0) -> dict:
    """logits [M, V] (any float type, read as they are), tokens [M]."""
    l = logits.astype(np.float64)
    M, V = l.shape
    out = dict(logprobs=np.zeros(M), entropy=np.zeros(M), lse=np.zeros(M),
               top_ids=np.zeros((M, top), np.int64), top_logprobs=np.zeros((M, top)))
    with np.errstate(invalid="ignore", divide="ignore"):
        for m in range(M):
            r = l[m]
            if np.all(r == -np.inf):
                lse, logp, ent = -np.inf, np.full(V, -np.inf), 0.0
            elif np.isnan(r).any() or (r == np.inf).any():
                lse, logp, ent = np.nan, np.full(V, np.nan), np.nan
            else:
                x = r - r.max()
                lz = np.log(np.exp(x).sum())
                lse, logp = r.max() + lz, x - lz
                p = np.exp(logp)
                ent = -np.where(p > 0, p * np.where(p > 0, logp, 0.0), 0.0).sum()
            out["lse"][m], out["entropy"][m] = lse, ent
            if 0 <= tokens[m] < V:
                out["logprobs"][m] = logp[tokens[m]]
            # NaN after everything, then by logit, then by id
            order = np.lexsort((np.arange(V), -np.where(np.isnan(r), -np.inf, r), np.isnan(r)))
            out["top_ids"][m] = order[:top]
            out["top_logprobs"][m] = logp[order[:top]]
    return out


def token_logprobs_backward(logits, tokens, lse, entropy, g, h) -> np.ndarray:
    """From the lse and entropy given, g and h the gradients of logprobs and
    entropy."""
    l = logits.astype(np.float64)
    out = np.zeros_like(l)
    for m in range(l.shape[0]):
        if lse[m] < -2.0 ** 24:      # ruled out from end to end
            continue
        logp = l[m] - np.float64(lse[m])
        p = np.exp(logp)
        gm = np.float64(g[m]) if 0 <= tokens[m] < l.shape[1] else 0.0
        inner = gm + np.float64(h[m]) * (np.where(p > 0, logp, 0.0) + np.float64(entropy[m]))
        out[m] = -p * inner
        if gm:
            out[m, tokens[m]] += gm
    return out


def gated(x: np.ndarray, w13: np.ndarray) -> np.ndarray:
    """x [M, H], w13 [2I, H], float64."""
    I = w13.shape[0] // 2
    g, u = x @ w13[:I].T, x @ w13[I:].T
    return g / (1.0 + np.exp(-g)) * u


def gated_backward(x, w13, d):
    """(grad_x, grad_w13) for the gradient d [M, I] of gated's output."""
    I = w13.shape[0] // 2
    g, u = x @ w13[:I].T, x @ w13[I:].T
    s = 1.0 / (1.0 + np.exp(-g))
    both = np.concatenate([d * u * (s + g * s * (1.0 - s)), d * g * s], axis=1)
    return both @ w13, both.T @ x


def adapters(x, a, b, scales, slots, addend=None, is_gated=False):
    """x [M, K], a [S, R, K], b [S, N, R], scales [S] or None, float64."""
    S = a.shape[0]
    y = np.zeros((x.shape[0], b.shape[1])) if addend is None else addend.astype(np.float64)
    y = y.copy()
    for m, s in enumerate(slots):
        if 0 <= s < S:
            y[m] += (1.0 if scales is None else float(scales[s])) * (b[s] @ (a[s] @ x[m]))
    if is_gated:
        n = y.shape[1] // 2
        y = y[:, :n] / (1.0 + np.exp(-y[:, :n])) * y[:, n:]
    return y
