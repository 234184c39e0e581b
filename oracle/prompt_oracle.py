"""Float64 oracle of the operators around a prompt: the norm with its 8-bit output, log probabilities, and the
attention of packed prompts. Plain statements of the formulas, a row at a time."""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


def add_rmsnorm(x, residual, weight, eps: float, group: int):
    """x, residual [n, D] and weight [D] float64. Returns h, y and the largest magnitude of each block [n, blocks]."""
    h = x if residual is None else x + residual
    y = h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * weight
    n, dim = y.shape
    width = group or dim
    amax = np.stack([np.abs(y[:, b:b + width]).max(1) for b in range(0, dim, width)], 1)
    return h, y, amax


def token_logprobs(x, tokens, top: int, scale: float = 1.0):
    """x [n, V] float64. Returns log p of the tokens, the entropy, the ids of the `top` largest logits (the lower id at
    a tie, -1 behind the last) and their log p."""
    z = x * scale
    with np.errstate(all="ignore"):
        m = z.max(1, keepdims=True)
        lp = z - m - np.log(np.exp(z - m).sum(1, keepdims=True))
        ent = -np.where(np.exp(lp) > 0, np.exp(lp) * lp, np.where(np.isnan(lp), np.nan, 0.0)).sum(1)
    n, v = x.shape
    given = np.zeros(tokens.shape)
    for r in range(n):
        for g, t in enumerate(tokens[r]):
            given[r, g] = 0.0 if t == -1 else lp[r, t] if 0 <= t < v else np.nan
    ids = np.full((n, top), -1, dtype=np.int64)
    alt = np.full((n, top), -np.inf)
    order = np.argsort(-(x + 0.0), axis=1, kind="stable")[:, :top]
    ids[:, :order.shape[1]] = order
    alt[:, :order.shape[1]] = np.take_along_axis(lp, order, 1)
    return given, ent, ids, alt


def visible(nq: int, nk: int, causal: bool, prefix: int = 0):
    """How many keys, from the first on, query i of nq sees of nk: its own position and what stands before it (the
    queries are the last of the keys), or the prefix where that reaches further."""
    i = np.arange(nq)
    if not causal:
        return np.full(nq, nk)
    return np.clip(np.maximum(nk - nq + i + 1, min(max(prefix, 0), nk)), 0, nk)


def prompt_attention(q, k, v, rope, cu_q, cu_k, sm_scale, causal=True, prefix=None, cap=0.0, slopes=None, sink=None):
    """q [T, H, 128 + rope], k and v [N, HK, 128], rope [N, 64] or None, float64. Rows of no request are NaN.
    Returns out [T, H, 128], lse [T, H], and A = sum p |v| with the largest |score term sum| of each row for bounds."""
    T, H, _ = q.shape
    HK = k.shape[1]
    out, lse = np.full((T, H, 128), np.nan), np.full((T, H), np.nan)
    A, big = np.zeros((T, H, 128)), np.zeros((T, H))
    for r in range(len(cu_q) - 1):
        q0, q1, k0, k1 = int(cu_q[r]), int(cu_q[r + 1]), int(cu_k[r]), int(cu_k[r + 1])
        nq, nk = q1 - q0, k1 - k0
        lim = visible(nq, nk, causal, 0 if prefix is None else int(prefix[r]))
        pos = nk - nq + np.arange(nq)
        hide = np.arange(nk)[None, :] >= lim[:, None]
        for h in range(H):
            key = k[k0:k1, h // (H // HK)]
            if rope is not None:
                key = np.concatenate([key, rope[k0:k1]], 1)
            val = v[k0:k1, h // (H // HK)]
            with np.errstate(all="ignore"):
                s = q[q0:q1, h] @ key.T * sm_scale
                mag = np.abs(q[q0:q1, h]) @ np.abs(key).T * abs(sm_scale)
                if cap:
                    s = cap * np.tanh(s / cap)
                if slopes is not None:
                    bias = slopes[h] * np.abs(pos[:, None] - np.arange(nk)[None, :])
                    s, mag = s - bias, mag + np.abs(bias)
                s = np.where(hide, -np.inf, s)
                mag = np.where(hide, 0.0, mag)
                top = np.full(nq, -np.inf if sink is None else float(sink[h]))
                if nk:
                    top = np.fmax(top, s.max(1))
                m = np.where(np.isfinite(top), top, 0.0)
                w = np.where(hide, 0.0, np.exp(s - m[:, None]))
                den = w.sum(1) + (0.0 if sink is None else np.exp(sink[h] - m))
                lse[q0:q1, h] = np.log(den) + m
                safe = np.where(den == 0, 1.0, den)
                # what a row does not see never reaches it, whatever its value
                for a in range(nq):
                    n = int(lim[a])
                    out[q0 + a, h] = (w[a, :n] @ val[:n]) / safe[a]
                    A[q0 + a, h] = (w[a, :n] @ np.abs(val[:n])) / safe[a]
                big[q0:q1, h] = mag.max(1) if nk else 0.0
    return out, lse, A, big
