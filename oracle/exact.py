"""Exact losses and gradients beside the estimators, in fp64: scores of a
head's logits, distillation from a teacher's top logits, and causal attention
with its gradient.

TEST INFRASTRUCTURE ONLY (see the package docstring).

These have no counterpart in the Dust pages, which train on hard-label
cross-entropy; they are the usual definitions:

* log softmax, entropy in nats, alternatives by descending logit with ties to
  the lower index;
* temperature^2 KL(teacher || student) with the teacher renormalised over the
  entries it kept;
* softmax attention with pairs j <= i of one sequence.
"""
from __future__ import annotations

import numpy as np


def _log_softmax_row(z):
    """Log softmax of one row; None for a row without a distribution (NaN or
    +inf), all -inf for a row of -inf alone."""
    if np.isnan(z).any() or np.isposinf(z).any():
        return None
    if np.isneginf(z).all():
        return z.copy()
    m = z.max()
    return z - m - np.log(np.exp(z - m).sum())


def token_logprobs(Z, tokens, top: int = 0) -> dict:
    Z = np.asarray(Z, dtype=np.float64)
    T = Z.shape[0]
    out = {"logp": np.zeros(T), "entropy": np.zeros(T),
           "top_ids": np.full((T, top), -1, dtype=np.int64),
           "top_logp": np.full((T, top), -np.inf)}
    for t in range(T):
        lp = _log_softmax_row(Z[t])
        if lp is None:
            out["logp"][t] = np.nan if tokens[t] >= 0 else 0.0
            out["entropy"][t] = np.nan
            out["top_logp"][t] = np.nan
            continue
        if tokens[t] >= 0:
            out["logp"][t] = lp[tokens[t]]
        live = np.flatnonzero(np.isfinite(lp))
        out["entropy"][t] = -(np.exp(lp[live]) * lp[live]).sum()
        best = live[np.argsort(-Z[t, live], kind="stable")][:top]
        out["top_ids"][t, :best.size] = best
        out["top_logp"][t, :best.size] = lp[best]
    return out


def distill(Z, ids, vals, temperature=1.0, weights=None) -> dict:
    Z = np.asarray(Z, dtype=np.float64)
    T, V = Z.shape
    loss, dZ = np.zeros(T), np.zeros((T, V))
    for t in range(T):
        w = 1.0 if weights is None else float(weights[t])
        kept = [(int(i), float(v)) for i, v in zip(ids[t], vals[t]) if i >= 0 and v != -np.inf]
        if not kept or w == 0.0:
            continue
        v = np.array([x for _, x in kept]) / temperature
        lq = v - v.max()
        lq -= np.log(np.exp(lq).sum())
        lp = _log_softmax_row(Z[t] / temperature)
        if lp is None:
            loss[t], dZ[t] = np.nan, np.nan
            continue
        q = np.exp(lq)
        loss[t] = temperature ** 2 * sum(
            qj * (lqj - lp[i]) for (i, _), qj, lqj in zip(kept, q, lq) if qj > 0)
        g = np.exp(lp)
        for (i, _), qj in zip(kept, q):
            g[i] -= qj
        dZ[t] = w * temperature * g
    return {"loss": loss, "dZ": dZ}


def exact_attention(Q, K, V, cu, n_heads, n_kv_heads, scale=None, E=None) -> dict:
    """Forward ("O", "lse") and, with E, the gradients of sum_t <o_t, e_t>.
    Rows that no sequence covers stay NaN in every output."""
    Q, K, V = (np.asarray(x, dtype=np.float64) for x in (Q, K, V))
    T = Q.shape[0]
    dh = Q.shape[1] // n_heads
    group = n_heads // n_kv_heads
    scale = dh ** -0.5 if scale is None else scale
    out = {"O": np.full(Q.shape, np.nan), "lse": np.full((T, n_heads), np.nan)}
    if E is not None:
        E = np.asarray(E, dtype=np.float64)
        out.update(dQ=np.full(Q.shape, np.nan), dK=np.full(K.shape, np.nan),
                   dV=np.full(K.shape, np.nan))
    for a, b in zip(cu[:-1], cu[1:]):
        n = b - a
        if n == 0:
            continue
        low = np.tril(np.ones((n, n), dtype=bool))
        if E is not None:
            out["dK"][a:b], out["dV"][a:b] = 0.0, 0.0
        for h in range(n_heads):
            c = slice(h * dh, (h + 1) * dh)
            g = slice(h // group * dh, (h // group + 1) * dh)
            q, k, v = Q[a:b, c], K[a:b, g], V[a:b, g]
            s = np.where(low, scale * (q @ k.T), -np.inf)
            m = s.max(1, keepdims=True)
            lse = m + np.log(np.exp(s - m).sum(1, keepdims=True))
            p = np.exp(s - lse)
            o = p @ v
            out["O"][a:b, c], out["lse"][a:b, h] = o, lse[:, 0]
            if E is None:
                continue
            e = E[a:b, c]
            ds = p * (e @ v.T - (o * e).sum(1, keepdims=True))
            out["dQ"][a:b, c] = scale * (ds @ k)
            out["dK"][a:b, g] += scale * (ds.T @ q)
            out["dV"][a:b, g] += p.T @ e
    return out
