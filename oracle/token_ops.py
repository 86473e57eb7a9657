"""Float64 oracle for the token log-probabilities, their gradient and the
distillation from a teacher's top logits (test infrastructure only).

Each function states its definition row by row: ``log p = x / T -
logsumexp(x / T)``; ``entropy = -sum p log p`` (0 log 0 = 0); the alternatives
ordered by (value descending, index ascending); the distillation loss
``T**2 sum_k q_k (log q_k - log p[id_k])``.
"""
from __future__ import annotations

import numpy as np


def _log_softmax(z: np.ndarray) -> np.ndarray:
    m = z.max()
    return z - (m + np.log(np.exp(z - m).sum()))


def token_logprobs(logits, index, top_k: int = 0, temperature: float = 1.0, ignore_index: int = -100):
    """(logprob, entropy, lse, top_logprob, top_index) of [B, V] logits."""
    x = np.asarray(logits, dtype=np.float64)
    B, V = x.shape
    lp, ent, lse = np.zeros(B), np.zeros(B), np.zeros(B)
    top, ids = np.full((B, top_k), -np.inf), np.full((B, top_k), -1, dtype=np.int64)
    for r in range(B):
        t = int(index[r])
        if t == ignore_index:
            continue
        if not 0 <= t < V:
            raise ValueError("index outside [0, V)")
        if np.isnan(x[r]).any() or np.isposinf(x[r]).any() or np.isneginf(x[r]).all():
            lp[r] = ent[r] = lse[r] = np.nan
            top[r] = np.nan
            continue
        z = x[r] / temperature
        m = z.max()
        lse[r] = m + np.log(np.exp(z - m).sum())
        logp = z - lse[r]
        p = np.exp(logp)
        lp[r] = logp[t]
        ent[r] = -(p[p > 0] * logp[p > 0]).sum()
        order = np.lexsort((np.arange(V), -x[r]))[:top_k]
        top[r], ids[r] = logp[order], order
    return lp, ent, lse, top, ids


def token_logprobs_vjp(logits, index, g_logprob, g_entropy, temperature: float = 1.0, ignore_index: int = -100):
    """Gradient of ``sum_r g_logprob[r] logprob[r] + g_entropy[r] entropy[r]``."""
    x = np.asarray(logits, dtype=np.float64)
    out = np.zeros_like(x)
    for r in range(x.shape[0]):
        t = int(index[r])
        if t == ignore_index:
            continue
        logp = _log_softmax(x[r] / temperature)
        p = np.exp(logp)
        some = p > 0
        inner = np.zeros_like(p)
        inner[some] = p[some] * logp[some]
        entropy = -inner.sum()
        g = -p * g_logprob[r] - g_entropy[r] * (inner + p * entropy)
        g[t] += g_logprob[r]
        out[r] = g / temperature
    return out


def topk_distill(logits, teacher_index, teacher_logits, temperature: float = 1.0, renormalize: bool = True,
                 reduction: str = "mean"):
    """Dict with ``loss``, ``row_loss``, ``grad`` and ``n_valid`` (rows with an entry)."""
    x = np.asarray(logits, dtype=np.float64)
    B, V = x.shape
    T = float(temperature)
    row, grad, valid = np.zeros(B), np.zeros_like(x), np.zeros(B, dtype=bool)
    for r in range(B):
        entries = [(int(i), float(v)) for i, v in zip(teacher_index[r], teacher_logits[r]) if i != -1 and v != -np.inf]
        if not entries:
            continue
        valid[r] = True
        ids = np.array([i for i, _ in entries])
        if (ids < 0).any() or (ids >= V).any():
            raise ValueError("id outside [0, V)")
        v = np.array([w for _, w in entries], dtype=np.float64)
        log_q = _log_softmax(v / T) if renormalize else v
        q = np.exp(log_q)
        logp = _log_softmax(x[r] / T)
        some = q > 0
        row[r] = T * T * (q[some] * (log_q[some] - logp[ids[some]])).sum()
        grad[r] = T * q.sum() * np.exp(logp)
        np.subtract.at(grad[r], ids, T * q)
    n = int(valid.sum())
    scale = 1.0 / max(n, 1) if reduction == "mean" else 1.0
    return {"loss": scale * row.sum(), "row_loss": row, "grad": scale * grad, "n_valid": n}
