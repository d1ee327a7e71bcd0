"""Plain float64 numpy forms of the item-table operators: row lookup and its
gradient, the distillation loss and the paired preference loss (definitions in
include/cutbce.h).  Test infrastructure, written dense and without the library's
split into a dense and a sparse part."""
from __future__ import annotations

from types import SimpleNamespace
from typing import Optional

import numpy as np


def embed(E, ids, scale=1.0):
    E = np.asarray(E, np.float64)
    out = np.zeros((len(ids), E.shape[1]))
    for n, v in enumerate(ids):
        if v >= 0:
            out[n] = scale * E[v]
    return out


def embed_grad(dX, ids, V, scale=1.0):
    dX = np.asarray(dX, np.float64)
    out = np.zeros((V, dX.shape[1]))
    np.add.at(out, np.asarray(ids)[np.asarray(ids) >= 0], scale * dX[np.asarray(ids) >= 0])
    return out


def _log_softmax(x):
    m = x.max(axis=-1, keepdims=True)
    return x - m - np.log(np.exp(x - m).sum(axis=-1, keepdims=True))


def teacher_weights(ids, logits, tau, V):
    """Dense q [T, V] and sum_k q_k ln q_k of every row (rows without a filled slot: zero)."""
    T, K = ids.shape
    q = np.zeros((T, V))
    ent = np.zeros(T)
    for t in range(T):
        k = [j for j in range(K) if ids[t, j] >= 0 and logits[t, j] > -np.inf]
        if not k:
            continue
        lq = _log_softmax(np.asarray(logits[t, k], np.float64) / tau)
        for j, l in zip(k, lq):
            q[t, ids[t, j]] += np.exp(l)
            ent[t] += np.exp(l) * l
    return q, ent


def _head(H, E, w, q, tau, g):
    """Shared by both losses: lse, p and the gradients of sum_t w_t (tau-scaled) with dz = w (p - q)."""
    z = H @ E.T / tau
    lse = np.log(np.exp(z - z.max(1, keepdims=True)).sum(1)) + z.max(1)
    p = np.exp(z - lse[:, None])
    G = g * w[:, None] * (p - q)
    return z, lse, p, G


def distill(H, E, ids, logits, mask=None, weights=None, tau=1.0, reduction="mean", grad_loss=1.0):
    H, E = np.array(H, np.float64), np.asarray(E, np.float64)
    T, V = H.shape[0], E.shape[0]
    w = np.ones(T) if weights is None else np.asarray(weights, np.float64).copy()
    if mask is not None:
        w[np.asarray(mask) == 0] = 0.0
    ids = np.where((w != 0)[:, None], ids, -1)
    logits = np.where(ids >= 0, logits, -np.inf)
    w[~((ids >= 0) & (logits > -np.inf)).any(1)] = 0.0
    valid = w != 0
    H[~valid] = 0.0
    q, ent = teacher_weights(np.where(valid[:, None], ids, -1), logits, tau, V)
    n = int(valid.sum())
    s = (1.0 / n if n else 0.0) if reduction == "mean" else 1.0
    z, lse, p, G = _head(H, E, w, q, tau, grad_loss * s * tau)
    row = tau * tau * (ent - (q * z).sum(1) + lse)
    return SimpleNamespace(loss=s * float((w * np.where(valid, row, 0.0)).sum()), lse=np.where(valid, lse, 0.0),
                           dH=np.where(valid[:, None], G @ E, 0.0), dE=G.T @ H, p=p, q=q, w=w, s=s, valid=valid, H=H)


def preference(H, E, ids, offsets, ref=None, mask=None, beta=0.1, reduction="mean", grad_loss=1.0):
    H, E = np.array(H, np.float64), np.asarray(E, np.float64)
    T, V = H.shape[0], E.shape[0]
    n = len(offsets) - 1
    seq = np.full(T, -1)
    for i in range(n):
        seq[offsets[i]:offsets[i + 1]] = i
    valid = (np.asarray(ids) >= 0) & (seq >= 0)
    if mask is not None:
        valid &= np.asarray(mask) != 0
    H[~valid] = 0.0
    y = np.zeros((T, V))
    y[np.nonzero(valid)[0], np.asarray(ids)[valid]] = 1.0
    z = H @ E.T
    lse = np.log(np.exp(z - z.max(1, keepdims=True)).sum(1)) + z.max(1)
    lp = np.where(valid, (y * z).sum(1) - lse, 0.0)
    L = np.array([lp[seq == i].sum() for i in range(n)])
    R = np.zeros(n) if ref is None else np.asarray(ref, np.float64)
    x = beta * ((L[0::2] - L[1::2]) - (R[0::2] - R[1::2]))
    s = 1.0 / len(x) if reduction == "mean" else 1.0
    loss = s * float(np.logaddexp(0.0, -x).sum())
    sig = np.exp(-np.logaddexp(0.0, x))                       # sigmoid(-x)
    w = np.zeros(T)
    for i in range(n):
        w[(seq == i) & valid] = sig[i // 2] * (1.0 if i % 2 == 0 else -1.0)
    z, lse, p, G = _head(H, E, w, y, 1.0, grad_loss * s * beta)
    return SimpleNamespace(loss=loss, logp=L, lse=np.where(valid, lse, 0.0), dH=np.where(valid[:, None], G @ E, 0.0),
                           dE=G.T @ H, p=p, q=y, w=w, s=s, valid=valid, H=H, x=x)


def offsets_of(lengths, first: int = 0, dtype=np.int32, total: Optional[int] = None):
    return (first + np.concatenate([[0], np.cumsum(lengths)])).astype(dtype)
