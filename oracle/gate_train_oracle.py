"""fp64 restatement of the calls that train the gate: balance loss, router
logit gradient, combine and router backward, clipping by the global norm.

Plain NumPy from the definitions in ``include/moe.h``; shares no code with the
library."""

from __future__ import annotations

import math

import numpy as np


def _rows(T, token_mask, seq_offsets, logits):
    """Row indices that count, one array per sequence."""
    off = [0, T] if seq_offsets is None else [int(v) for v in seq_offsets]
    ok = ~np.all(np.isneginf(logits), axis=1)
    if token_mask is not None:
        ok &= np.asarray(token_mask) != 0
    return [np.array([t for t in range(a, b) if ok[t]], dtype=np.int64)
            for a, b in zip(off[:-1], off[1:])]


def softmax_lse(row):
    m = np.max(row)
    e = np.exp(row - m)
    return e / e.sum(), m + math.log(e.sum())


def balance_loss(logits, idx, balance_coef, z_coef, token_mask=None, seq_offsets=None,
                 counts=None):
    """(loss [3], counts [S, E], tokens [S + 2], prob_mean [S, E]).  ``counts``
    replaces the batch's own (a constant of the gradient)."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    k = idx.shape[1]
    rows = _rows(T, token_mask, seq_offsets, logits)
    S = len(rows)
    c = np.zeros((S, E), dtype=np.int64)
    mean = np.zeros((S, E))
    n = np.array([len(r) for r in rows], dtype=np.int64)
    bal, z = 0.0, 0.0
    for i, r in enumerate(rows):
        if not len(r):
            continue
        for t in r:
            p, lse = softmax_lse(logits[t])
            mean[i] += p
            z += lse * lse
            for e in idx[t]:
                c[i, e] += 1
        mean[i] /= len(r)
        use = c[i] if counts is None else counts[i]
        bal += E / (k * len(r)) * float(np.dot(use, mean[i]))
    live, total = int((n > 0).sum()), int(n.sum())
    lb = balance_coef * bal / live if live and balance_coef else 0.0
    lz = z_coef * z / total if total and z_coef else 0.0
    return np.array([lb + lz, lb, lz]), c, np.concatenate([n, [total, live]]), mean


def gate_bwd(logits, idx, w, dw, counts, balance_coef, z_coef, dloss=1.0, token_mask=None,
             seq_offsets=None):
    """dlogits [T, E]; dw or counts None leaves its part out."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    out = np.zeros((T, E))
    if counts is not None:
        k = idx.shape[1]
        rows = _rows(T, token_mask, seq_offsets, logits)
        live = sum(len(r) > 0 for r in rows)
        total = sum(len(r) for r in rows)
        for i, r in enumerate(rows):
            for t in r:
                p, lse = softmax_lse(logits[t])
                f = counts[i].astype(np.float64) * balance_coef * E / (live * k * len(r) ** 2)
                out[t] = dloss * p * (f - np.dot(f, p))
                if z_coef:
                    out[t] += dloss * p * 2.0 * z_coef * lse / total
    if dw is not None:
        for t in range(T):
            dot = float(np.dot(w[t], dw[t]))
            for j, e in enumerate(idx[t]):
                out[t, e] += w[t, j] * (dw[t, j] - dot)
    return out


def combine_bwd(dy, z, row_of, w):
    """(dw [T, k], dz [T*k, d])."""
    T, k = row_of.shape
    dw = np.zeros((T, k))
    dz = np.zeros((T * k, dy.shape[1]))
    for t in range(T):
        for j in range(k):
            r = int(row_of[t, j])
            dw[t, j] = np.dot(dy[t], z[r])
            dz[r] = w[t, j] * dy[t]
    return dw, dz


def router_bwd(x, w_g, dlogits):
    """(dw_g [d, E], dbias [E], dx [T, d])."""
    return x.T @ dlogits, dlogits.sum(axis=0), dlogits @ w_g.T


def clip_grads(grads, max_norm):
    """(norm, scaled gradients)."""
    norm = math.sqrt(math.fsum(float(np.dot(g, g)) for g in grads))
    c = min(1.0, max_norm / (norm + 1e-6)) if math.isfinite(norm) else 1.0
    return norm, [c * g for g in grads]
