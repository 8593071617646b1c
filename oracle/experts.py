"""Plain fp64 oracles of gradient clipping and of the expert-layer calls
(numpy; test infrastructure only). Written from the definitions, loop by
loop; no blocking, no shared code with the kernels."""
from __future__ import annotations

import numpy as np

from . import sign_matrix


def clip(grads, max_norm):
    """(norm, coef, scaled gradients) of a list of arrays."""
    norm = float(np.sqrt(sum(float(np.sum(np.square(np.asarray(g, np.float64)))) for g in grads)))
    coef = max_norm / norm if np.isfinite(norm) and norm > max_norm else 1.0
    return norm, coef, [coef * np.asarray(g, np.float64) for g in grads]


def expert_sort(ids, n_experts):
    """(offsets, order, slots) of T x K ids: pairs appended to their expert's list one by one."""
    lists = [[] for _ in range(n_experts)]
    flat = np.asarray(ids).reshape(-1)
    for p, e in enumerate(flat.tolist()):
        if 0 <= e < n_experts:
            lists[e].append(p)
    offsets = np.concatenate([[0], np.cumsum([len(q) for q in lists])]).astype(np.int32)
    order = np.full(flat.size, -1, np.int32)
    kept = [p for q in lists for p in q]
    order[:len(kept)] = kept
    slots = np.full(flat.size, -1, np.int32)
    slots[kept] = np.arange(len(kept))
    return offsets, order, slots.reshape(np.asarray(ids).shape)


def gather(X, slots, w, Xs):
    """Xs with the rows that slots name replaced."""
    out = np.array(Xs, np.float64)
    for t, j in zip(*np.nonzero(np.asarray(slots) >= 0)):
        out[slots[t, j]] = (1.0 if w is None else w[t, j]) * X[t]
    return out


def combine(Ys, slots, w):
    """(Y, sum of |w Ys|) per token."""
    T, K = slots.shape
    Y, mag = np.zeros((T, Ys.shape[1])), np.zeros((T, Ys.shape[1]))
    for j in range(K):
        for t in np.nonzero(slots[:, j] >= 0)[0]:
            row = (1.0 if w is None else w[t, j]) * Ys[slots[t, j]]
            Y[t] += row
            mag[t] += np.abs(row)
    return Y, mag


def combine_backward(dY, Ys, slots, w, dYs):
    """(dYs with the named rows replaced, dw, sum of |dY Ys| per weight)."""
    out = np.array(dYs, np.float64)
    dw, mag = np.zeros(slots.shape), np.zeros(slots.shape)
    for t, j in zip(*np.nonzero(slots >= 0)):
        s = slots[t, j]
        out[s] = w[t, j] * dY[t]
        dw[t, j] = np.dot(dY[t], Ys[s])
        mag[t, j] = np.dot(np.abs(dY[t]), np.abs(Ys[s]))
    return out, dw, mag


def sketch_experts(X, dY, offsets, d, k, r, seed, step, first_id, id_stride, order=None, topk=1):
    """(S, P magnitudes for error bounds): S_e = dY_e^T (X_e A_e^T); the
    second and third results are sum_t |dY_ti| |P_tl| and
    sum_t |dY_ti| c sum_j |X_tj| per entry of S."""
    E = len(offsets) - 1
    S = np.zeros((E, d, r))
    mag_p, mag_x = np.zeros((E, d, r)), np.zeros((E, d, r))
    for e in range(E):
        A = sign_matrix(seed, step, first_id + e * id_stride, r, k)
        rows = np.arange(offsets[e], offsets[e + 1])
        if rows.size == 0:
            continue
        Xe = X[rows] if order is None else X[np.asarray(order)[rows] // topk]
        P = Xe @ A.T
        dYe = dY[rows]
        S[e] = dYe.T @ P
        mag_p[e] = np.abs(dYe).T @ np.abs(P)
        mag_x[e] = (np.abs(dYe).T @ np.abs(Xe).sum(1))[:, None] / np.sqrt(r)
    return S, mag_p, mag_x
