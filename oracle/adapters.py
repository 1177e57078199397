"""Adapters of many requests beside one shared projection (oracle side) --
TEST INFRASTRUCTURE ONLY.

Every token m of a batch has a slot a(m) in [0, S) or -1; slot a holds A_a
[r, K], B_a [N, r] and a scale c_a.  With D the dropout of the adapter input
(the mask of ``dropout_mask``, kept values times 1 / (1 - p), unrounded):

    T[m] = D(X[m]) A_a^T,   out[m] = Y[m] + c_a T[m] B_a^T

and the derivatives with U[m] = dY[m] B_a, the mask held fixed.  Written token
by token, in fp64.
"""
from __future__ import annotations

import numpy as np

from .dropout import dropout_scale
from .qlora import _f64

PLAN_TILE = 64


def adapter_plan(lengths, slots, M: int, S: int):
    """(token_slot [M], order [M], start [S + 2], tiles [n, 3]) of requests that
    cover ``lengths`` consecutive rows each."""
    token_slot = []
    for n, s in zip(lengths, slots):
        token_slot += [int(s) if 0 <= s < S else -1] * max(int(n), 0)
    token_slot = (token_slot + [-1] * M)[:M]
    classes = [[m for m in range(M) if token_slot[m] == a] for a in list(range(S)) + [-1]]
    order = [m for c in classes for m in c]
    start, tiles = [0], []
    for a, c in zip(list(range(S)) + [-1], classes):
        tiles += [(a, start[-1] + f, min(PLAN_TILE, len(c) - f)) for f in range(0, len(c), PLAN_TILE)]
        start.append(start[-1] + len(c))
    rows = M // PLAN_TILE + min(M, S + 1)
    tiles += [(-1, 0, 0)] * (rows - len(tiles))
    return tuple(np.asarray(v, np.int32) for v in (token_slot, order, start, tiles))


def _dropped(X, mask, p):
    X = _f64(X)
    if mask is None:
        return X
    return np.where(mask, X, 0.0) * np.float64(dropout_scale(p))


def adapters_forward(X, Y, A, B, scale, token_slot, mask=None, p: float = 0.0):
    """(out, T) in fp64; Y may be None (zeros)."""
    Xd, A, B = _dropped(X, mask, p), _f64(A), _f64(B)
    M, (S, N, r) = Xd.shape[0], B.shape
    out = np.zeros((M, N)) if Y is None else _f64(Y).copy()
    T = np.zeros((M, r))
    for m, a in enumerate(token_slot):
        if a >= 0:
            T[m] = A[a] @ Xd[m]
            out[m] += np.float64(scale[a]) * (B[a] @ T[m])
    return out, T


def adapters_backward(dY, X, A, B, scale, token_slot, dX0=None, mask=None, p: float = 0.0,
                      T=None):
    """(dX, dA, dB) in fp64; T as the forward gave it (None: computed)."""
    Xd, A, B, dY = _dropped(X, mask, p), _f64(A), _f64(B), _f64(dY)
    keep = 1.0 if mask is None else np.asarray(mask, np.float64) * np.float64(dropout_scale(p))
    dX, dA, dB = np.zeros(Xd.shape), np.zeros(A.shape), np.zeros(B.shape)
    for m, a in enumerate(token_slot):
        if a < 0:
            continue
        c, u = np.float64(scale[a]), dY[m] @ B[a]
        t = A[a] @ Xd[m] if T is None else np.asarray(T[m], np.float64)
        dX[m] = c * (u @ A[a])
        dA[a] += c * np.outer(u, Xd[m])
        dB[a] += c * np.outer(dY[m], t)
    dX = dX * keep
    return (dX if dX0 is None else dX + _f64(dX0)), dA, dB
