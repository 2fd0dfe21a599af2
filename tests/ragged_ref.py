"""Plain references of the ragged products in 64 bits, with error bounds.

Everything is computed group by group (row by row for the adapters) from the
definitions.  Each reference returns (value, bound): the value unrounded, and
how far a result may be from it that accumulates the exact products in 32 bits
in any order and rounds once to the element type:

    e     = n * 2^-23 * sum |terms|      n terms, one rounding (or truncation
                                         to 24 bits) per addition
    bound = e + u * (|value| + e) + d    u, d: unit roundoff and half the
                                         smallest subnormal of the type
"""
from __future__ import annotations

import numpy as np
import torch

UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def _f64(t):
    return t.detach().double().cpu().numpy()


def rounded(value, e, dtype):
    return e + UNIT[dtype] * (np.abs(value) + e) + TINY[dtype]


def bounds_of(offsets, T):
    o = [int(v) for v in offsets.cpu().tolist()]
    return list(zip(o[:-1], o[1:]))


def grouped(x, w, offsets, relu, layout):
    X, W = _f64(x), _f64(w)
    if layout == "nk":
        W = W.transpose(0, 2, 1)
    T, K, N = X.shape[0], X.shape[1], W.shape[2]
    y, e = np.zeros((T, N)), np.zeros((T, N))
    for g, (lo, hi) in enumerate(bounds_of(offsets, T)):
        y[lo:hi] = X[lo:hi] @ W[g]
        e[lo:hi] = K * 2.0 ** -23 * (np.abs(X[lo:hi]) @ np.abs(W[g]))
    if relu:
        y = np.maximum(y, 0.0)
    return y, rounded(y, e, x.dtype)


def grouped_dx(dy, w, offsets, act, layout):
    D, W = _f64(dy), _f64(w)
    if layout == "nk":
        W = W.transpose(0, 2, 1)
    T, N, K = D.shape[0], D.shape[1], W.shape[1]
    dx, e = np.zeros((T, K)), np.zeros((T, K))
    for g, (lo, hi) in enumerate(bounds_of(offsets, T)):
        dx[lo:hi] = D[lo:hi] @ W[g].T
        e[lo:hi] = N * 2.0 ** -23 * (np.abs(D[lo:hi]) @ np.abs(W[g]).T)
    if act is not None:
        keep = _f64(act) > 0
        dx, e = np.where(keep, dx, 0.0), np.where(keep, e, 0.0)
    return dx, rounded(dx, e, dy.dtype)


def grouped_dw(x, dy, offsets, layout):
    X, D = _f64(x), _f64(dy)
    dw, e = [], []
    for lo, hi in bounds_of(offsets, X.shape[0]):
        dw.append(X[lo:hi].T @ D[lo:hi])
        e.append((hi - lo) * 2.0 ** -23 * (np.abs(X[lo:hi]).T @ np.abs(D[lo:hi])))
    dw, e = np.stack(dw), np.stack(e)
    if layout == "nk":
        dw, e = dw.transpose(0, 2, 1), e.transpose(0, 2, 1)
    return dw, rounded(dw, e, x.dtype)


def adapters(x, w, a, b, ids, scale, relu, layout):
    """The low-rank products go through two numbers of the element type, hi and
    the rounded rest: what is left out is the rounding of a rest of at most
    u |low|.  That and their accumulation and scale go through |B|."""
    X, W, A, B = _f64(x), _f64(w), _f64(a), _f64(b)
    if layout == "nk":
        W = W.T
    K, rank, dtype = X.shape[1], A.shape[1], x.dtype
    s = np.ones(A.shape[0]) if scale is None else _f64(scale)
    y = X @ W
    terms = np.abs(X) @ np.abs(W)
    e = np.zeros_like(y)
    for t, i in enumerate(ids.cpu().tolist()):
        if i < 0:
            continue
        low = s[i] * (X[t] @ A[i].T)
        low_e = (K + 2) * 2.0 ** -23 * abs(s[i]) * (np.abs(X[t]) @ np.abs(A[i]).T)
        low_e = low_e + UNIT[dtype] ** 2 * (np.abs(low) + low_e) + TINY[dtype]
        y[t] += low @ B[i]
        terms[t] += (np.abs(low) + low_e) @ np.abs(B[i])
        e[t] += low_e @ np.abs(B[i])
    e += (K + 2 * rank) * 2.0 ** -23 * terms
    if relu:
        y = np.maximum(y, 0.0)
    return y, rounded(y, e, dtype)


def check(out, ref, what):
    value, bound = ref
    got = _f64(out)
    assert got.shape == value.shape, f"{what}: shape {got.shape}, not {value.shape}"
    assert np.isfinite(got).all(), f"{what}: non-finite outputs"
    off = np.abs(got - value)
    bad = np.argwhere(~(off <= bound))
    if len(bad):
        at = tuple(bad[0])
        raise AssertionError(f"{what}: {len(bad)} of {got.size} outside the bound; first at {at}: {got[at]!r}, "
                             f"reference {value[at]!r}, bound {bound[at]!r}")
