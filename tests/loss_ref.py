"""Plain references of the losses over a vocabulary in 64 bits, with error
bounds.

Each returns (value, bound) per output: the value unrounded and how far a
result may be from it that computes in 32 bits and rounds where the header
says.  With e32 = 2^-23 for every operation in 32 bits (rounded, or truncated
to 24 bits):

    z        D e32 sum |x w|                                      (ez)
    2^(c z - r)  its argument is off by ez / tau and 2 e32 (|z| / tau + |r|), and
             the function by 2 units of 2^-23: a term is off by
             et = ez / tau + 2 e32 (|z| / tau + |r|) + 2 e32, relatively
    lse      max et (r: the row's maximum) + e32 (the additions that a term goes
             through: 64 in its chunk, one per chunk of 64 words, one per part) + 4 e32 |lse|
    q        its argument 4 e32 (1 + |x|), exp and the sum of k terms: eq = (4 |x| + 8 + k) e32, relatively
    g        |a| (p et + q eq) + 4 e32 |a| (p + q), then rounded to the type
             (binary16: held times a power of two that brings max |a| to at least 2^14);
             up to 32 rows held in two numbers of the type, the second the rounded
             rest of at most u |g|.  Up to 128 rows, at a wanted word of p > 1/2, z is summed
             with ceil(D / 2048) terms in each number of 32 bits: ez = that many e32 sum |x w|
    dX, dW   those through |W| and |X|, n e32 sum |g| |w| for the accumulation, rounded to the type
"""
from __future__ import annotations

import math

import numpy as np
import torch

from ragged_ref import TINY, UNIT, check  # noqa: F401

E32 = 2.0 ** -23


def _f64(t):
    return t.detach().double().cpu().numpy()


def words_of(targets=None, ids=None, logits=None, tau=1.0):
    """(valid rows, ids, q, x = log q + const, log q, eq) as (T, k) arrays; no word: id -1, q 0."""
    if targets is not None:
        i = targets.cpu().numpy().astype(np.int64)[:, None]
        has = i >= 0
        return has[:, 0], np.where(has, i, -1), has * 1.0, np.zeros(i.shape), np.zeros(i.shape)
    i, l = ids.cpu().numpy().astype(np.int64), _f64(logits)
    has = (i >= 0) & (l > -np.inf)
    valid = has.any(axis=1)
    l = np.where(has, l, -np.inf)
    top = np.where(valid, l.max(axis=1), 0.0)[:, None]
    x = np.where(has, (l - top) / tau, -np.inf)
    q = np.exp(x)
    total = np.where(valid, q.sum(axis=1), 1.0)[:, None]
    q = q / total
    with np.errstate(divide="ignore"):
        log_q = np.where(q > 0, np.log(np.where(q > 0, q, 1.0)), 0.0)
    eq = np.where(q > 0, (4 * np.abs(np.where(has, x, 0.0)) + 8 + i.shape[1]) * E32, 0.0)
    return valid, np.where(has, i, -1), q, log_q, eq


def _logits(x, w, layout, tau):
    X, W = _f64(x), _f64(w)
    if layout == "nk":
        W = W.T
    return X, W, X @ W / tau, X.shape[1] * E32 * (np.abs(X) @ np.abs(W)) / tau


def losses(x, w, words, layout, tau=1.0, cross=True):
    """((loss, bound), (lse, bound))"""
    valid, ids, q, log_q, eq = words
    X, W, z, ez = _logits(x, w, layout, tau)
    V, k = z.shape[1], ids.shape[1]
    top = z.max(axis=1)
    lse = top + np.log(np.exp(z - top[:, None]).sum(axis=1))
    et = ez + 2 * E32 * (np.abs(z) + np.abs(top)[:, None]) + 2 * E32
    e_lse = et.max(axis=1) + (V / 64 + 64 + V / 64) * E32 + 4 * E32 * np.abs(lse)
    at = np.maximum(ids, 0)
    zi, ezi = np.take_along_axis(z, at, axis=1), np.take_along_axis(ez, at, axis=1)
    e = (q * (eq * np.abs(zi) + ezi) + (k + V / 32 + 8) * E32 * q * np.abs(zi)).sum(axis=1) + e_lse + 8 * E32 * np.abs(lse)
    loss = (q * (log_q - zi)).sum(axis=1) + lse
    e += (q * (eq * (1 + np.abs(log_q)) + (k + 8) * E32 * np.abs(log_q))).sum(axis=1)
    if not cross:
        loss, e = tau * tau * loss, tau * tau * e
    e += 4 * E32 * np.abs(loss)
    zero = np.zeros_like(lse)
    return (np.where(valid, loss, zero), np.where(valid, e, zero)), (np.where(valid, lse, zero), np.where(valid, e_lse, zero))


def gradients(x, w, words, lse, dloss, layout, tau=1.0, cross=True):
    """((dx, bound), (dw, bound))"""
    valid, ids, q, _, eq = words
    dtype = x.dtype
    x = torch.where(torch.from_numpy(valid).to(x.device)[:, None], x, torch.zeros_like(x))
    X, W, z, ez = _logits(x, w, layout, tau)
    T, V = z.shape
    r = np.where(valid, np.nan_to_num(_f64(lse)), 0.0)[:, None]
    a = np.where(valid, np.broadcast_to(np.nan_to_num(_f64(dloss)), (T,)), 0.0)[:, None] * (1.0 if cross else tau)
    p = np.exp(z - r)
    e = p * (ez + 2 * E32 * (np.abs(z) + np.abs(r)) + 2 * E32)
    rows = np.arange(T)[:, None]
    sure = (ids >= 0) & (p[rows, np.maximum(ids, 0)] > 0.501) & (T <= 128)  # (of half: either)
    rows, at = np.broadcast_to(rows, ids.shape)[sure], ids[sure]
    ez[rows, at] *= math.ceil(X.shape[1] / 2048) / X.shape[1]
    e[rows, at] = p[rows, at] * (ez[rows, at] + 2 * E32)
    g, size = p.copy(), p.copy()
    for j in range(ids.shape[1]):
        rows = np.flatnonzero(ids[:, j] >= 0)
        np.subtract.at(g, (rows, ids[rows, j]), q[rows, j])
        np.add.at(size, (rows, ids[rows, j]), q[rows, j])
        np.add.at(e, (rows, ids[rows, j]), q[rows, j] * eq[rows, j])
    g, e = a * g, np.abs(a) * (e + 4 * E32 * size)
    tiny = TINY[dtype]
    if dtype == torch.float16:
        tiny = 2.0 ** -25 * 2.0 ** -14 * np.abs(a).max(initial=0.0)
    e = e + UNIT[dtype] ** (2 if T <= 32 else 1) * (np.abs(g) + e) + np.where(valid, tiny, 0.0)[:, None]
    g, e = g * valid[:, None], e * valid[:, None]
    n = np.abs(g) + e
    dx, ex = g @ W.T, e @ np.abs(W).T + (V + 32) * E32 * (n @ np.abs(W).T)
    dw, ew = X.T @ g, np.abs(X).T @ e + T * E32 * (np.abs(X).T @ n)
    if layout == "nk":
        dw, ew = dw.T, ew.T
    done = lambda v, b: (v, b + UNIT[dtype] * (np.abs(v) + b) + TINY[dtype])  # noqa: E731
    dx, ex = done(dx, ex)
    ex = np.where(valid[:, None], ex, 0.0)  # rows that are not in use: exactly zero
    return (dx, ex), done(dw, ew)


def make_words(T, V, k, seed, ignored=0.0, few=0.2):
    """Words and logits of a teacher on the CPU: some twice in a row, some missing, some rows without any."""
    rs = np.random.RandomState(seed)
    ids = rs.randint(0, V, (T, k)).astype(np.int32)
    if k > 1:
        ids[::3, k - 1] = ids[::3, 0]
    ids[rs.random_sample((T, k)) < few * (k > 1)] = -1
    ids[rs.random_sample(T) < ignored] = -7
    logits = (3 * rs.standard_normal((T, k)) + 5).astype(np.float32)
    return torch.from_numpy(ids), torch.from_numpy(logits)


def make_targets(T, V, seed, ignored=0.0):
    rs = np.random.RandomState(seed)
    y = rs.randint(0, V, T).astype(np.int32)
    y[rs.random_sample(T) < ignored] = -100
    return torch.from_numpy(y)


__all__ = ["check", "gradients", "losses", "make_targets", "make_words", "math", "words_of"]
