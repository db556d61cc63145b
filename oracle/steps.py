"""References of the operators between and behind the layers of a serving step, from their
definitions, in float64 (the verification: in fractions) on the CPU. They share nothing with the GPU
path. Next to each result stands what its tolerance is derived from.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np

from .layers import STEP, encode_row, f64

EPS = 2.0 ** -24        # half a float32 step, relative to the value


def rms_norm(x, weight=None, residual=None, gate=None, groups=1, eps=1e-5):
    """out [rows,hidden], v = x, x + residual or x silu(gate), and how far a float32 evaluation of
    out may be off, before it is rounded to its own type."""
    v = f64(x)
    rows, h = v.shape
    rel = np.zeros_like(v)
    if gate is not None:
        z = f64(gate)
        v = v * z / (1 + np.exp(-z))
        # exp's argument z log2(e) is rounded twice and its result once, then a sum, a quotient and
        # the product: relative to v
        rel = (2 * np.abs(z) + 8) * EPS
    if residual is not None:
        v = v + f64(residual)
        rel = np.full_like(v, EPS)
    per = h // groups
    g = v.reshape(rows, groups, per)
    out = (g / np.sqrt((g ** 2).mean(-1, keepdims=True) + eps)).reshape(rows, h)
    w = np.ones(h) if weight is None else f64(weight)
    # the sum of squares: one rounding a term of a thread's chain (of at most 32: longer ones go on
    # in 64 bits), rounded to float32 once, then 6 over the wave and at most 16 over the block; quotient,
    # eps, root, two products
    worst = rel.reshape(rows, groups, per).max(-1, keepdims=True).repeat(per, -1).reshape(rows, h)
    off = rel + worst + ((min(per, 32) + 1 + 6 + 16) / 2 + 8) * EPS
    return out * w, v, np.abs(out * w) * off + 1e-37


def encode_blocks(row):
    """8-bit rows of linear_w4: values and scale bytes of every 32 elements."""
    row = np.asarray(row, dtype=np.float64)
    got = [encode_row(b) for b in row.reshape(-1, 32)]
    return (np.concatenate([c * 2.0 ** (b - 127) for c, b in got]).reshape(row.shape),
            np.array([b for _, b in got]).reshape(row.shape[:-1] + (-1,)))


FOUR_BITS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def weights(codes, scale):
    """What 4-bit weights stand for: codes [N,K/2], scale [N,K/32] -> [N,K]."""
    c = codes.cpu().numpy().astype(np.int64)
    n, k = c.shape[0], 2 * c.shape[1]
    w = np.zeros((n, k))
    for half in (0, 1):
        v = (c >> (4 * half)) & 15
        w[:, half::2] = np.where(v >= 8, -1.0, 1.0) * FOUR_BITS[v & 7]
    b = scale.cpu().numpy().astype(np.float64)
    b = np.where(b == 255, np.nan, 2.0 ** (b - 127))
    return (w.reshape(n, -1, 32) * b[..., None]).reshape(n, k)


def encode_weights(row):
    """Values and scale byte of 32 weights: the least power of two 2^s, -126 <= s <= 125, with
    |w| <= 6 2^s for every finite w (125 where there is none); each to the nearest value, of two
    equally near ones the one at an even place."""
    row = np.asarray(row, dtype=np.float64)
    fin = np.isfinite(row)
    top = np.abs(row[fin]).max() if fin.any() else 0.0
    s = -126
    while top > 6.0 * 2.0 ** s and s < 125:
        s += 1
    got = np.zeros(row.shape)
    for i, v in enumerate(row):
        if np.isnan(v):
            continue
        m = 6.0 if np.isinf(v) else abs(v) / 2.0 ** s
        d = np.abs(FOUR_BITS - m)
        c = int(np.argmin(d))
        if c + 1 < 8 and d[c + 1] == d[c] and c % 2 == 1:
            c += 1
        got[i] = np.copysign(FOUR_BITS[c], v) * 2.0 ** s
    return got, s + 127


def rows8(x, x_scale):
    """What 8-bit rows stand for."""
    v = f64(x)
    b = 2.0 ** (x_scale.cpu().numpy().astype(np.float64) - 127)
    return (v.reshape(v.shape[0], -1, 32) * b[..., None]).reshape(v.shape)


def linear(x, w, bias=None):
    """x [T,K], w [N,K] values: y, and the same sum over magnitudes."""
    b = 0.0 if bias is None else f64(bias)
    return x @ w.T + b, np.abs(x) @ np.abs(w).T + np.abs(b)


def linear_tolerance(y, mag, k, dtype, cut=0.0):
    """Products are exact in float32; of their sum's K + 8 additions each is off by at most a step
    (2^-23, should the matrix unit cut off instead of rounding) of a partial sum, which is never
    larger than mag; then the result's own rounding. `cut`: cut_products, where the caller lets
    products be cut."""
    return (k + 8) * 2 * EPS * mag + cut + STEP[dtype] * (np.abs(y) + cut) + 1e-37


def cut_products(x, w):
    """The matrix instruction of 8-bit rows lines up the products of 32 values and cuts each off at
    2^-13 of the largest one's power of two: 32 such cuts a block, the largest bounded by the
    largest factors."""
    top = lambda v: np.abs(v).reshape(v.shape[0], -1, 32).max(-1)               # noqa: E731
    return 32 * 2.0 ** -13 * (top(x) @ top(w).T)


def probs(logits, temperature=None):
    """probs [R,T,V] and how far a float32 evaluation may be off."""
    x = f64(logits)
    out, tol = np.zeros_like(x), np.zeros_like(x)
    V = x.shape[-1]
    for r in range(x.shape[0]):
        t = 1.0 if temperature is None else float(temperature[r])
        for i in range(x.shape[1]):
            row = x[r, i]
            if not t > 0:
                m = np.nanmax(row) if not np.isnan(row).all() else -np.inf
                if m > -np.inf:
                    out[r, i, int(np.flatnonzero(row == m)[0])] = 1
                continue
            if np.isnan(row).any() or np.isposinf(row).any():
                out[r, i] = np.nan
                continue
            m = row.max()
            if m == -np.inf:
                continue
            with np.errstate(under="ignore"):
                d = np.where(np.isneginf(row), 0, (row - m) / t)
                e = np.where(np.isneginf(row), 0, np.exp(d))
                out[r, i] = e / e.sum()
            # x - m is rounded once, |d| 2^-24 in the exponent; the exponential, its correction, the
            # reciprocal and the product: 8 more; the sum goes by its terms and its own additions
            # (at least 256 threads share a row, a few dozen steps over the block and the parts, and the
            # terms' exponents are rounded: |d| 2^-24, over a row's probabilities at most ln V 2^-24)
            rel = (np.abs(d) + 8) * EPS
            tol[r, i] = out[r, i] * (rel + (out[r, i] * rel).sum() + (V / 64 + 64) * EPS) + 1e-37
    return out, tol


def verify(target, draft, drafts, num_drafts, uniform):
    """num_accepted [R], tokens [R,T], in fractions: every comparison is exact."""
    tp = target.cpu().double().numpy()
    R, T, V = tp.shape
    frac = lambda v: Fraction(float(v)) if v > 0 else Fraction(0)              # noqa: E731
    acc, tokens = [], []
    for r in range(R):
        n = T - 1 if num_drafts is None else min(max(int(num_drafts[r]), 0), T - 1)
        got, cut = [], None
        for i in range(n):
            d, u = int(drafts[r, i]), float(uniform[r, i])
            if 0 <= d < V:
                q = Fraction(1) if draft is None else frac(float(draft[r, i, d]))
                if Fraction(u) * q < frac(tp[r, i, d]):
                    got.append(d)
                    continue
            cut = i
            break
        acc.append(len(got))
        p = [frac(v) for v in tp[r, len(got)]]
        w = p
        if cut is not None:
            if draft is None:
                w = [Fraction(0) if v == int(drafts[r, cut]) else p[v] for v in range(V)]
            else:
                w = [max(a - frac(float(b)), Fraction(0)) for a, b in zip(p, draft[r, cut])]
            if not any(w):
                w = p
        want, c, tok = sum(w) * Fraction(float(uniform[r, T - 1])), Fraction(0), -1
        for v in range(V):
            c += w[v]
            if w[v] > 0 and c > want:
                tok = v
                break
        got.append(tok)
        tokens.append(got + [-1] * (T - len(got)))
    return np.array(acc, dtype=np.int32).reshape(R), np.array(tokens, dtype=np.int32).reshape(R, T)
