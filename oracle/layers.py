"""References of the operators around the scan, from their definitions, in
float64 on the CPU: one token, one query or one element at a time where that
is affordable. They share nothing with the GPU path.

Next to each result stands what its tolerance is derived from: the same sum
taken over magnitudes ("mag"), which bounds how far roundings of its terms can
move it.
"""
from __future__ import annotations

import numpy as np
import torch

# half a unit in the last place, relative to the value
STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def f64(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def _silu(v):
    with np.errstate(over="ignore"):
        return v / (1.0 + np.exp(-v))


def conv(x, weight, bias, cu, cache, idx, has, silu=True):
    """y [T,C], cache rows per slot as left, mag [T,C] = |bias| + sum |w x|."""
    x, w, cache = f64(x), f64(weight), f64(cache).copy()
    T, C = x.shape
    W = w.shape[1]
    b = np.zeros(C) if bias is None else f64(bias)
    y, mag, snap = np.zeros((T, C)), np.zeros((T, C)), cache.copy()
    for s in range(len(cu) - 1):
        a, e, slot = int(cu[s]), int(cu[s + 1]), int(idx[s])
        ok = 0 <= slot < len(cache)
        old = snap[slot] if ok and has is not None and int(has[s]) else np.zeros((W - 1, C))
        line = np.concatenate([old, x[a:e]])
        for t in range(e - a):
            y[a + t] = b + sum(w[:, k] * line[t + k] for k in range(W))
            mag[a + t] = np.abs(b) + sum(np.abs(w[:, k] * line[t + k]) for k in range(W))
        if ok:
            cache[slot] = line[len(line) - (W - 1):]
    return (_silu(y) if silu else y), cache, mag


def softplus(v):
    return np.logaddexp(0.0, v)


def scan(x, dt, A, B, C, D, z, cu, cache, idx, has, bias=None, lo=None, hi=None):
    """y [T,C], states after every token [T,C,N], cache as left, and the magnitudes of y and of
    the states. bias None and lo None: dt as given."""
    x, dt, A, B, C, cache = f64(x), f64(dt), f64(A), f64(B), f64(C), f64(cache).copy()
    T, ch = x.shape
    N, G = A.shape[1], B.shape[1]
    grp = np.arange(ch) // (ch // G)
    if lo is not None:
        dt = np.clip(softplus(dt + (0.0 if bias is None else f64(bias))), lo, hi)
    Dv = np.zeros(ch) if D is None else f64(D)
    gate = np.ones((T, ch)) if z is None else _silu(f64(z))
    y, ymag = np.zeros((T, ch)), np.zeros((T, ch))
    st, smag = np.zeros((T, ch, N)), np.zeros((T, ch, N))
    snap = cache.copy()
    cmag = np.abs(cache)
    for s in range(len(cu) - 1):
        a, e, slot = int(cu[s]), int(cu[s + 1]), int(idx[s])
        ok = 0 <= slot < len(cache)
        h = snap[slot].copy() if ok and has is not None and int(has[s]) else np.zeros((ch, N))
        m = np.abs(h)
        for t in range(a, e):
            da = np.exp(dt[t][:, None] * A)
            u = (dt[t] * x[t])[:, None] * B[t][grp]
            h, m = da * h + u, da * m + np.abs(u)
            st[t], smag[t] = h, m
            y[t] = ((h * C[t][grp]).sum(1) + Dv * x[t]) * gate[t]
            ymag[t] = ((m * np.abs(C[t][grp])).sum(1) + np.abs(Dv * x[t])) * np.abs(gate[t])
        if ok:
            cache[slot], cmag[slot] = h, m
    return y, st, cache, ymag, smag, cmag


def attention(q, k, v, cuq, cuk, causal=True, scale=None):
    """out [Tq,H,D], lse [Tq,H], mag = softmax @ |v|, and top = max over the keys seen of
    scale * sum |q_d k_d| (what rounding the products and sums of a score goes by)."""
    q, k, v = f64(q), f64(k), f64(v)
    Tq, H, D = q.shape
    group = H // k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    out, mag = np.zeros((Tq, H, D)), np.zeros((Tq, H, D))
    lse, top = np.full((Tq, H), -np.inf), np.zeros((Tq, H))
    with np.errstate(invalid="ignore", over="ignore"):
        for s in range(len(cuq) - 1):
            a, e, ka, ke = int(cuq[s]), int(cuq[s + 1]), int(cuk[s]), int(cuk[s + 1])
            for i in range(e - a):
                n = ke - ka if not causal else min(ke - ka, i + (ke - ka) - (e - a) + 1)
                if n <= 0:
                    continue
                for h in range(H):
                    kk, vv = k[ka:ka + n, h // group], v[ka:ka + n, h // group]
                    sc = scale * (kk @ q[a + i, h])
                    p = np.exp(sc - sc.max())
                    tot = p.sum()
                    out[a + i, h] = (p @ vv) / tot
                    mag[a + i, h] = (p @ np.abs(vv)) / tot
                    lse[a + i, h] = sc.max() + np.log(tot)
                    top[a + i, h] = scale * (np.abs(kk) @ np.abs(q[a + i, h])).max()
    return out, lse, mag, top


def attention_tolerance(out, mag, top, D, nk, dtype):
    """How far a result may be off: a score is a float32 sum of D products (D + 2 roundings of up
    to 2^-24 of their magnitudes, and as many again for the exponential's argument), which moves a
    weight and the sum of the weights by that much; nk + 8 roundings in the sums; in bf16 the
    weight is rounded too, and the result."""
    delta = (2 * D + 8) * 2.0 ** -24 * top + 2.0 ** -20
    rel = 2 * delta + (nk + 8) * 2.0 ** -24
    if dtype == torch.bfloat16:
        rel = rel + 2.0 ** -8
    return rel[..., None] * mag + STEP[dtype] * np.abs(out) + 1e-30


# every finite value of the 8-bit type, by its code: sign, 4 exponent bits (bias 7), 3 mantissa
# bits; exponent 0 is subnormal, the code of all ones is NaN
CODES = np.array([(-1.0 if c & 128 else 1.0) * (
    (c & 7) / 8 * 2.0 ** -6 if (c >> 3) & 15 == 0 else (1 + (c & 7) / 8) * 2.0 ** (((c >> 3) & 15) - 7))
    if c & 127 != 127 else np.nan for c in range(256)])


def encode_row(row):
    """Codes' values and scale byte of one row: the least power of two 2^s, s >= -126, with
    |x| <= 448 2^s for every finite x (1 for a row of zeros); each x / 2^s to the nearest value of
    the type, of two equally near ones the one with the even code; non-finite ones to NaN."""
    row = np.asarray(row, dtype=np.float64)
    fin = np.isfinite(row)
    top = np.abs(row[fin]).max() if fin.any() else 0.0
    s = -126
    while top > 448.0 * 2.0 ** s:
        s += 1
    pos = CODES[:127]
    got = np.full(row.shape, np.nan)
    for i, v in enumerate(row):
        if not fin[i]:
            continue
        d = np.abs(pos - abs(v) / 2.0 ** s)
        c = int(np.argmin(d))
        if c + 1 < 127 and d[c + 1] == d[c] and c % 2 == 1:
            c += 1
        got[i] = np.copysign(pos[c], v)
    return got, s + 127


def decode_attention(q, rows_k, rows_v, lens, scale=None):
    """q [R,T,H,D]; rows_k, rows_v: per request its cached rows [L,Hkv,D] (values)."""
    R, T, H, D = q.shape
    res = []
    for r in range(R):
        L = len(rows_k[r])
        cuq, cuk = [0, T], [0, L]
        res.append(attention(q[r], torch.as_tensor(rows_k[r]), torch.as_tensor(rows_v[r]), cuq, cuk,
                             True, scale))
    return tuple(np.stack([x[i] for x in res]) for i in range(4))
