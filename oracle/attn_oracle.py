"""Attention sublayer in fp64 on the CPU: per-head norm with rotation, masked
attention and its backward, written from the formulas, with elementwise bounds
on what a kernel may differ by.

The bounds count roundings.  Stored values are off by at most r = half a step
of their type, relative (bf16 2⁻⁸, fp32 2⁻²⁴).  A score is a sum of Dh fp32
products, off by at most E = (Dh + 8)·2⁻²⁴·scale·Σ|q||k| + 2⁻²¹·(1 + |s|); a
probability then by 2·max E of its row relative, plus r where it is rounded for
the matrix cores; sums of n terms by n·2⁻²⁴ of their absolute terms.
"""

from __future__ import annotations

import numpy as np

U = 2.0 ** -24
R = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def rope(x, w, pos, freqs, eps, interleaved):
    """[T, H, Dh] normed, weighted and rotated."""
    x = np.asarray(x, np.float64)
    D, h = x.shape[-1], len(freqs)
    u = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1.0 if w is None else np.asarray(w, np.float64))
    ang = np.asarray(pos, np.float64)[:, None, None] * np.asarray(freqs, np.float64)
    c, s = np.cos(ang), np.sin(ang)
    ia = np.arange(h) * 2 if interleaved else np.arange(h)
    ib = ia + 1 if interleaved else ia + h
    y = u.copy()
    y[..., ia] = u[..., ia] * c - u[..., ib] * s
    y[..., ib] = u[..., ia] * s + u[..., ib] * c
    assert 2 * h <= D
    return y


def rope_bwd(dy, x, w, pos, freqs, eps, interleaved):
    """(dx, dw) of rope."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    h = len(freqs)
    w = np.ones(x.shape[-1]) if w is None else np.asarray(w, np.float64)
    ang = np.asarray(pos, np.float64)[:, None, None] * np.asarray(freqs, np.float64)
    c, s = np.cos(ang), np.sin(ang)
    ia = np.arange(h) * 2 if interleaved else np.arange(h)
    ib = ia + 1 if interleaved else ia + h
    g = dy.copy()
    g[..., ia] = dy[..., ia] * c + dy[..., ib] * s
    g[..., ib] = -dy[..., ia] * s + dy[..., ib] * c
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    dw = (g * x * r).sum((0, 1))
    return r * w * g - x * r ** 3 * (w * g * x).mean(-1, keepdims=True), dw


def visible(T, docs=None, causal=True, prefix=None, window=0):
    """[T, T] truth values: row i sees key j."""
    docs = [0, T] if docs is None else list(docs)
    ok = np.zeros((T, T), bool)
    i = np.arange(T)
    for d, (a, b) in enumerate(zip(docs, docs[1:])):
        m = np.ones((b - a, b - a), bool)
        if causal:
            away = i[a:b, None] - i[None, a:b]
            m = away >= 0
            if window:
                m &= away < window
            if prefix is not None:
                m[:, :max(0, int(prefix[d]))] = True
        ok[a:b, a:b] = m
    return ok


def _scores(q, k, ok, dist, scale, softcap, slope):
    x = scale * (q @ k.T)
    t = np.tanh(x / softcap) if softcap else None
    s = softcap * t if softcap else x
    if slope is not None:
        s = s - slope * dist
    err = (q.shape[1] + 8) * U * scale * (np.abs(q) @ np.abs(k).T) + 2.0 ** -21 * (1.0 + np.abs(s))
    s = np.where(ok, s, -np.inf)
    m = s.max(-1, keepdims=True, initial=-np.inf)
    p = np.exp(s - np.where(np.isfinite(m), m, 0.0))
    z = p.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = np.where(z > 0, np.where(np.isfinite(m), m, 0.0) + np.log(z), -np.inf)[:, 0]
    p = p / np.where(z > 0, z, 1.0)
    err = np.where(ok, err, 0.0).max(-1, keepdims=True, initial=0.0)
    return p, lse, (1.0 - t * t if softcap else 1.0), 2.0 * err


def attention(q, k, v, ok, dist, *, io, scale, softcap=0.0, slopes=None):
    """Rows q[m, Hq, Dh] over keys k, v[n, Hk, Dh]: (o, lse[Hq, m], bound of o)."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    m, Hq, D = q.shape
    G = Hq // k.shape[1]
    o, bound, lse = np.zeros(q.shape), np.zeros(q.shape), np.zeros((Hq, m))
    ro, rp = R[io], (R["bf16"] if io == "bf16" else 0.0)
    for h in range(Hq):
        kk, vv = k[:, h // G], v[:, h // G]
        p, lse[h], _, e = _scores(q[:, h], kk, ok, dist, scale, softcap, None if slopes is None else slopes[h])
        o[:, h] = p @ vv
        bound[:, h] = (rp + e + 2 * (len(kk) + 8) * U) * (p @ np.abs(vv)) + 1.01 * ro * np.abs(o[:, h])
    return o, lse, 1.01 * bound + 1e-30


def attention_bwd(do, q, k, v, ok, dist, *, io, scale, softcap=0.0, slopes=None):
    """(dq, dk, dv) and their bounds, for a kernel that is given its own o and lse."""
    do, q, k, v = (np.asarray(a, np.float64) for a in (do, q, k, v))
    Hq = q.shape[1]
    G = Hq // k.shape[1]
    o, _, eo = attention(q, k, v, ok, dist, io=io, scale=scale, softcap=softcap, slopes=slopes)
    g = [np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)]
    b = [np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)]
    ro, rp = R[io], (R["bf16"] if io == "bf16" else 0.0)
    for h in range(Hq):
        kk, vv = k[:, h // G], v[:, h // G]
        p, _, dcap, e = _scores(q[:, h], kk, ok, dist, scale, softcap, None if slopes is None else slopes[h])
        dp = do[:, h] @ vv.T
        delta = (do[:, h] * o[:, h]).sum(-1, keepdims=True)
        ds = p * (dp - delta) * dcap * scale
        n = len(kk) + q.shape[2] + 8
        # probability, δ (from the stored o), dP, the capping's derivative, and the sums
        edelta = (np.abs(do[:, h]) * eo[:, h]).sum(-1, keepdims=True) + n * U * (np.abs(do[:, h]) * np.abs(o[:, h])).sum(-1, keepdims=True)
        edp = n * U * (np.abs(do[:, h]) @ np.abs(vv).T)
        eds = (rp + 2 * e + 2 * n * U) * np.abs(ds) + p * scale * (edelta + edp) + 4 * e * p * np.abs(dp - delta) * scale * bool(softcap)
        g[0][:, h] = ds @ kk
        b[0][:, h] = (eds + n * U * np.abs(ds)) @ np.abs(kk)
        g[1][:, h // G] += ds.T @ q[:, h]
        b[1][:, h // G] += (eds + G * n * U * np.abs(ds)).T @ np.abs(q[:, h])
        g[2][:, h // G] += p.T @ do[:, h]
        b[2][:, h // G] += ((rp + 2 * e + 2 * G * n * U) * p).T @ np.abs(do[:, h])
    return g, [1.01 * (x + 1.01 * ro * np.abs(y)) + 1e-30 for x, y in zip(b, g)]
