"""The operators around the routed experts in 64 bits on the CPU (test side; numpy only)."""
import math

import numpy as np

U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}  # the largest relative error of one rounding
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -24, "f32": 2.0 ** -149}  # the smallest subnormal: underflow is absolute


def route(logits, k, score, bias=None, n_group=1, topk_group=1, group_top=1, renormalize=True, scale=1.0,
          lowest=-np.finfo(np.float32).max):
    """(ids [T, k], weights [T, k], gap [T]): gap is the smallest distance between two values that were compared."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    ids = np.zeros((T, k), np.int64)
    w = np.zeros((T, k))
    gap = np.full(T, np.inf)

    def nearest(v):
        v = np.sort(v[np.isfinite(v)])
        return np.min(np.diff(v)) if v.size > 1 else np.inf

    for t in range(T):
        out = ~(l[t] > lowest)
        s = np.zeros(E)
        here = ~out
        if score == "sigmoid":
            s[here] = 1.0 / (1.0 + np.exp(-l[t, here]))
        elif here.any():
            m = l[t, here].max()
            e = np.where(l[t, here] == m, 1.0, np.exp(l[t, here] - m))
            s[here] = e / e.sum()
        c = s.copy() if (score == "sigmoid" or bias is not None) else l[t].copy()
        if bias is not None:
            c = s + np.asarray(bias, np.float64)
        c[out] = -np.inf
        gap[t] = nearest(c)
        if n_group > 1:
            gs = E // n_group
            best = -np.sort(-c.reshape(n_group, gs), axis=1)[:, :group_top].sum(axis=1)
            gap[t] = min(gap[t], nearest(best))
            order = np.argsort(-best, kind="stable")[:topk_group]
            keep = np.zeros(n_group, bool)
            keep[order] = True
            c[~np.repeat(keep, gs)] = -np.inf
        ids[t] = np.argsort(-c, kind="stable")[:k]
        w[t] = np.where(np.isneginf(c[ids[t]]), 0.0, s[ids[t]])
        if renormalize:
            w[t] /= w[t].sum() + 1e-20
    return ids, w * scale, gap


def norm(v, kind, w, b, eps):
    """(norm(v), bound of its fp32 error where v is exact up to `dv`) as a function of dv."""
    H = v.shape[1]
    if kind == "none":
        return v, lambda dv: dv
    mean = v.mean(axis=1, keepdims=True) if kind == "layer" else 0.0
    d = v - mean
    inv = 1.0 / np.sqrt((d * d).mean(axis=1, keepdims=True) + eps)
    wv = 1.0 if w is None else np.asarray(w, np.float64)[None, :]
    y = d * inv * wv + (0.0 if b is None else np.asarray(b, np.float64)[None, :])
    # one lane adds at most 32 terms and a tree joins at most 1024 lanes: 48 roundings of 2^-24 in every sum,
    # 16 more for the elementwise steps
    c = 64 * 2.0 ** -24

    def bound(dv):
        dd = dv + (np.abs(dv).mean(axis=1, keepdims=True) + c * np.abs(v).mean(axis=1, keepdims=True)
                   if kind == "layer" else 0.0)
        rel = c + np.sqrt((dd * dd).mean(axis=1, keepdims=True)) * inv  # of the scale factor
        return np.abs(wv) * inv * dd + (c + rel) * (np.abs(d) * inv * np.abs(wv)) + c * np.abs(y)

    return y, bound


def block_norm(f, r, post, w_post, b_post, gate, branch, resid, pre, w_pre, b_pre, eps, rows_per_gate=1):
    """((h, bound), (y, bound)) before the roundings to the output types."""
    f = np.asarray(f, np.float64)
    u, bu = norm(f, post, w_post, b_post, eps)
    g = 1.0
    if gate is not None:
        g = np.repeat(np.asarray(gate, np.float64), rows_per_gate, axis=0)
    h = branch * g * u
    dh = np.abs(branch * g) * bu(np.zeros_like(f)) + 8 * 2.0 ** -24 * np.abs(h)
    if r is not None:
        h = h + resid * np.asarray(r, np.float64)
        dh = dh + 8 * 2.0 ** -24 * np.abs(resid * np.asarray(r, np.float64))
    y, by = norm(h, pre, w_pre, b_pre, eps)
    return (h, dh), (y, by(dh))


_erf = np.vectorize(math.erf)


def act(z, name):
    if name == "relu":
        return np.maximum(z, 0.0)
    if name == "silu":
        return z / (1.0 + np.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1.0 + _erf(z / math.sqrt(2.0)))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def linear(x, w, bias=None, name="none", gated=False, residual=None):
    """(out, bound of the fp32 error) before the rounding to the output type."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    z = x @ w.T
    # products of 16-bit values are exact in fp32; the tensor core adds 16 of them at a time, and each of the
    # K / 16 accumulations (plus 16 for splits and their sums) is off by at most one unit in the last place
    dz = (x.shape[1] / 16 + 16) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)
    if bias is not None:
        z = z + np.asarray(bias, np.float64)[None, :]
        dz = dz + 2.0 ** -23 * np.abs(z)
    n = w.shape[0] // 2 if gated else w.shape[0]
    # |act'| <= 1.13 for all of them; the functions themselves are good to a few units of fp32, absolute ones
    # where 1 + erf or 1 + tanh cancels
    a = act(z[:, :n], name)
    da = 1.13 * dz[:, :n] + (0.0 if name == "none" else 16 * 2.0 ** -24 * (np.abs(a) + np.abs(z[:, :n])))
    if gated:
        a, da = a * z[:, n:], da * np.abs(z[:, n:]) + np.abs(a) * dz[:, n:] + da * dz[:, n:]
    if residual is not None:
        a = a + np.asarray(residual, np.float64)
        da = da + 2.0 ** -23 * np.abs(a)
    return a, da


def check(got, ref, bound, dtype, what=""):
    """got (of `dtype`, as float64) is ref within its fp32 error bound and one rounding to its type."""
    got = np.asarray(got, np.float64)
    lim = bound + U[dtype] * (np.abs(ref) + bound) + TINY[dtype]
    bad = ~(np.abs(got - ref) <= lim)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], ref[bad][:4], lim[bad][:4])
