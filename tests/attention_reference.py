"""The operators of the attention half in 64 bits (numpy), with bounds on what their fp32 arithmetic may be off."""
import math

import numpy as np

HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}  # half a step of a rounding, relative
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150}  # half a step among the smallest numbers
U = 2.0 ** -24


def inv_freq(R, base=10000.0):
    return base ** (-2.0 * np.arange(R // 2) / R)


def rotate(x, pos, f, interleaved=False, start=0, scale=1.0, inverse=False):
    """x [T, H, D] -> (rotated, bound): fractions of a turn are in fp32 (2^-25 half-turns: 1.6 u of an angle), sincospif is
    within 2 units (2 u), then the scale, two products and their sum are rounded: below 8 u (|a| + |b|) * scale."""
    R = 2 * len(f)
    out, size = x.copy(), np.zeros_like(x)
    part = x[:, :, start:start + R]
    a, b = (part[..., 0::2], part[..., 1::2]) if interleaved else (part[..., :R // 2], part[..., R // 2:])
    t = pos.astype(np.float64)[:, None, None] * np.asarray(f)[None, None, :] * (-1 if inverse else 1)
    p, q = scale * (a * np.cos(t) - b * np.sin(t)), scale * (b * np.cos(t) + a * np.sin(t))
    m = abs(scale) * (np.abs(a) + np.abs(b))
    if interleaved:
        out[:, :, start:start + R] = np.stack([p, q], -1).reshape(part.shape)
        size[:, :, start:start + R] = np.stack([m, m], -1).reshape(part.shape)
    else:
        out[:, :, start:start + R] = np.concatenate([p, q], -1)
        size[:, :, start:start + R] = np.concatenate([m, m], -1)
    return out, 8 * U * size


def rounded(want, dtype, slack):
    return HALF[dtype] * np.abs(want) + TINY[dtype] + slack * (1 + HALF[dtype])


def attend(q, k, v, scale, dtype, piece):
    """One sequence: q [Hq, D], k, v [n, Hkv, D] -> (out, its bound, lse, its bound).  `piece`: what a weight is off by when
    it goes to the product with the values, relative."""
    Hq, D = q.shape
    n, Hkv, _ = k.shape
    if n == 0:
        return np.zeros((Hq, D)), np.zeros((Hq, D)), np.full(Hq, -np.inf), np.zeros(Hq)
    G = Hq // Hkv
    out, bound, lse, lb = np.empty((Hq, D)), np.empty((Hq, D)), np.empty(Hq), np.empty(Hq)
    for h in range(Hq):
        kk, vv = k[:, h // G], v[:, h // G]
        s = scale * (kk @ q[h])
        # sums on the tensor core are cut off at each of D / 16 additions of 16 products, at most a unit of each product
        # and of the sum: 17 * 2 u of the sum of the products' sizes each; then three rounded factors
        ds = abs(scale) * (np.abs(kk) @ np.abs(q[h])).max() * (34 * math.ceil(D / 16) + 6) * U
        top = s.max()
        p = np.exp(s - top)
        w = p / p.sum()
        out[h] = w @ vv
        lse[h] = top + np.log(p.sum())
        # weights: scores and the exponential (2 units); sums of n weights and rescalings, 16 at a time on the tensor core
        rel = 2 * ds + 8 * U + (2 * n / 16 + 64) * 2 * U
        size = w @ np.abs(vv)
        bound[h] = rounded(out[h], dtype, size * (piece + 2 * rel) + 2.0 ** -24 * np.abs(vv).max() / p.sum())
        lb[h] = ds + (2 * n / 16 + 64) * 2 * U + 4 * U * (1 + abs(lse[h]) + abs(top))
    return out, bound, lse, lb


def e4m3_values():
    """The value of every E4M3 code."""
    c = np.arange(256)
    s, e, m = np.where(c & 128, -1.0, 1.0), (c >> 3) & 15, c & 7
    v = s * np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))
    v[[0x7F, 0xFF]] = np.nan
    return v


def block_linear(a, a_s, b, b_s, dtype):
    """a [M, K], b [N, K] values of codes, a_s [M, G], b_s [ceil(N/128), G] -> (out, bound): a group is four additions of 32
    products on the tensor core, each cut off at most a unit (2 u) of its 33 terms' largest; then a rounding of the scale,
    the product and the sum for each group."""
    M, K = a.shape
    N, G = b.shape[0], K // 128
    out, size = np.zeros((M, N)), np.zeros((M, N))
    for g in range(G):
        c = slice(128 * g, 128 * g + 128)
        s = a_s[:, g:g + 1] * np.repeat(b_s[:, g], 128)[:N][None, :]
        out += s * (a[:, c] @ b[:, c].T)
        size += np.abs(s) * (np.abs(a[:, c]) @ np.abs(b[:, c]).T)
    return out, rounded(out, dtype, size * (4 * 33 * 2 + 2 * G + 4) * U)
