"""The gated linear recurrence in 64 bits, token by token, with the bounds its
fp32 evaluation keeps.

Bounds.  w = sigmoid(k) in fp32 has a relative error of at most
(|k| + 6) 2^-23: the argument of the exponential is rounded (|k| 2^-24 after
the exponential), the exponential and the reciprocal are good to one unit in
the last place, the sum to half of one.  A step h + w (v - h) rounds twice, by at
most 2^-24 of values no larger than H = the running maximum of |v|, |h0| and
|h| (times 2 for the difference), and carries the error of the state before it
with the weight 1 - w; the weights (1 - w)^j of the steps before add up to at most
n = min(longest sequence, 1 / min w), and sum_j (1 - w)^j w <= 1 takes the
error of w itself.  Cutting the chain into chunks adds the products A, which
round once a step: the same n again.  So
    |h - h64| <= H ((kmax + 6) 2^-22 + 8 n 2^-24).
The gradient chain is the same with G, the chain of |dy s|, in the place of H
and the relative error of s added.  dK, dV, dR multiply these with factors of
the relative errors above, and every output in a type of fewer bits adds half a
step of that type.  n 2^-24 counts rounding errors as if all had one sign.
"""
import numpy as np


def sig(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def sequences(offsets, T):
    off = [0, T] if offsets is None else list(offsets)
    return [(s, off[s], off[s + 1]) for s in range(len(off) - 1)]


def forward(K, V, R, h0, offsets):
    """(Y, hT, h, h_before) in f64; rows of no sequence hold NaN."""
    T, C = K.shape
    seqs = sequences(offsets, T)
    w, s = sig(K), sig(R)
    h = np.full((T, C), np.nan)
    hb = np.full((T, C), np.nan)
    hT = np.array(h0, dtype=np.float64)
    for i, a, b in seqs:
        x = hT[i].copy()
        for t in range(a, b):
            hb[t] = x
            x = x + w[t] * (V[t] - x)
            h[t] = x
        hT[i] = x
    return s * h, hT, h, hb


def backward(K, V, R, h0, offsets, dY, dhT):
    """(dK, dV, dR, dh0, g, G): G is the gradient chain of the absolute values."""
    T, C = K.shape
    _, _, h, hb = forward(K, V, R, h0, offsets)
    w, s = sig(K), sig(R)
    g = np.full((T, C), np.nan)
    G = np.full((T, C), np.nan)
    dh0 = np.array(dhT, dtype=np.float64)
    for i, a, b in sequences(offsets, T):
        p, P = dh0[i].copy(), np.abs(dh0[i])
        for t in range(b - 1, a - 1, -1):
            g[t] = dY[t] * s[t] + p
            G[t] = np.abs(dY[t] * s[t]) + P
            p, P = (1 - w[t]) * g[t], (1 - w[t]) * G[t]
        dh0[i] = p
    return g * (V - hb) * w * sig(-K), g * w, dY * h * s * sig(-R), dh0, g, G


def _n(K, offsets, T):
    longest = max([b - a for _, a, b in sequences(offsets, T)] + [1])
    return min(longest, 1.0 / max(sig(K).min(), 1e-30)) if K.size else 1.0


def _max(*xs):
    return max([float(np.nanmax(np.abs(x))) for x in xs if x.size and not np.all(np.isnan(x))] + [0.0])


def tol_h(K, V, h0, offsets):
    e = 2.0 ** -24
    return _max(V, h0) * ((_max(K) + 6) * 4 * e + 8 * _n(K, offsets, len(K)) * e) + 1e-30


def tol_fwd(K, V, R, h0, offsets, u):
    """Bounds of Y and hT; u: half a step of Y's type, relative."""
    Y, _, h, _ = forward(K, V, R, h0, offsets)
    th = tol_h(K, V, h0, offsets)
    return sig(R) * th + np.abs(Y) * ((np.abs(R) + 8) * 2.0 ** -23 + u) + 1e-30, th


def tol_bwd(K, V, R, h0, offsets, dY, dhT, u):
    """Bounds of dK, dV, dR, dh0."""
    e23 = 2.0 ** -23
    dK, dV, dR, dh0, g, G = backward(K, V, R, h0, offsets, dY, dhT)
    _, _, h, hb = forward(K, V, R, h0, offsets)
    th = tol_h(K, V, h0, offsets)
    n = _n(K, offsets, len(K))
    tg = _max(G, dhT) * ((_max(K) + _max(R) + 12) * 2 * e23 + 8 * n * 2.0 ** -24) + 1e-30
    w, wd, sd = sig(K), sig(K) * sig(-K), sig(R) * sig(-R)
    rel = (2 * np.abs(K) + 16) * e23
    d = np.abs(V - hb)
    tK = wd * (tg * d + np.abs(g) * (th + d * rel) + tg * th) + np.abs(dK) * u + 1e-30
    tV = w * (tg + np.abs(g) * rel) + np.abs(dV) * u + 1e-30
    tR = np.abs(dY) * sd * (th + np.abs(h) * (2 * np.abs(R) + 16) * e23) + np.abs(dR) * u + 1e-30
    return tK, tV, tR, tg
