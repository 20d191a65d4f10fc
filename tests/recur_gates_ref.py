"""Bounds of the gated linear recurrence element by element, relative to what
reaches an element and not to the largest value anywhere, for gates that are
wide open.

With e = 2^-24, w = sigmoid(k) and its complement sigmoid(-k), evaluated in
fp32, each have a relative error of at most d = (|k| + 8) 2e (recur_ref derives
it).  Along a chain of kept shares, h_t = keep_t h_{t-1} + w_t v_t, let
H_t = keep_t H_{t-1} + w_t |v_t|, H_0 = |h0|, the same with everything positive.
A step may be evaluated from either end, h + w (v - h) or v + keep (h - v); with
the smaller of the two gates as the factor, both the rounded difference and the
error of the gate are multiplied by it, min(w, keep) |v - h| <= H_t, and the sum
rounds once: a step adds at most H_t (d + 2e) and passes on what it was given
times keep_t.  A chain cut into pieces rounds each piece's product of shares and
each composition besides: twice the steps' own errors cover them.  So
    E_t = keep_t E_{t-1} + 2 H_t (d_t + 4e).
The gradient chain p_t = keep_t g_t, g_t = dy_t s_t + p_{t+1} is the same with
G_t = |dy_t s_t| + P_{t+1}, P_t = keep_t G_t.  Results multiply these with
factors of the relative errors above; a type of fewer bits adds half a step.
Values below 1e-36 may be lost (a gate of K = 88 is below the normal fp32 range).
With w as the factor where it is near 1, the error is e |h_{t-1}| or e g_t, which
the bounds do not allow once keep_t |h_{t-1}| or the rest of H_t is smaller.
"""
import numpy as np

import recur_ref as ref

E = 2.0 ** -24
FLOOR = 1e-36


def _d(x):
    return (np.abs(x) + 8) * 2 * E


def definition(K, V, R, h0, offsets, dY, dhT):
    """(Y, hT, dK, dV, dR, dh0, h, h before, g) in 64 bits, with sigmoid(-k) for
    the kept share: 1 - sigmoid(k) has nothing left of it from k = 37 on."""
    T, C = K.shape
    w, keep, s, soff = ref.sig(K), ref.sig(-K), ref.sig(R), ref.sig(-R)
    h, hb, g = (np.full((T, C), np.nan) for _ in range(3))
    hT, dh0 = np.array(h0, dtype=np.float64), np.array(dhT, dtype=np.float64)
    for i, a, b in ref.sequences(offsets, T):
        for t in range(a, b):
            hb[t] = hT[i]
            hT[i] = keep[t] * hT[i] + w[t] * V[t]
            h[t] = hT[i]
        for t in range(b - 1, a - 1, -1):
            g[t] = dY[t] * s[t] + dh0[i]
            dh0[i] = keep[t] * g[t]
    return s * h, hT, g * (V - hb) * w * keep, g * w, dY * h * s * soff, dh0, h, hb, g


def bounds(K, V, R, h0, offsets, dY, dhT, u):
    """Bounds of Y, hT, dK, dV, dR, dh0 (rows of no sequence: NaN); u: half a step
    of the activations' type."""
    T, C = K.shape
    w, keep, s, soff = ref.sig(K), ref.sig(-K), ref.sig(R), ref.sig(-R)
    Y, hT, dK, dV, dR, dh0, h, hb, g = definition(K, V, R, h0, offsets, dY, dhT)
    nan = lambda: np.full((T, C), np.nan)
    H, Eh, Ehb = nan(), nan(), nan()
    ET = np.zeros_like(hT)
    for i, a, b in ref.sequences(offsets, T):
        x, err = np.abs(h0[i]).astype(np.float64), np.zeros(C)
        for t in range(a, b):
            Ehb[t] = err
            x = keep[t] * x + w[t] * np.abs(V[t])
            err = keep[t] * err + 2 * x * (_d(K[t]) + 4 * E)
            H[t], Eh[t] = x, err
        ET[i] = err
    Eg, Ep = nan(), np.zeros_like(dh0)
    for i, a, b in ref.sequences(offsets, T):
        P, err = np.abs(dhT[i]).astype(np.float64), np.zeros(C)
        for t in range(b - 1, a - 1, -1):
            own = np.abs(dY[t] * s[t])
            G = own + P
            Eg[t] = err + own * (_d(R[t]) + 2 * E) + E * G
            P = keep[t] * G
            err = keep[t] * Eg[t] + 2 * P * (_d(K[t]) + 4 * E)
        Ep[i] = err
    x = np.abs(V - hb)
    Ex = Ehb + E * x
    return [s * Eh + np.abs(Y) * (_d(R) + u) + FLOOR, ET + FLOOR,
            w * keep * (Eg * x + np.abs(g) * Ex + Eg * Ex) + np.abs(dK) * (3 * _d(K) + u) + FLOOR,
            w * Eg + np.abs(dV) * (2 * _d(K) + u) + FLOOR,
            np.abs(dY) * s * soff * Eh + np.abs(dR) * (3 * _d(R) + u) + FLOOR,
            Ep + FLOOR]


def evaluate(K, V, R, h0, offsets, dY, dhT, forward_from_w=False, backward_from_w=False):
    """The recurrence and its gradients in fp32, token by token, with the
    smaller gate as every step's factor; *_from_w: with w always, which loses
    the kept share of an open gate."""
    f = np.float32
    K, V, R, h0, dY, dhT = (np.asarray(x, dtype=f) for x in (K, V, R, h0, dY, dhT))
    T, C = K.shape
    sig = lambda x: (f(1) / (f(1) + np.exp(-x))).astype(f)
    w, keep, s, soff = sig(K), sig(-K), sig(R), sig(-R)
    nan = lambda: np.full((T, C), np.nan, dtype=f)
    Y, dK, dV, dR, hb, h = (nan() for _ in range(6))
    hT, dh0 = h0.copy(), dhT.copy()
    for i, a, b in ref.sequences(offsets, T):
        x = h0[i].copy()
        for t in range(a, b):
            hb[t] = x
            low = x + w[t] * (V[t] - x)
            x = low if forward_from_w else np.where(K[t] < 0, low, V[t] + keep[t] * (x - V[t]))
            h[t] = x
        Y[a:b], hT[i] = s[a:b] * h[a:b], x
        p = dhT[i].copy()
        for t in range(b - 1, a - 1, -1):
            g = dY[t] * s[t] + p
            dR[t] = dY[t] * s[t] * soff[t] * h[t]
            dV[t] = g * w[t]
            dK[t] = dV[t] * (V[t] - hb[t]) * keep[t]
            low = g - w[t] * g
            p = low if backward_from_w else np.where(K[t] < 0, low, keep[t] * g)
        dh0[i] = p
    return Y, hT, dK, dV, dR, dh0


def inputs(T, C, lens, gate, seed, what):
    """K of the given range of biases and, by `what`:
    'late'   dY only on the last 3 tokens of each sequence, so that what reaches the
             tokens before has passed every gate in between;
    'reset'  states of 1e4 that meet values of 1e-3;
    'still'  V zero but for the first token of a sequence."""
    rng = np.random.default_rng(seed)
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    S = len(lens)
    f = lambda *s: rng.normal(0, 1, s).astype(np.float32)
    d = dict(K=f(T, C) + rng.uniform(*gate, C).astype(np.float32), V=f(T, C), R=f(T, C), h0=0.5 * f(S, C), offsets=off,
             dY=0.5 * f(T, C), dhT=0.5 * f(S, C))
    inside = np.arange(T)[:, None] - off[None, :-1]
    here = (inside >= 0) & (np.arange(T)[:, None] < off[None, 1:])
    if what == "late":
        left = off[None, 1:] - np.arange(T)[:, None]
        d["dY"] *= np.any(here & (left <= 3), axis=1)[:, None]
        d["dhT"] *= 0
    elif what == "reset":
        d["h0"] *= 2e4
        d["V"] *= 1e-3
    elif what == "still":
        d["V"] *= np.any(here & (inside == 0), axis=1)[:, None]
    return d


GATES = [(-2.0, 4.0), (6.0, 12.0), (14.0, 20.0), (20.0, 60.0)]
NAMES = ("Y", "hT", "dK", "dV", "dR", "dh0")
