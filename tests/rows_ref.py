"""64-bit references of the row operators (layer norm, token log probabilities,
distillation loss) in plain torch, and how far a result in 32 bits may be off.

U is half a step of fp32.  A sum of terms x_i in which no term passes more than n
additions is off by at most n U sum |x_i|."""
import math

import torch

U = 2.0 ** -24
F64 = torch.float64


def half_step(dt):
    return torch.finfo(dt).eps / 2


def assert_within(got, want, bound, tag=""):
    """Each element within its bound; where the wanted value is not finite, the same."""
    got, want, bound = got.double().cpu(), want.double().cpu(), torch.as_tensor(bound, dtype=F64).cpu()
    assert got.shape == want.shape, (tag, got.shape, want.shape)
    bound = bound.expand_as(want)
    odd = ~torch.isfinite(want)
    same = torch.where(torch.isnan(want), torch.isnan(got), got == want)
    ok = torch.where(odd, same, (got - want).abs() <= bound)
    if not bool(ok.all()):
        i = tuple(torch.nonzero(~ok)[0].tolist())
        raise AssertionError(f"{tag}: element {list(i)} is {got[i]!r}, wanted {want[i]!r} +- {bound[i]!r} "
                             f"({int((~ok).sum())} elements out of bound)")


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------

def row_chain(C):
    """Additions a term of a row's sum passes: a wave at least shares a row, eight
    neighbours a lane, then six steps in the wave and up to 16 waves."""
    return math.ceil(C / 64) + 8 + 6 + 16


def norm_fwd(S, w, b, eps):
    """Y, mu, r of the rows of S (as stored), and the bounds of each for a result
    of the steps: mean, squares of the differences, their mean, root, product."""
    x = S.to(F64)
    C = x.shape[1]
    w = torch.ones(C, dtype=F64, device=x.device) if w is None else w.to(F64)
    b = torch.zeros(C, dtype=F64, device=x.device) if b is None else b.to(F64)
    mu = x.mean(1, keepdim=True)
    var = ((x - mu) ** 2).mean(1, keepdim=True)
    r = (var + eps) ** -0.5
    xh = (x - mu) * r
    Y = xh * w + b
    n = row_chain(C)
    dmu = (n + 1) * U * x.abs().mean(1, keepdim=True) + U * mu.abs()
    # the squares are taken around mu + dmu: their mean gains dmu^2; each difference rounds by U
    rel = 0.5 * ((n + 6) * U + dmu ** 2 / (var + eps)) + 4 * U
    dY = w.abs() * r * dmu * (1 + rel) + (xh * w).abs() * (rel + 4 * U) + 2 * U * ((xh * w).abs() + b.abs())
    return Y, mu, r, dY, dmu, rel * r


def norm_bwd(S, stats, w, dY, dS):
    """dX, dw, db from the statistics as given, and the bounds of each."""
    x, dy = S.to(F64), dY.to(F64)
    T, C = x.shape
    w = torch.ones(C, dtype=F64, device=x.device) if w is None else w.to(F64)
    mu, r = stats[:, :1].to(F64), stats[:, 1:].to(F64)
    xh, g = (x - mu) * r, dy * w
    m1, m2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    inner = g - m1 - xh * m2
    dX = r * inner
    ds = torch.zeros_like(x) if dS is None else dS.to(F64)
    n = row_chain(C)
    e1 = (n + 2) * U * g.abs().mean(1, keepdim=True)
    e2 = (n + 5) * U * (g * xh).abs().mean(1, keepdim=True)
    err = r * (e1 + xh.abs() * e2 + 6 * U * (g.abs() + m1.abs() + (xh * m2).abs()))
    err = err + 2 * U * (ds.abs() + dX.abs())
    # a column's sum: the rows of a group (T / 256 and 64 at most), then the groups in 64 bits
    nt = T / 256 + 64
    dw, db = (dy * xh).sum(0), dy.sum(0)
    return (dX + ds, dw, db, err, (nt + 4) * U * (dy * xh).abs().sum(0) + U * dw.abs(),
            nt * U * dy.abs().sum(0) + U * db.abs())


# ---------------------------------------------------------------------------
# softmax rows
# ---------------------------------------------------------------------------

# additions a term of a row's sum passes: at most 512 in a lane (a row of 2^20 logits
# is cut into segments of at most 2^17), six in the wave, 16 waves, and the segments
ROW_SUM = 512 + 6 + 16 + 16


def log_softmax(z):
    """In 64 bits, and the log-sum-exp; a row of nothing but -inf has log p = -inf
    everywhere.  (From the largest on: a row of the type's lowest value alone is uniform,
    and loses log V next to that value.)"""
    m = z.amax(1, keepdim=True)
    dead = m == -math.inf
    m0 = torch.where(dead, torch.zeros_like(m), m)
    logs = torch.log(torch.exp(z - m0).sum(1, keepdim=True))
    return torch.where(dead, torch.full_like(z, -math.inf), z - m0 - logs), m0 + logs


def _spread(z, L):
    """Mean over the row's distribution, and each element's distance, from the
    largest logit: what a relative error of the exponents costs."""
    m = z.amax(1, keepdim=True)
    d = torch.where(torch.isfinite(z), (z - m).abs(), torch.zeros_like(z))
    p = torch.where(L > -math.inf, torch.exp(L), torch.zeros_like(L))
    return d, (p * torch.nan_to_num(d)).sum(1, keepdim=True)


def log_error(z, L):
    """Bound of log p of every element: the factor's and the exponent's rounding and
    exp2's last place on each term (each in proportion to the distance from the
    largest), the sum, and the result's rounding."""
    d, mean = _spread(z, L)
    return U * (4 * d + 4 * mean + ROW_SUM + 8) + U * torch.nan_to_num(L, neginf=0.0).abs()


def top(Z, k):
    """The k largest of each row by falling value, ties by rising index."""
    return torch.sort(Z.float(), dim=1, descending=True, stable=True).indices[:, :k]


def logprob(Z, scale, tokens, k):
    """dict of (value, bound) of each output; top_ids is exact."""
    z = Z.to(F64) * scale
    V = z.shape[1]
    L, lse = log_softmax(z)
    err = log_error(z, L)
    d, mean = _spread(z, L)
    p = torch.where(L > -math.inf, torch.exp(L), torch.where(torch.isnan(L), L, torch.zeros_like(L)))
    H = -torch.where(p > 0, p * L, p * 0).sum(1)
    H = torch.where(torch.isnan(lse[:, 0]), lse[:, 0], H)
    out = dict(lse=(lse[:, 0], (U * (4 * lse.abs() + 4 * mean + ROW_SUM + 8))[:, 0]),
               entropy=(H, U * (ROW_SUM + 16) * (1 + 2 * mean[:, 0]) + U * H.abs()))
    if tokens is not None:
        ok = (tokens >= 0) & (tokens < V)
        at = tokens.clamp(0, V - 1)[:, None]
        zero = torch.zeros_like(H)
        out["logp"] = (torch.where(ok, L.gather(1, at)[:, 0], zero), torch.where(ok, err.gather(1, at)[:, 0], zero))
    if k:
        ids = top(Z, k)
        out["top_ids"] = ids
        out["top_logp"] = (L.gather(1, ids), err.gather(1, ids))
    return out


def teacher(ids, lp, V):
    """p and log p of the teacher's entries (0 and -inf where there is none), and
    which rows have any."""
    lp = lp.to(F64)
    live = (ids >= 0) & (ids < V) & (lp != -math.inf)
    masked = torch.where(live, lp, torch.full_like(lp, -math.inf))
    L = log_softmax(masked)[0] if lp.shape[1] else masked
    return torch.where(live, L, torch.full_like(L, -math.inf)), live


def distill(Z, targets, ids, lp, alpha, tau, dloss):
    """loss, dZ and their bounds."""
    z = Z.to(F64)
    T, V = z.shape
    zero = torch.zeros(T, dtype=F64, device=z.device)
    G, GE = torch.zeros_like(z), torch.zeros_like(z)
    loss, le = zero.clone(), zero.clone()
    ce = torch.zeros(T, dtype=torch.bool, device=z.device)
    kl = ce.clone()
    if targets is not None and alpha > 0:
        L, _ = log_softmax(z)
        E = log_error(z, L)
        q = torch.exp(L)
        ce = (targets >= 0) & (targets < V)
        at = targets.clamp(0, V - 1)[:, None]
        loss = loss - torch.where(ce, alpha * L.gather(1, at)[:, 0], zero)
        le = le + torch.where(ce, alpha * E.gather(1, at)[:, 0], zero)
        part = alpha * q
        part = part.scatter_add(1, at, torch.full_like(at, -alpha, dtype=F64))
        G = G + torch.where(ce[:, None], part, 0.0)
        e = (alpha * q) * (E + 8 * U)
        e = e.scatter_add(1, at, torch.full_like(at, 2 * U * alpha, dtype=F64))
        GE = GE + torch.where(ce[:, None], e, 0.0)
    if ids is not None and ids.shape[1] and alpha < 1:
        L, _ = log_softmax(z / tau)
        E = log_error(z / tau, L)
        q = torch.exp(L)
        LP, live = teacher(ids, lp, V)
        kl = live.any(1)
        p = torch.where(live, torch.exp(LP), torch.zeros_like(LP))
        at = ids.clamp(0, V - 1)
        lq, eq = L.gather(1, at), E.gather(1, at)
        some = (p > 0) | torch.isnan(p)
        term = torch.where(some, p * (LP - lq), torch.zeros_like(p))
        # p: the exponent's rounding, exp2, the sum of 64, the quotient
        rel = (80 + 4 * torch.nan_to_num(LP, neginf=0.0).abs()) * U
        et = torch.where(some, p * (rel * (1 + torch.nan_to_num(LP - lq, posinf=0.0).abs()) + torch.nan_to_num(eq)), 0.0)
        f = (1 - alpha) * tau
        loss = loss + torch.where(kl, f * tau * term.sum(1), zero)
        le = le + torch.where(kl, f * tau * (et.sum(1) + 8 * U * torch.nan_to_num(term, posinf=0.0).abs().sum(1)), zero)
        part = (f * q).scatter_add(1, at, torch.where(live, -f * p, 0.0))
        G = G + torch.where(kl[:, None], part, 0.0)
        e = (f * q * (E + 8 * U)).scatter_add(1, at, torch.where(live, f * p * (rel + 8 * U), 0.0))
        GE = GE + torch.where(kl[:, None], e, 0.0)
    w = torch.ones(T, dtype=F64, device=z.device) if dloss is None else dloss.to(F64)
    gone = (w == 0) | ~(ce | kl)
    loss = torch.where(ce | kl, loss, zero)
    dZ = torch.where(gone[:, None], torch.zeros_like(G), G * w[:, None])
    # below 2^-126 a probability may be flushed to zero
    GE = torch.where(gone[:, None], torch.zeros_like(GE), GE * w.abs()[:, None])
    return loss, torch.where(ce | kl, le + U * torch.nan_to_num(loss, posinf=0.0).abs(), zero), dZ, GE + 2.0 ** -120
