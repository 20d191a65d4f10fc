"""Rows of logits of which some are 0 and the others -inf (tokens that are not
allowed): every exponential is exactly 1 or 0 and every sum a whole number below
2^24, so that a row's log-sum-exp and entropy are log n of its n allowed tokens, to
the rounding of one logarithm, and one token lost or counted twice shows.

U is half a step of fp32; a logarithm is off by two steps at most."""
import torch

from rows_ref import F64, U

LOG = 4 * U      # a logarithm's error, in proportion


def allowed_rows(T, V, seed, device):
    """[T, V] truth values: all tokens; half of them at random; few; those of the last, partial eight;
    those at the borders of strides of 512 and 2048; a single one: the first, the last, any."""
    g = torch.Generator(device=device).manual_seed(seed)
    i = torch.arange(V, device=device)
    rest = i >= min(V // 8 * 8, V - 1)
    out = torch.zeros(T, V, dtype=torch.bool, device=device)
    for t in range(T):
        kind = t % 9
        if kind == 0:
            row = i >= 0
        elif kind == 1:
            row = torch.rand(V, generator=g, device=device) < 0.5
        elif kind == 2:
            row = torch.rand(V, generator=g, device=device) < 8.0 / V
        elif kind == 3:
            row = rest
        elif kind == 4:
            row = (i % 512 == 0) | (i % 512 == 511)
        elif kind == 5:
            row = (i % 2048 >= 2040) | rest
        elif kind == 6:
            row = i == 0
        elif kind == 7:
            row = i == V - 1
        else:
            row = i == int(torch.randint(0, V, (1,), generator=g, device=device))
        out[t] = row
        if kind in (1, 2, 4, 5):
            out[t, int(torch.randint(0, V, (1,), generator=g, device=device))] = True
    return out


def logits_of(allowed, dt):
    T, V = allowed.shape
    buf = torch.full((T, (V + 7) // 8 * 8), float("nan"), dtype=dt, device=allowed.device)
    buf[:, :V] = torch.where(allowed, 0.0, -float("inf")).to(dt)
    return buf[:, :V]


def some_allowed(allowed, k, seed):
    """[T, k] allowed tokens of each row, at random, the same one more than once among them."""
    n = allowed.sum(1)
    g = torch.Generator(device=allowed.device).manual_seed(seed)
    rank = (torch.rand(allowed.shape[0], k, generator=g, device=allowed.device, dtype=F64) * n[:, None]).long()
    rank = torch.minimum(rank, n[:, None] - 1)
    before = torch.cumsum(allowed, 1, dtype=torch.int32)            # the r-th allowed token is where this gets to r + 1
    return torch.searchsorted(before, (rank + 1).int())


def log_count(n):
    """log n and its bound."""
    L = torch.log(n.to(F64))
    return L, LOG * L


def loss(n, alpha, tau):
    """Against a teacher of four entries of probability 1/4 each, which are allowed tokens, and an allowed target:
    alpha log n + (1 - alpha) tau^2 (log n - log 4), and its bound: each logarithm, the difference, the
    sum of four equal terms, three factors and the sum of the two parts."""
    L, four = torch.log(n.to(F64)), torch.log(torch.tensor(4.0, dtype=F64))
    f = (1 - alpha) * tau ** 2
    return alpha * L + f * (L - four), 12 * U * (alpha * L + f * (L + four))


def gradient(allowed, y, ids, alpha, tau, w):
    """dZ of that loss, and its bound but for the rounding to dZ's type."""
    n = allowed.sum(1).to(F64)
    q = torch.where(allowed, (w.to(F64) / n)[:, None], 0.0)
    f = (1 - alpha) * tau
    G = (alpha + f) * q
    E = G.clone()
    for at, p in ((y[:, None], alpha), (ids, f / 4)):
        less = (w.to(F64)[:, None] * p).expand_as(at).contiguous()
        G.scatter_add_(1, at, -less)
        E.scatter_add_(1, at, less)
    return G, 8 * U * E
