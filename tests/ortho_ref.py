"""The Newton-Schulz orthogonalisation in 64 bits, and the same with the
roundings the library documents (X, A and A's polynomial held in fp16 under
power-of-two scales), whose distance from the former sets the tests' bounds:
the kernel makes the same roundings on values that differ from these by fp32
sums only, so its error is of the same size, though not the same."""
import torch

A, B, C, EPS = 3.4445, -4.7750, 2.0315, 1e-7


def _wide(G):
    return (G.t(), True) if G.shape[0] > G.shape[1] else (G, False)


def exact(G, steps=5):
    X, tall = _wide(G.double())
    X = X / (torch.sqrt((X * X).sum()) + EPS)
    for _ in range(steps):
        P = X @ X.t().contiguous()
        X = A * X + (B * P + C * (P @ P)) @ X
    return X.t() if tall else X


def rounded(G, steps=5):
    q = lambda t, s: (t * s).to(torch.float16).double() / s
    X, tall = _wide(G.double())
    X = q(X / (torch.sqrt((X * X).sum()) + EPS), 2.0 ** 14)
    for i in range(steps):
        P = q(X @ X.t().contiguous(), 2.0 ** 14)
        X = A * X + q(B * P + C * (P @ P), 2.0 ** 13) @ X
        if i < steps - 1:
            X = q(X, 2.0 ** 14)
    return X.t() if tall else X


def bounds(G, steps=5):
    """(exact, Frobenius bound, element bound): twice the emulation's distance,
    plus half a step of bf16; for a single element eight times the emulation's
    rms in its row or its column, whichever is larger, plus half a step.

    An element's error is a sum of hundreds of roundings and so close to normal,
    with a deviation that follows the size of its column (the roundings of X
    are relative to it: columns of G that are 10 times larger carry errors 10
    times larger) or row; 8 deviations are exceeded once in 10^15 elements.  The rms
    of the whole matrix would not do: columns drawn from [0.01, 0.1] reach 1.7
    times it, so that 8 of it are 4.7 deviations there, once in 4 10^5.
    """
    E = exact(G, steps)
    d = rounded(G, steps) - E
    rms = torch.maximum(d.pow(2).mean(1, keepdim=True).sqrt(), d.pow(2).mean(0, keepdim=True).sqrt())
    return E, 2 * float(d.norm()) + 2.0 ** -8 * float(E.norm()) + 1e-30, 8 * rms + 2.0 ** -8 * E.abs() + 1e-30
