"""Layer norm on the GPU against the formulas in 64 bits, element by element
within bounds that count the roundings (tests/rows_ref.py)."""
import itertools

import pytest
import torch

import rows_ref as ref
import ternary_weight_linear_tern_amd as tl

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
WIDTHS = [8, 64, 72, 512, 520, 1024, 1032, 2048, 2056, 4096, 4104, 8192, 8200, 16384, 16392, 20000]


def rand(shape, seed, dt=F32, size=1.0, shift=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * size + shift).to(dt)


def fwd(X, y, w=None, b=None, A=None, eps=1e-5, stats=True):
    T, C = X.shape
    Y = torch.full((T, C), 7.0, dtype=y, device="cuda")
    S = torch.empty_like(X) if A is not None else None
    st = tl.empty_norm_stats(T) if stats else None
    tl.tern_norm_fwd(X, Y, w=w, b=b, A=A, S=S, stats=st, eps=eps)
    return Y, S, st


def check_fwd(X, y, w=None, b=None, A=None, eps=1e-5, tag=""):
    Y, S, st = fwd(X, y, w, b, A, eps)
    src = X
    if A is not None:
        want = (X.float() + A.float()).to(X.dtype)
        assert torch.equal(S, want), tag
        src = want
    Yr, mu, r, e, emu, er = ref.norm_fwd(src, w, b, eps)
    ref.assert_within(st[:, :1], mu, emu, tag + " mu")
    ref.assert_within(st[:, 1:], r, er, tag + " r")
    ref.assert_within(Y, Yr, e + ref.half_step(y) * (Yr.abs() + e), tag + " Y")
    return Y, S, st


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("T", [1, 5, 67])
def test_forward_sizes(T, C):
    X, w, b = rand((T, C), C, size=2.0, shift=0.5), rand((C,), 1, shift=1.0), rand((C,), 2)
    check_fwd(X, F32, w, b, tag=f"{T} x {C} f32")
    check_fwd(X.to(BF), BF, w, b, A=rand((T, C), 3, BF), tag=f"{T} x {C} bf16")


@pytest.mark.parametrize("x,a,y", list(itertools.product([BF, F32], [None, BF, F32], [BF, F32])))
def test_forward_types(x, a, y):
    for T, C in ((3, 264), (9, 2048), (4, 5000)):
        check_fwd(rand((T, C), 5, x), y, rand((C,), 6), rand((C,), 7), A=None if a is None else rand((T, C), 8, a),
                  tag=f"{x} {a} {y} {T} x {C}")


def test_forward_without_weight_or_bias():
    X, w = rand((6, 328), 1), rand((328,), 2)
    check_fwd(X, F32)
    check_fwd(X, F32, w=w)
    check_fwd(X, BF, b=w)
    Y, _, st = fwd(X, F32, stats=False)
    assert st is None and torch.equal(Y, fwd(X, F32)[0])


def test_forward_hard_rows():
    """Equal elements, a mean far from zero, one large element, tiny and large rows."""
    C = 1032
    X = rand((8, C), 1)
    X[0] = 3.0
    X[1] = 0.0
    X[2] += 1e4
    X[3, 17] = 1e4
    X[4] *= 1e-12
    X[5] *= 1e15
    X[6] = torch.arange(C, device="cuda") % 2 * 2.0 - 1.0
    w, b = rand((C,), 2), rand((C,), 3)
    check_fwd(X, F32, w, b, eps=1e-5)
    check_fwd(X, F32, w, b, eps=1e-12)


def test_forward_strides_and_in_place():
    T, C = 37, 520
    wide = rand((T, 3 * C), 4, BF)
    keep = wide.clone()
    X, A, Y = wide[:, :C], wide[:, C:2 * C], wide[:, 2 * C:]
    w = rand((C,), 5)
    want = (X.float() + A.float()).to(BF)
    Yr, *_ = fwd(X.contiguous(), BF, w, A=A.contiguous())
    st = tl.empty_norm_stats(T)
    tl.tern_norm_fwd(X, Y, w=w, A=A, S=X, stats=st)             # the stream updated in place
    assert torch.equal(X, want) and torch.equal(A, keep[:, C:2 * C]) and torch.equal(Y, Yr)
    # rows of a wider matrix stay as they are between the columns
    big = torch.full((T, C + 64), -5.0, device="cuda")
    tl.tern_norm_fwd(rand((T, C), 6), big[:, 8:8 + C])
    assert bool((big[:, :8] == -5).all()) and bool((big[:, 8 + C:] == -5).all())


def test_non_finite_rows_stay_alone():
    X = rand((6, 2048), 1)
    good = fwd(X, F32)[0]
    X[1, 5], X[3, 2047] = float("nan"), float("inf")
    Y = fwd(X, F32)[0]
    for t in range(6):
        assert bool(torch.isnan(Y[t]).any()) if t in (1, 3) else torch.equal(Y[t], good[t])


def test_empty():
    tl.tern_norm_fwd(torch.empty(0, 64, device="cuda"), torch.empty(0, 64, device="cuda"))
    tl.tern_norm_fwd(torch.empty(4, 0, device="cuda"), torch.empty(4, 0, device="cuda"))
    dw, db = torch.full((64,), 3.0, device="cuda"), torch.full((64,), 3.0, device="cuda")
    e = torch.empty(0, 64, device="cuda")
    tl.tern_norm_bwd(e, tl.empty_norm_stats(0), e, torch.empty_like(e), tl.empty_norm_workspace(0, 64), dw=dw, db=db)
    assert bool((dw == 0).all()) and bool((db == 0).all())


def check_bwd(S, y, dx, w=None, ds=False, weights=True, seed=1, tag=""):
    T, C = S.shape
    _, _, st = fwd(S, F32, w)
    dY = rand((T, C), seed + 10, y, 0.1, 0.03)
    dS = rand((T, C), seed + 11, dx) if ds else None
    dX = torch.full((T, C), 9.0, dtype=dx, device="cuda")
    dw, db = (torch.full((C,), 9.0, device="cuda") if weights else None for _ in range(2))
    ws = tl.empty_norm_workspace(T, C) if weights else None
    tl.tern_norm_bwd(S, st, dY, dX, ws, w=w, dS=dS, dw=dw, db=db)
    X, W, B, e, ew, eb = ref.norm_bwd(S, st, w, dY, dS)
    ref.assert_within(dX, X, e + ref.half_step(dx) * (X.abs() + e), tag + " dX")
    if weights:
        ref.assert_within(dw, W, ew, tag + " dw")
        ref.assert_within(db, B, eb, tag + " db")
    return dX, dw, db


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("T", [1, 6, 131])
def test_backward_sizes(T, C):
    w = rand((C,), 1, shift=1.0)
    check_bwd(rand((T, C), C, F32, 2.0, 0.5), F32, F32, w, ds=True, tag=f"{T} x {C} f32")
    check_bwd(rand((T, C), C, BF, 2.0, 0.5), F32, BF, w, tag=f"{T} x {C} bf16")


@pytest.mark.parametrize("s,y,dx", [(F32, F32, F32), (F32, BF, F32), (BF, F32, F32), (BF, BF, F32), (BF, F32, BF),
                                    (BF, BF, BF)])
@pytest.mark.parametrize("ds", [False, True])
def test_backward_types(s, y, dx, ds):
    for T, C in ((3, 264), (40, 2048), (4, 5000)):
        check_bwd(rand((T, C), 5, s), y, dx, rand((C,), 6), ds, tag=f"{s} {y} {dx} {T} x {C}")


@pytest.mark.parametrize("T", [2000, 5003, 40000])
def test_backward_many_rows(T):
    check_bwd(rand((T, 136), 3, BF), BF, BF, rand((136,), 4), tag=str(T))


def test_backward_parts():
    S, w = rand((50, 1032), 1), rand((1032,), 2)
    dX, dw, db = check_bwd(S, F32, F32, w)
    alone, _, _ = check_bwd(S, F32, F32, w, weights=False)
    assert torch.equal(dX, alone)
    check_bwd(S, F32, F32)
    st = fwd(S, F32, w)[2]
    dY, only, out = rand((50, 1032), 11, F32, 0.1, 0.03), torch.empty(1032, device="cuda"), torch.empty_like(S)
    ws = tl.empty_norm_workspace(50, 1032)
    tl.tern_norm_bwd(S, st, dY, out, ws, w=w, dw=only)
    assert torch.equal(only, dw)
    tl.tern_norm_bwd(S, st, dY, out, ws, w=w, db=only)
    assert torch.equal(only, db) and torch.equal(out, dX)


def test_backward_strides_and_in_place():
    T, C = 37, 520
    wide = rand((T, 3 * C), 4)
    S, dY, acc = wide[:, :C], wide[:, C:2 * C], wide[:, 2 * C:]
    w = rand((C,), 5)
    st = fwd(S.contiguous(), F32, w)[2]
    want = torch.empty(T, C, device="cuda")
    ws = tl.empty_norm_workspace(T, C)
    dw, db, dw2, db2 = (torch.empty(C, device="cuda") for _ in range(4))
    tl.tern_norm_bwd(S.contiguous(), st, dY.contiguous(), want, ws, w=w, dS=acc.contiguous(), dw=dw, db=db)
    keep = wide[:, :2 * C].clone()
    tl.tern_norm_bwd(S, st, dY, acc, ws, w=w, dS=acc, dw=dw2, db=db2)      # the stream's gradient in place
    assert torch.equal(acc, want) and torch.equal(dw, dw2) and torch.equal(db, db2)
    assert torch.equal(wide[:, :2 * C], keep)


def test_backward_against_differences():
    """sum(Y dY) moved along one element: the formula's gradient (which the kernel is held to above) is the
    difference quotient in 64 bits."""
    T, C, eps, h = 3, 40, 1e-5, 1e-5
    S, w, b = rand((T, C), 1), rand((C,), 2), rand((C,), 3)
    dY = rand((T, C), 4).double()
    st = fwd(S, F32, w, b, eps=eps)[2]
    dX, dw, db = torch.empty_like(S), torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
    tl.tern_norm_bwd(S, st, dY.float(), dX, tl.empty_norm_workspace(T, C), w=w, dw=dw, db=db)
    f = lambda S, w, b: (ref.norm_fwd(S, w, b, eps)[0] * dY).sum()
    for t, c in ((0, 0), (1, 17), (2, 39)):
        step = torch.zeros(T, C, dtype=torch.float64, device="cuda")
        step[t, c] = h
        q = (f(S.double() + step, w, b) - f(S.double() - step, w, b)) / (2 * h)
        # third derivatives of this row are below 50: h^2 / 6 of them; 2^-53 of sums below 300, over h
        assert abs(float(q) - float(dX[t, c])) < 1e-7 + 64 * ref.U * 30
        q = (f(S, w.double() + step[t], b) - f(S, w.double() - step[t], b)) / (2 * h)
        assert abs(float(q) - float(dw[c])) < 1e-7 + 64 * ref.U * 30
        q = (f(S, w, b.double() + step[t]) - f(S, w, b.double() - step[t])) / (2 * h)
        assert abs(float(q) - float(db[c])) < 1e-7 + 64 * ref.U * 30


@pytest.mark.parametrize("T,C", [(1, 64), (63, 64), (64, 64), (65, 8), (1000, 128), (777, 136), (300, 256), (40, 264)])
def test_narrow_rows(T, C):
    """Rows that take part of a wave: next to each other, and less than a workgroup has."""
    w, b = rand((C,), 1, shift=1.0), rand((C,), 2)
    check_fwd(rand((T, C), 3, F32, 2.0, 0.5), BF, w, b, A=rand((T, C), 4, BF), tag=f"{T} x {C}")
    check_bwd(rand((T, C), 5, BF, 2.0, 0.5), BF, F32, w, ds=True, tag=f"{T} x {C}")


def test_far_rows():
    """Offsets past 2^31 elements: the last rows of a matrix of 2.3e9."""
    T, C = 140000, 16384
    tail, w = rand((3, C), 1, BF), rand((C,), 2)
    X = torch.zeros(T, C, dtype=BF, device="cuda")
    X[-3:] = tail
    st = tl.empty_norm_stats(T)
    Y = torch.full((T, C), 9.0, dtype=BF, device="cuda")
    tl.tern_norm_fwd(X, Y, w=w, stats=st)
    want, _, wst = fwd(tail, BF, w)
    assert torch.equal(Y[-3:], want) and torch.equal(st[-3:], wst) and not bool(Y[:4].any())
    dw, db = torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
    dY = X                                            # zero but for the last rows
    tl.tern_norm_bwd(X, st, dY, Y, tl.empty_norm_workspace(T, C), w=w, dw=dw, db=db)
    dX, gw, gb, e, ew, eb = ref.norm_bwd(tail, wst, w, tail, None)
    ref.assert_within(Y[-3:], dX, e + ref.half_step(BF) * (dX.abs() + e), "dX")
    ref.assert_within(dw, gw, ew, "dw")
    ref.assert_within(db, gb, eb, "db")
    assert not bool(Y[:4].any())


def test_repeats_bitwise():
    S, w = rand((3000, 1032), 1, BF), rand((1032,), 2)
    first = check_bwd(S, BF, BF, w)
    for _ in range(3):
        again = check_bwd(S, BF, BF, w)
        assert all(torch.equal(x, y) for x, y in zip(first, again))
