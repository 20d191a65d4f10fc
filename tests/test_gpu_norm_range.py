"""Layer norm of rows whose differences square beyond fp32's range (above about
1e19), against the formulas in 64 bits: alone, beside ordinary rows, in one wave of
several, and where only the waves' means are that far apart."""
import pytest
import torch

import rows_ref as ref
import ternary_weight_linear_tern_amd as tl
from test_gpu_norm import fwd, rand

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
WIDTHS = [8, 64, 200, 264, 512, 520, 1032, 2048, 5000, 8192, 8200, 16384, 16392, 20000]
ORDINARY = [3, 9, 11]


def far_rows(C, dt, seed=1):
    i = torch.arange(C, device="cuda")
    R = lambda s, size=1.0, shift=0.0: rand((C,), seed * 100 + s, size=size, shift=shift)
    return torch.stack([
        R(0, 1e20), R(1, 1e30), R(2, 3e37), R(3),
        torch.where(i == C // 2, 3e38, R(4)),                       # one element far from the others
        torch.where(i % 4 == 1, -3e38, 3e38),                       # differences beyond the range itself
        torch.where(i // 512 % 2 == 0, 8e18, -8e18),                # each wave's own squares are small
        R(7, 1e25, 1e30), R(8, 5e17), R(9, 2.0, 0.5),
        torch.where(i < 8, R(10, 1e30), R(10)),                     # one lane's
        R(11, 1e15), torch.full((C,), 3e38, device="cuda")]).to(dt)


def check(X, y, w, b, A=None, tag=""):
    Y, S, st = fwd(X, y, w, b, A)
    src = X if A is None else (X.float() + A.float()).to(X.dtype)
    if A is not None:
        assert torch.equal(S, src), tag
    want, mu, r, e, emu, er = ref.norm_fwd(src, w, b, 1e-5)
    ref.assert_within(st[:, :1], mu, emu, tag + " mu")
    # r of deviations above 2^126 is one of fp32's denormal numbers, in steps of 2^-149
    ref.assert_within(st[:, 1:], r, er + 2.0 ** -149, tag + " r")
    ref.assert_within(Y, want, e + ref.half_step(y) * (want.abs() + e), tag + " Y")
    return Y, st


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("dt", [F32, BF])
def test_forward(C, dt):
    X, w, b = far_rows(C, dt), rand((C,), 1, shift=1.0), rand((C,), 2)
    Y, st = check(X, F32, w, b, tag=f"{C} {dt}")
    check(X.repeat(7, 1), BF, w, b, A=rand((7 * X.shape[0], C), 3, BF), tag=f"{C} {dt} + A")
    # rows of ordinary size are not touched by what their neighbours hold
    plain = X.clone()
    plain[[t for t in range(X.shape[0]) if t not in ORDINARY]] = 1.0
    Y1, _, st1 = fwd(plain, F32, w, b)
    assert torch.equal(Y[ORDINARY], Y1[ORDINARY]) and torch.equal(st[ORDINARY], st1[ORDINARY])


@pytest.mark.parametrize("C", [64, 520, 2048, 8200, 20000])
def test_non_finite_rows_among_them(C):
    X, w = far_rows(C, F32), rand((C,), 1, shift=1.0)
    good = fwd(X, F32, w)[0]
    X[1, C // 3], X[3, 5], X[8, C - 1] = float("nan"), float("inf"), -float("inf")
    Y = fwd(X, F32, w)[0]
    for t in range(X.shape[0]):
        assert bool(torch.isnan(Y[t]).any()) if t in (1, 3, 8) else torch.equal(Y[t], good[t]), t


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("dt", [F32, BF])
def test_backward(C, dt):
    X, w = far_rows(C, dt), rand((C,), 1, shift=1.0)
    st = fwd(X, F32, w)[2]
    T = X.shape[0]
    dY, dS = rand((T, C), 4, size=0.1, shift=0.03), rand((T, C), 5, size=1e-3)
    dX, dw, db = torch.full((T, C), 9.0, device="cuda"), torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
    tl.tern_norm_bwd(X, st, dY, dX, tl.empty_norm_workspace(T, C), w=w, dS=dS, dw=dw, db=db)
    want, gw, gb, e, ew, eb = ref.norm_bwd(X, st, w, dY, dS)
    ref.assert_within(dX, want, e + ref.half_step(F32) * (want.abs() + e), f"{C} {dt} dX")
    ref.assert_within(dw, gw, ew, f"{C} {dt} dw")
    ref.assert_within(db, gb, eb, f"{C} {dt} db")


@pytest.mark.parametrize("T,C", [(70001, 64), (35001, 200), (9001, 512), (5003, 1024), (4500, 2048), (2100, 12000)])
@pytest.mark.parametrize("dt", [F32, BF])
def test_many_rows_in_place(T, C, dt):
    """Far rows in any turn of a workgroup, the stream updated in place."""
    X, A, w, b = rand((T, C), 1, dt, 2.0, 0.5), rand((T, C), 2, BF), rand((C,), 3, shift=1.0), rand((C,), 4)
    far = far_rows(C, dt)
    for i in range(far.shape[0]):
        X[(i * 2741 + 5) % T] = far[i]
    X[T - 1], X[T - 2] = far[1], far[4]
    S = (X.float() + A.float()).to(dt)
    Y, st = torch.empty(T, C, device="cuda"), tl.empty_norm_stats(T)
    tl.tern_norm_fwd(X, Y, w=w, b=b, A=A, S=X, stats=st)
    assert torch.equal(X, S)
    want, mu, r, e, emu, er = ref.norm_fwd(S, w, b, 1e-5)
    ref.assert_within(st[:, :1], mu, emu, f"{T} x {C} {dt} mu")
    ref.assert_within(st[:, 1:], r, er + 2.0 ** -149, f"{T} x {C} {dt} r")
    ref.assert_within(Y, want, e + ref.half_step(F32) * (want.abs() + e), f"{T} x {C} {dt} Y")
