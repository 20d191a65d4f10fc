"""Layer norm where workgroups go on to further rows, every row another one and checked:
forward (sum, statistics and result) and backward, within bounds that count the
additions which the rule for the rows' groups gives."""
import math

import pytest
import torch

import rows_ref as ref
import ternary_weight_linear_tern_amd as tl
from test_gpu_norm import check_fwd, rand

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = ref.U


def rows_at_once(C, waves):
    """Rows that a workgroup of about this many waves takes at once (up to 16384 columns)."""
    if C <= 512:
        return waves * 64 // (8 if C <= 64 else 16 if C <= 128 else 32 if C <= 256 else 64)
    return max(1, waves // math.ceil(C / (512 if C <= 8192 else 1024)))


def turns(T, C):
    """Row groups of the backward, and the rows that a lane adds up."""
    groups = tl.tern_norm_bwd_workspace_bytes(T, C) // (8 * C)
    return groups, math.ceil(T / (groups * (rows_at_once(C, 8) if C <= 16384 else 1)))


@pytest.mark.parametrize("T,C", [(70001, 64), (35001, 128), (17003, 200), (9001, 512), (5003, 1032), (4500, 2048), (2100, 2056),
                                 (2100, 8192), (2100, 12000)])
@pytest.mark.parametrize("x,y", [(F32, BF), (BF, F32)])
def test_forward(T, C, x, y):
    assert T > 2048 * rows_at_once(C, 4)                 # more than the workgroups take at once
    w, b = rand((C,), 1, shift=1.0), rand((C,), 2)
    X, A = rand((T, C), 3, x, 2.0, 0.5), rand((T, C), 4, BF)
    X[::7] *= 3.0                                        # neighbours of other sizes
    check_fwd(X, y, w, b, A=A, tag=f"{T} x {C} {x}")
    check_fwd(X, y, w, b, tag=f"{T} x {C} {x} without A")


def test_forward_longest_rows():
    """More rows than workgroups, each longer than the registers: the last ones and the first."""
    T, C = 65600, 16392
    X = torch.empty(T, C, dtype=BF, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    w, b, st = rand((C,), 1, shift=1.0), rand((C,), 2), tl.empty_norm_stats(T)
    Y = torch.empty(T, C, dtype=BF, device="cuda")
    tl.tern_norm_fwd(X, Y, w=w, b=b, stats=st)
    for s in (slice(0, 70), slice(65500, T)):
        want, mu, r, e, emu, er = ref.norm_fwd(X[s], w, b, 1e-5)
        ref.assert_within(st[s, :1], mu, emu, "mu")
        ref.assert_within(st[s, 1:], r, er, "r")
        ref.assert_within(Y[s], want, e + ref.half_step(BF) * (want.abs() + e), "Y")


@pytest.mark.parametrize("T,C", [(70001, 64), (9001, 512), (5003, 1032), (1500, 2056), (1500, 4096), (1100, 8192), (300, 16384),
                                 (1000, 16384), (300, 20000), (3000, 20000), (1000, 1048576 // 8)])
@pytest.mark.parametrize("s,dy,dx", [(F32, F32, F32), (BF, F32, BF)])
def test_backward(T, C, s, dy, dx):
    groups, chain = turns(T, C)
    assert chain > 1
    w, b = rand((C,), 1, shift=1.0), rand((C,), 2)
    S = rand((T, C), 3, s, 2.0, 0.5)
    tag = f"{T} x {C} {s}"
    _, _, st = check_fwd(S, F32, w, b, tag=tag)
    dY, dS = rand((T, C), 5, dy, 0.1, 0.03), rand((T, C), 6, dx)
    dX = torch.full((T, C), 9.0, dtype=dx, device="cuda")
    dw, db = torch.full((C,), 9.0, device="cuda"), torch.full((C,), 9.0, device="cuda")
    tl.tern_norm_bwd(S, st, dY, dX, tl.empty_norm_workspace(T, C), w=w, dS=dS, dw=dw, db=db)
    want, gw, gb, e, _, _ = ref.norm_bwd(S, st, w, dY, dS)
    ref.assert_within(dX, want, e + ref.half_step(dx) * (want.abs() + e), tag + " dX")
    # a lane's rows, then those side by side in its workgroup; the groups in 64 bits; a product adds its own three
    n = chain + (rows_at_once(C, 8) if C <= 16384 else 1)
    xh = (S.double() - st[:, :1].double()) * st[:, 1:].double()
    mine = (dY.double() * xh).abs().sum(0)
    ref.assert_within(dw, gw, (n + 3) * U * mine + U * gw.abs(), tag + " dw")
    ref.assert_within(db, gb, n * U * dY.double().abs().sum(0) + U * gb.abs(), tag + " db")
