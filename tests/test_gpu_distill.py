"""The distillation loss and its gradient on the GPU against the formulas in 64
bits, element by element (tests/rows_ref.py)."""
import math

import pytest
import torch

import rows_ref as ref
import ternary_weight_linear_tern_amd as tl
from test_gpu_logprob import hard_rows, logits

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
INF = math.inf


def teacher(T, V, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.stack([torch.randperm(V, generator=g, device="cuda")[:K] for _ in range(T)]) if T else torch.zeros(
        0, K, dtype=torch.int64, device="cuda")
    lp = torch.log_softmax(torch.randn(T, K + 1, generator=g, device="cuda") * 2, 1)[:, :K].contiguous()
    return ids, lp


def run(Z, targets=None, ids=None, lp=None, alpha=0.0, tau=1.0, dloss=None, grad=True, in_place=False):
    T, V = Z.shape
    loss = torch.full((T,), 77.0, device="cuda")
    dZ = None
    if in_place:
        dZ = Z
    elif grad:
        ld = Z.stride(0) + 8 if T > 1 else (V + 15) // 8 * 8
        buf = torch.full((T, ld), 55.0, dtype=Z.dtype, device="cuda")
        dZ = buf[:, :V]
    tl.tern_distill(Z, tl.empty_distill_workspace(T, V), targets=targets, teacher_ids=ids, teacher_logp=lp, alpha=alpha,
                    tau=tau, loss=loss, dloss=dloss, dZ=dZ)
    if grad and not in_place:
        assert bool((buf[:, V:] == 55.0).all())          # columns from V on are left
    return loss, dZ


def check(Z, targets=None, ids=None, lp=None, alpha=0.0, tau=1.0, dloss=None, tag=""):
    loss, dZ = run(Z, targets, ids, lp, alpha, tau, dloss)
    L, le, G, ge = ref.distill(Z, targets, ids, lp, alpha, tau, dloss)
    ref.assert_within(loss, L, le, tag + " loss")
    ref.assert_within(dZ, G, ge + ref.half_step(Z.dtype) * (G.abs() + ge), tag + " dZ")
    alone, _ = run(Z, targets, ids, lp, alpha, tau, dloss, grad=False)
    # (the loss alone may cut rows otherwise: the same sums in another order, within the same bound)
    ref.assert_within(alone, L, le, tag + " loss alone")
    return loss, dZ


def targets_of(T, V, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-1, V + 1, (T,), generator=g, device="cuda")


@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 65, 255, 256, 257, 513, 1000, 2048, 4100, 8191, 16384, 32771, 50021, 65536,
                               65544, 131072, 131077, 262147, 1048576])
@pytest.mark.parametrize("dt", [F32, BF])
def test_sizes(V, dt):
    for T in (1, 5 if V < 300000 else 2):
        K = min(V, 20)
        ids, lp = teacher(T, V, K, V)
        w = torch.linspace(0.5, 1.5, T, device="cuda")
        check(logits(T, V, V + T, dt), targets_of(T, V), ids, lp, 0.3, 2.0, w, tag=f"{T} x {V} {dt}")
        check(logits(T, V, V + T, dt, extra=16), None, ids, lp, 0.0, 1.0, tag=f"{T} x {V} {dt} kl")
    check(logits(2, V, 6, dt), targets_of(2, V), alpha=1.0, tag=f"{V} {dt} ce")


@pytest.mark.parametrize("T,V", [(300, 256), (1500, 1000), (700, 8200), (600, 65536), (260, 131072), (20000, 64)])
@pytest.mark.parametrize("dt", [F32, BF])
def test_many_rows(T, V, dt):
    ids, lp = teacher(min(T, 64), V, 32, 1)
    n = -(-T // ids.shape[0])
    ids, lp = ids.repeat(n, 1)[:T].contiguous(), lp.repeat(n, 1)[:T].contiguous()
    check(logits(T, V, 2, dt), targets_of(T, V), ids, lp, 0.1, 2.0, tag=f"{T} x {V} {dt}")


@pytest.mark.parametrize("alpha", [0.0, 0.25, 1.0])
@pytest.mark.parametrize("tau", [1.0, 2.0, 0.5])
@pytest.mark.parametrize("K", [0, 1, 63, 64])
def test_factors(alpha, tau, K):
    T, V = 6, 3001
    ids, lp = teacher(T, V, K, 3) if K else (None, None)
    check(logits(T, V, 1), targets_of(T, V), ids, lp, alpha, tau, tag=f"{alpha} {tau} {K}")
    check(logits(T, V, 1), None, ids, lp, alpha, tau, tag=f"{alpha} {tau} {K} no targets")


@pytest.mark.parametrize("V", [300, 60000, 200000])
@pytest.mark.parametrize("dt", [F32, BF])
def test_teachers_entries(V, dt):
    """Padding, entries that are none, the same token twice, the target among them,
    one entry far above the others, probabilities that do not sum to one."""
    T, K = 9, 16
    ids, lp = teacher(T, V, K, 5)
    y = targets_of(T, V)
    ids[0, 3:] = -1
    ids[1] = -1                                  # no entries at all
    lp[2] = -INF                                 # nor here
    ids[3, 5] = ids[3, 2]                        # twice
    ids[3, 9] = ids[3, 2]                        # three times
    y[3] = ids[3, 2]
    y[4] = ids[4, 7]
    lp[5] += 40.0
    lp[6, 1:] -= 200.0                           # p of the others is nothing
    ids[7, 4], ids[7, 5] = V, 1 << 40
    ids[8, ::2] = 0
    y[8] = 0
    check(logits(T, V, 1, dt), y, ids, lp, 0.5, 2.0, tag=str(V))
    check(logits(T, V, 1, dt), None, ids, lp, 0.0, 1.0, tag=str(V))


@pytest.mark.parametrize("V", [64, 1000, 40000, 131072])
@pytest.mark.parametrize("dt", [F32, BF])
def test_hard_rows(V, dt):
    Z = hard_rows(V, dt)
    T = Z.shape[0]
    ids, lp = teacher(T, V, 8, 2)
    y = targets_of(T, V).clamp(0, V - 1)
    loss, dZ = check(Z, y, ids, lp, 0.5, 1.0, tag=f"{V} {dt}")
    assert float(loss[1]) == INF                 # the row in which nothing is allowed
    # nothing asked of that row: nothing comes of it
    y[1], ids[1] = -1, -1
    loss, dZ = check(Z, y, ids, lp, 0.5, 1.0, tag=f"{V} {dt} none")
    assert float(loss[1]) == 0 and bool((dZ[1] == 0).all())


@pytest.mark.parametrize("V", [100, 3000, 131072])
def test_non_finite_rows_stay_alone(V):
    T = 8
    Z = logits(T, V, 4)
    ids, lp = teacher(T, V, 5, 1)
    y = targets_of(T, V).clamp(0, V - 1)
    good = run(Z, y, ids, lp, 0.5, 2.0)
    w = torch.ones(T, device="cuda")
    Z[1, 5], Z[3, V - 1], Z[5] = math.nan, INF, math.nan
    lp[6, 2] = math.nan
    Z[7, 0], w[7] = math.nan, 0.0                # a row without weight is 0 whatever it holds
    loss, dZ = run(Z, y, ids, lp, 0.5, 2.0, w)
    for t in (0, 2, 4):
        assert torch.equal(loss[t], good[0][t]) and torch.equal(dZ[t], good[1][t])
    for t in (1, 3, 5):
        assert bool(torch.isnan(loss[t])) and bool(torch.isnan(dZ[t]).all())
    assert bool(torch.isnan(loss[6])) and bool(torch.isnan(dZ[6, ids[6]]).all())
    assert bool((dZ[7] == 0).all())


@pytest.mark.parametrize("T,V", [(4, 256), (300, 5003), (3, 131072), (300, 131072), (2, 400000)])
@pytest.mark.parametrize("dt", [F32, BF])
def test_in_place(T, V, dt):
    Z = logits(T, V, 1, dt, extra=8)
    ids, lp = teacher(2, V, 9, 1)
    ids, lp = ids.repeat(T, 1)[:T].contiguous(), lp.repeat(T, 1)[:T].contiguous()
    y = targets_of(T, V)
    loss, dZ = run(Z, y, ids, lp, 0.4, 2.0)
    over = logits(T, V, 1, dt, extra=8)
    loss2, dZ2 = run(over, y, ids, lp, 0.4, 2.0, in_place=True)
    assert torch.equal(loss, loss2) and torch.equal(dZ, dZ2)


def test_gradient_against_differences():
    """The loss itself, moved along one logit, has the gradient's slope: in 64 bits
    through the formula, which holds the kernel's dZ to its bounds above."""
    T, V, h = 3, 50, 1e-4
    Z = logits(T, V, 1)
    ids, lp = teacher(T, V, 6, 1)
    y = torch.tensor([3, int(ids[1, 0]), -1], device="cuda")
    w = torch.tensor([1.0, 0.5, 2.0], device="cuda")
    _, dZ = run(Z, y, ids, lp, 0.3, 2.0, w)
    f = lambda z: float((ref.distill(z, y, ids, lp, 0.3, 2.0, w)[0] * w.double()).sum())
    for t, v in ((0, 3), (0, int(ids[0, 2])), (1, int(ids[1, 0])), (1, 20), (2, int(ids[2, 5])), (2, 49)):
        step = torch.zeros(T, V, dtype=torch.float64, device="cuda")
        step[t, v] = h
        q = (f(Z.double() + step) - f(Z.double() - step)) / (2 * h)
        # third derivatives below 2: h^2 / 3; the sums' 2^-53 over h; dZ's own bound below 200 roundings of 2
        assert abs(q - float(dZ[t, v])) < 1e-8 + 1e-10 + 400 * ref.U


def test_parts_are_optional():
    T, V = 5, 3000
    Z, y = logits(T, V, 1), targets_of(T, V)
    ids, lp = teacher(T, V, 6, 1)
    loss, dZ = run(Z, y, ids, lp, 0.3, 2.0)
    ws = tl.empty_distill_workspace(T, V)
    only = torch.empty_like(dZ)
    kw = dict(targets=y, teacher_ids=ids, teacher_logp=lp, alpha=0.3, tau=2.0)
    tl.tern_distill(Z, ws, dZ=only, **kw)
    assert torch.equal(only, dZ)
    tl.tern_distill(Z, ws, **kw)                 # nothing asked for
    tl.tern_distill(torch.empty(0, 64, device="cuda"), loss=torch.empty(0, device="cuda"))


def test_far_rows():
    """Offsets past 2^31 elements: the last rows of a matrix of 2.3e9 logits, in place."""
    T, V = 17600, 131072
    tail = logits(3, V, 9, BF)
    y = torch.full((T,), -1, device="cuda")
    y[-3:] = torch.tensor([4, 5, 131071], device="cuda")
    Z = torch.zeros(T, V, dtype=BF, device="cuda")
    Z[-3:] = tail
    loss = torch.empty(T, device="cuda")
    tl.tern_distill(Z, tl.empty_distill_workspace(T, V), targets=y, alpha=1.0, loss=loss, dZ=Z)
    L, le, G, ge = ref.distill(tail, y[-3:], None, None, 1.0, 1.0, None)
    ref.assert_within(loss[-3:], L, le, "loss")
    ref.assert_within(Z[-3:], G, ge + ref.half_step(BF) * (G.abs() + ge), "dZ")
    assert bool((loss[:-3] == 0).all()) and not bool(Z[:4].any())


@pytest.mark.parametrize("T,V", [(300000, 64), (70000, 5003), (66000, 8200), (65600, 33000), (65600, 65608)])
def test_more_rows_than_workgroups(T, V):
    """Workgroups go on to further rows: equal rows but for the last ones, in place."""
    ld = (V + 7) // 8 * 8
    tail = logits(5, V, 2, BF)
    Z = torch.zeros(T, ld, dtype=BF, device="cuda")[:, :V]
    Z[-5:] = tail
    i5, l5 = teacher(5, V, 7, 1)
    ids, lp = i5[:1].repeat(T, 1), l5[:1].repeat(T, 1)
    ids[-5:], lp[-5:] = i5, l5
    y = torch.full((T,), 5, device="cuda")
    y[-5:] = targets_of(5, V)
    w = torch.full((T,), 0.5, device="cuda")
    loss, dZ = run(Z, y, ids, lp, 0.3, 1.5, w, in_place=True)
    L, le, G, ge = ref.distill(tail, y[-5:], i5, l5, 0.3, 1.5, w[-5:])
    ref.assert_within(loss[-5:], L, le, "loss")
    ref.assert_within(dZ[-5:], G, ge + ref.half_step(BF) * (G.abs() + ge), "dZ")
    assert bool((loss[:-5] == loss[0]).all())
    for t in range(0, T - 5, 8192):
        assert bool((dZ[t:min(t + 8192, T - 5)] == dZ[:1]).all())


@pytest.mark.parametrize("T,V", [(3, 131072), (700, 50024), (4000, 256)])
def test_repeats_bitwise(T, V):
    Z, y = logits(T, V, 1, BF), targets_of(T, V)
    ids, lp = teacher(2, V, 9, 1)
    ids, lp = ids.repeat(T, 1)[:T].contiguous(), lp.repeat(T, 1)[:T].contiguous()
    first = run(Z, y, ids, lp, 0.4, 2.0)
    for _ in range(3):
        again = run(Z, y, ids, lp, 0.4, 2.0)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
