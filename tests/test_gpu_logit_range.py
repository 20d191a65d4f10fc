"""Logits farther apart than fp32's range, which the scale or the temperature
brings back into it, and temperatures whose square is below fp32's smallest number:
against the formulas in 64 bits."""
import math

import pytest
import torch

import rows_ref as ref
import ternary_weight_linear_tern_amd as tl
from test_gpu_distill import run as distill
from test_gpu_distill import targets_of, teacher
from test_gpu_logprob import check, logits

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def far_logits(T, V, dt, seed=1):
    """Over nearly all of fp32's range: at random, rising, the largest first, few of the largest."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    i = torch.arange(V, device="cuda")
    kinds = [(torch.rand(V, generator=g, device="cuda") * 2 - 1) * 3.3e38, (i / V * 2 - 1) * 3.3e38,
             torch.where(i < V // 2, 3.3e38, -3.3e38), torch.where(i == V - 1, 3.2e38, -3.2e38),
             torch.where(i < V // 3, -3.38e38, torch.randn(V, generator=g, device="cuda"))]
    ld = (V + 7) // 8 * 8
    buf = torch.zeros(T, ld, dtype=dt, device="cuda")
    for t in range(T):
        buf[t, :V] = kinds[t % len(kinds)].to(dt)
    return buf[:, :V]


# fp32's nearest to 1e-38, so that the reference takes the scale that the call takes
TINY = float(torch.tensor(1.2e-38))


@pytest.mark.parametrize("T,V", [(5, 9), (5, 300), (5, 5003), (5, 50021), (5, 131077), (520, 20000), (520, 40000)])
@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("scale", [TINY, float(torch.tensor(1e-30)), 0.25])
def test_log_probabilities(T, V, dt, scale):
    check(far_logits(T, V, dt), k=min(V, 20), scale=scale, tag=f"{T} x {V} {dt} {scale}")


@pytest.mark.parametrize("T,V", [(5, 300), (5, 5003), (5, 131077), (200, 20000), (520, 40000)])
@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("alpha,tau", [(0.0625, 1.0), (0.0625, 0.5), (0.0625, 0.3), (0.0, 1e-3), (0.125, 2.0)])
def test_distillation(T, V, dt, alpha, tau):
    """Targets and a teacher's entry that are nearly the whole range below the largest: finite
    times alpha, and times tau p."""
    Z = far_logits(T, V, dt)
    ids, lp = teacher(T, V, 6, 1)
    ids[:, 0], lp[:, 0] = 1, -3.0
    lp[:, 1:] += 2.0
    y = targets_of(T, V)
    y[::3] = 2
    alpha, tau = float(torch.tensor(alpha)), float(torch.tensor(tau))
    L, le, G, ge = ref.distill(Z, y, ids, lp, alpha, tau, None)
    for grad in (True, False):
        loss, dZ = distill(Z, y, ids, lp, alpha, tau, grad=grad)
        # (what passes fp32's range is infinite)
        over = L > 3.4e38
        assert bool((loss[over].double() > 3.3e38).all())
        ref.assert_within(loss[~over], L[~over], le[~over], f"{T} x {V} {dt} {alpha} {tau} loss")
    loss, dZ = distill(Z, y, ids, lp, alpha, tau)
    ref.assert_within(dZ, G, ge + ref.half_step(dt) * (G.abs() + ge), f"{T} x {V} {dt} {alpha} {tau} dZ")


@pytest.mark.parametrize("tau", [1e-12, 1e-19, 1e-20, 1e-22, 1e-30])
@pytest.mark.parametrize("T,V", [(5, 300), (5, 131077), (300, 5003)])
def test_smallest_temperatures(T, V, tau):
    """tau^2 KL is about tau times a difference of logits, however small tau^2 is."""
    tau = float(torch.tensor(tau))
    Z = logits(T, V, 3)
    ids, lp = teacher(T, V, 6, 2)
    loss, dZ = distill(Z, None, ids, lp, 0.0, tau)
    L, le, G, ge = ref.distill(Z, None, ids, lp, 0.0, tau, None)
    assert bool((L > tau).all()) and math.isfinite(float(L.max()))
    ref.assert_within(loss, L, le, f"{T} x {V} {tau} loss")
    ref.assert_within(dZ, G, ge + ref.half_step(F32) * (G.abs() + ge), f"{T} x {V} {tau} dZ")
