"""The distillation loss where both parts need exponentials of their own, or one is the
square of the other, in rows that are cut, rows taken in turn, and rows whose logits are so
large that differences are taken first; in place too."""
import pytest
import torch

import rows_ref as ref
from test_gpu_distill import check, run, targets_of, teacher
from test_gpu_logprob import hard_rows, logits

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
INF = float("inf")


def entries(T, V, K, seed):
    ids, lp = teacher(min(T, 16), V, K, seed)
    n = -(-T // ids.shape[0])
    return ids.repeat(n, 1)[:T].contiguous(), lp.repeat(n, 1)[:T].contiguous()


@pytest.mark.parametrize("T,V", [(3, 131077), (3, 400000), (150, 140000), (600, 50021), (600, 70001)])
@pytest.mark.parametrize("tau", [1.5, 2.0, 0.75])
@pytest.mark.parametrize("dt", [F32, BF])
def test_cut_rows_and_rows_in_turn(T, V, tau, dt):
    ids, lp = entries(T, V, 20, 1)
    w = torch.linspace(0.5, 1.5, T, device="cuda")
    check(logits(T, V, 2, dt), targets_of(T, V), ids, lp, 0.3, tau, w, tag=f"{T} x {V} {dt} {tau}")


def large_logits(T, V, dt, seed):
    """Around a value that is large next to their spread, above and below 0; every third row as usual."""
    Z = logits(T, V, seed, dt, size=2.0)
    for t in range(T):
        shift = (0.0, 3e6, -3e6)[t % 3]
        # (steps of bf16 are 16384 there)
        step = 1.0 if dt is F32 else 16384.0
        if shift:
            Z[t] = (torch.round(Z[t].float()) * step + shift).to(dt)
    return Z


@pytest.mark.parametrize("V", [200, 3001, 50021, 131077])
@pytest.mark.parametrize("tau", [1.0, 1.5, 2.0])
@pytest.mark.parametrize("dt", [F32, BF])
def test_large_logits(V, tau, dt):
    for T in (9, 520 if V < 60000 else 140):
        Z = large_logits(T, V, dt, 1)
        ids, lp = entries(T, V, 12, 2)
        y = targets_of(T, V)
        w = torch.linspace(0.5, 1.5, T, device="cuda")
        loss, dZ = check(Z, y, ids, lp, 0.3, tau, w, tag=f"{T} x {V} {dt} {tau}")
        loss2, dZ2 = run(Z, y, ids, lp, 0.3, tau, w, in_place=True)
        assert torch.equal(loss, loss2) and torch.equal(dZ, dZ2)


@pytest.mark.parametrize("V", [64, 1000, 40000, 131072])
@pytest.mark.parametrize("tau", [1.5, 2.0])
@pytest.mark.parametrize("dt", [F32, BF])
def test_hard_rows(V, tau, dt):
    for times in (1, 12):
        Z = hard_rows(V, dt, times)
        Z[(Z < -1e38) & (Z > -INF)] = -1e38              # (losses stay within fp32 at these factors)
        T = Z.shape[0]
        ids, lp = entries(T, V, 8, 2)
        y = targets_of(T, V).clamp(0, V - 1)
        loss, dZ = check(Z, y, ids, lp, 0.5, tau, tag=f"{V} {dt} {tau}")
        assert float(loss[1]) == INF                     # the row in which nothing is allowed
        loss2, dZ2 = run(Z, y, ids, lp, 0.5, tau, in_place=True)
        assert torch.equal(loss, loss2) and torch.equal(dZ.isnan(), dZ2.isnan())
        assert torch.equal(dZ.nan_to_num(), dZ2.nan_to_num())
