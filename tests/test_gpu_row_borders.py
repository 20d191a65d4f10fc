"""Every token of a row counts once, wherever the row is cut: rows of equal logits and
masked tokens, whose sums are exact (tests/rows_count_ref.py), through the log
probabilities and the distillation loss, at lengths off every stride, for numbers of rows
that are taken whole, in segments one after the other, and in parts."""
import pytest
import torch

import rows_count_ref as cr
import rows_ref as ref
from test_gpu_distill import run as distill
from test_gpu_logprob import run as logprob

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
INF = float("inf")
LENGTHS = [1, 7, 9, 63, 257, 511, 513, 1001, 2049, 4099, 8191, 16385, 32771, 50021, 65537, 131077, 262147]


@pytest.mark.parametrize("V", LENGTHS)
@pytest.mark.parametrize("T", [9, 150, 600])
@pytest.mark.parametrize("dt", [F32, BF])
def test_log_probabilities(T, V, dt):
    a = cr.allowed_rows(T, V, V + T, "cuda")
    Z, n = cr.logits_of(a, dt), a.sum(1)
    y = cr.some_allowed(a, 1, 2)[:, 0]
    y[4::9] = V // 3                                     # (allowed or not)
    y[8::9] = V - 1
    L, e = cr.log_count(n)
    k = min(V, 20)
    o = logprob(Z, k=k, tokens=y)
    tag = f"{T} x {V} {dt}"
    ref.assert_within(o["lse"], L, e, tag + " lse")
    ref.assert_within(o["entropy"], L, e, tag + " entropy")
    ref.assert_within(o["logp"], torch.where(a.gather(1, y[:, None])[:, 0], -L, -INF), e, tag + " logp")
    # the allowed tokens by rising index, then the others
    ids = torch.sort((~a).to(torch.uint8), dim=1, stable=True).indices[:, :k]
    assert torch.equal(o["top_ids"], ids), tag
    ref.assert_within(o["top_logp"], torch.where(a.gather(1, ids), -L[:, None], -INF), e[:, None], tag + " top_logp")


@pytest.mark.parametrize("V", LENGTHS)
@pytest.mark.parametrize("T", [9, 150, 600])
@pytest.mark.parametrize("dt", [F32, BF])
def test_distillation(T, V, dt):
    a = cr.allowed_rows(T, V, V + T, "cuda")
    Z, n = cr.logits_of(a, dt), a.sum(1)
    y, ids = cr.some_allowed(a, 1, 2)[:, 0], cr.some_allowed(a, 4, 3)
    lp = torch.full((T, 4), -1.25, device="cuda")
    w = torch.linspace(0.5, 1.5, T, device="cuda")
    for alpha, tau in ((0.5, 2.0), (0.25, 1.5), (0.0, 1.0), (1.0, 1.0)):
        tag = f"{T} x {V} {dt} {alpha} {tau}"
        L, e = cr.loss(n, alpha, tau)
        got, dZ = distill(Z, y, ids, lp, alpha, tau, w)
        ref.assert_within(got, L, e, tag + " loss")
        alone, _ = distill(Z, y, ids, lp, alpha, tau, w, grad=False)
        ref.assert_within(alone, L, e, tag + " loss alone")
        G, ge = cr.gradient(a, y, ids, alpha, tau, w)
        ref.assert_within(dZ, G, ge + ref.half_step(dt) * (G.abs() + ge), tag + " dZ")
        del G, ge, dZ
