"""The closed forms of rows_count_ref.py on the CPU: against the general formulas, and
what their bounds see."""
import pytest
import torch

import rows_count_ref as cr
import rows_ref as ref


@pytest.mark.parametrize("V", [1, 9, 50, 520, 2300])
def test_closed_forms(V):
    a = cr.allowed_rows(20, V, 1, "cpu")
    Z, n = cr.logits_of(a, torch.float32), a.sum(1)
    assert bool((n > 0).all())
    y, ids = cr.some_allowed(a, 1, 2)[:, 0], cr.some_allowed(a, 4, 3)
    assert bool(a.gather(1, ids).all()) and bool(a.gather(1, y[:, None]).all())
    o = ref.logprob(Z, 1.0, y, 1)
    L, _ = cr.log_count(n)
    assert torch.allclose(o["lse"][0], L) and torch.allclose(o["entropy"][0], L) and torch.allclose(o["logp"][0], -L)
    w = torch.linspace(0.5, 1.5, 20)
    for alpha, tau in ((0.3, 2.0), (0.0, 1.5), (1.0, 1.0)):
        want, _, G, _ = ref.distill(Z, y, ids, torch.full((20, 4), -1.25), alpha, tau, w)
        assert torch.allclose(want, cr.loss(n, alpha, tau)[0], atol=1e-12)
        assert torch.allclose(G, cr.gradient(a, y, ids, alpha, tau, w)[0], atol=1e-12)


@pytest.mark.parametrize("V", [2, 1000, 16385, 32771, 50021, 131077, 262147])
def test_a_lost_token_shows(V):
    """Any token: lost, or counted twice, in a row that allows all."""
    n = torch.tensor([V])
    for other in (V - 1, V + 1):
        L, e = cr.log_count(n)
        with pytest.raises(AssertionError):
            ref.assert_within(torch.log(torch.tensor([float(other)], dtype=torch.float64)), L, e)
        # every element of the gradient (fp32: half a step more)
        g, eg = torch.tensor([1.0 / V], dtype=torch.float64), torch.tensor([8 * ref.U / V], dtype=torch.float64)
        with pytest.raises(AssertionError):
            ref.assert_within(torch.tensor([1.0 / other], dtype=torch.float64), g, eg + ref.U * g)


@pytest.mark.parametrize("n", [2, 8, 300, 2048, 20000])
def test_a_lost_token_shows_in_the_loss(n):
    for alpha, tau in ((0.5, 2.0), (0.0, 1.5), (1.0, 1.0)):
        want, e = cr.loss(torch.tensor([n]), alpha, tau)
        for other in (n - 1, n + 1):
            got, _ = cr.loss(torch.tensor([other]), alpha, tau)
            with pytest.raises(AssertionError):
                ref.assert_within(got, want, e)
