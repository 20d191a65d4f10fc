"""Rows of a padded batch in the distillation loss: no weight, or neither a target nor an
entry.  Their gradient is 0 whatever they hold, at any length, in place and beside columns that
stay as they are; the other rows are those of the batch without padding."""
import pytest
import torch

import ternary_weight_linear_tern_amd as tl
from test_gpu_distill import run, targets_of, teacher
from test_gpu_logprob import logits

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("T,V", [(9, 1), (9, 7), (9, 64), (9, 513), (2100, 257), (300, 5003), (9, 50021), (150, 65537), (9, 131077),
                                 (2, 400000)])
@pytest.mark.parametrize("dt", [F32, BF])
def test_padding(T, V, dt):
    K = min(V, 9)
    ids, lp = teacher(min(T, 8), V, K, 1)
    n = -(-T // ids.shape[0])
    ids, lp = ids.repeat(n, 1)[:T].contiguous(), lp.repeat(n, 1)[:T].contiguous()
    y, w = targets_of(T, V).clamp(0, V - 1), torch.linspace(0.5, 1.5, T, device="cuda")
    Z = logits(T, V, 2, dt)
    loss, dZ = run(Z, y, ids, lp, 0.3, 2.0, w)
    pad = torch.arange(T, device="cuda") % 3 == 1
    full = pad & (torch.arange(T, device="cuda") % 2 == 0)
    w[pad & ~full] = 0.0
    y[full], ids[full] = -1, -1
    Z[pad] = float("nan")
    got, G = run(Z, y, ids, lp, 0.3, 2.0, w)
    assert torch.equal(got[~pad], loss[~pad]) and torch.equal(G[~pad], dZ[~pad])
    assert bool((got[full] == 0).all()) and bool((G[pad] == 0).all())
    # in place, beside columns that are not the logits'
    wide = torch.full((T, (V + 7) // 8 * 8 + 8), 7.0, dtype=dt, device="cuda")
    wide[:, :V] = Z
    tl.tern_distill(wide[:, :V], tl.empty_distill_workspace(T, V), targets=y, teacher_ids=ids, teacher_logp=lp, alpha=0.3,
                    tau=2.0, dloss=w, dZ=wide[:, :V])
    assert torch.equal(wide[:, :V], G) and bool((wide[:, V:] == 7.0).all())
