"""A ternary projection served through the 4-bit products: the ternary matrix,
packed once with the projection's scale in every group, gives tern_linear_fwd's
Y.

Both sum the same exact products x * tern, in fp32 and in different orders.
test_gpu_q4's bound holds for the 4-bit sums (terms up to 31 |x s|), and
gpu_util's for the forward's, 2 (n_in + 2) 2^-24 sum |x s|; in bf16 each result is
rounded once more, by at most 2^-8 of itself.
"""
import numpy as np
import pytest
import torch

import ternary_weight_linear_tern_amd as tl
from gpu_util import log

pytestmark = pytest.mark.gpu

THETA = 2


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    tl.lib()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("y", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,n_in,n_out,group", [(1, 512, 2048, 128), (5, 2048, 520, 64), (33, 264, 136, 32)])
def test_served_projection_is_the_layers(T, n_in, n_out, group, y):
    rng = np.random.default_rng(T + n_in)
    q = torch.from_numpy(rng.integers(-7, 8, (n_in, n_out)).astype(np.int8)).cuda()
    scale = torch.from_numpy(rng.uniform(0.01, 0.1, n_out).astype(np.float32)).cuda()
    X = torch.from_numpy(rng.normal(0, 1, (T, n_in))).to(torch.bfloat16).cuda()
    handle, want = tl.empty_packed(n_in, n_out), torch.full((T, n_out), 7.0, dtype=y, device="cuda")
    tl.tern_materialize(q, THETA, handle)
    tl.tern_linear_fwd(X, handle, scale, want)

    tern = (q.sign() * (q.abs() >= THETA)).to(torch.int8)
    packed, got = tl.empty_q4_packed(n_in, n_out), torch.full((T, n_out), 7.0, dtype=y, device="cuda")
    tl.tern_q4_pack(tern, packed)
    gscale = scale.expand(-(-n_in // group), -1).contiguous()
    tl.tern_q4_matvec(X, packed, gscale, group, got)
    torch.cuda.synchronize()
    x, s, t = (a.double().cpu().numpy() for a in (X, scale, tern))
    size = np.sqrt((x * x).sum(1))[:, None] * s
    bound = 8 * 2.0 ** -24 * np.sqrt(n_in) * 31 * size + 2 * (n_in + 2) * 2.0 ** -24 * (np.abs(x) @ np.abs(t)) * s
    a, b = got.double().cpu().numpy(), want.double().cpu().numpy()
    if y == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (np.abs(a) + np.abs(b))
    err = np.abs(a - b)
    log(f"served {T} x {n_in} x {n_out}: worst {float((err / bound).max()):.3f} of its bound")
    assert (err <= bound).all()
