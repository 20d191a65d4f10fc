"""How near the 4-bit products come to their definition, with activations whose sum
does not cancel among them."""
import numpy as np
import pytest
import torch

import ternary_weight_linear_tern_amd as tl
from gpu_util import log

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    tl.lib()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("mean", [0.0, 3.0])
def test_activations_of_one_sign(act, mean):
    """Activations that a squared or shifted nonlinearity leaves: no sum of the 24 x
    that are taken off again cancels, and the roundings of that part all lie on one
    side of it.  A 32-row chunk starts from the accumulator at -24 sum x (at most
    24 * 32 * max|x| of 32 terms, each rounding by 2^-24 of the sum so far) and adds 32 terms
    up to 31 x: at most 64 roundings (192 for fp32's three terms) of 2^-24 times
    24 sum |x| + sum |q x|, and as many again in all sums of chunks and groups."""
    T, n_in, n_out, group = 4, 2056, 264, 128
    rng = np.random.default_rng(3)
    q = torch.from_numpy(rng.integers(-7, 8, (n_in, n_out)).astype(np.int8)).cuda()
    s = torch.from_numpy(rng.uniform(0.01, 0.1, (-(-n_in // group), n_out)).astype(np.float32)).cuda()
    X = torch.from_numpy(np.abs(rng.normal(mean, 1, (T, n_in)))).to(act).cuda()
    packed, Y = tl.empty_q4_packed(n_in, n_out), torch.full((T, n_out), 7.0, device="cuda")
    tl.tern_q4_pack(q, packed)
    tl.tern_q4_matvec(X, packed, s, group, Y)
    torch.cuda.synchronize()
    x, w = X.double().cpu().numpy(), q.double().cpu().numpy()
    sc = np.repeat(s.double().cpu().numpy(), group, axis=0)[:n_in]
    want = x @ (w * sc)
    terms = 64 if act == torch.bfloat16 else 192
    bound = 2 * terms * 2.0 ** -24 * (np.abs(x) @ ((24 + np.abs(w)) * sc))
    err = np.abs(Y.double().cpu().numpy() - want)
    rel = float(np.linalg.norm(err) / np.linalg.norm(want))
    log(f"  mean {mean} {act}: {rel:.2e} relative L2, worst {float((err / bound).max()):.4f} of its bound")
    assert (err <= bound).all()


@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("law", ["normal", "abs", "shifted", "squared relu"])
def test_no_less_accurate_than_an_fp32_sum(law, group, act):
    """The whole result's error against that of adding up x w in fp32, one after the
    other.  There the k-th sum, about sqrt(k) of a term, rounds by at most 2^-24 of
    itself, evenly between and over the mantissa 0.41 times that rms; over n terms
    0.41 sqrt(sum_k k) = 0.29 n, against the result's sqrt(n): 0.29 sqrt(n) 2^-24."""
    T, n_in, n_out = 8, 2056, 264
    rng = np.random.default_rng(3)
    q = torch.from_numpy(rng.integers(-7, 8, (n_in, n_out)).astype(np.int8)).cuda()
    s = torch.from_numpy(rng.uniform(0.01, 0.1, (-(-n_in // group), n_out)).astype(np.float32)).cuda()
    x = rng.normal(0, 1, (T, n_in))
    x = {"normal": x, "abs": np.abs(x), "shifted": np.abs(x + 3), "squared relu": np.maximum(x, 0) ** 2}[law]
    X = torch.from_numpy(x).to(act).cuda()
    packed, Y = tl.empty_q4_packed(n_in, n_out), torch.full((T, n_out), 7.0, device="cuda")
    tl.tern_q4_pack(q, packed)
    tl.tern_q4_matvec(X, packed, s, group, Y)
    torch.cuda.synchronize()
    want = X.double().cpu().numpy() @ (q.double().cpu().numpy() * np.repeat(s.double().cpu().numpy(), group, axis=0)[:n_in])
    e, bound = float(np.linalg.norm(Y.double().cpu().numpy() - want) / np.linalg.norm(want)), 0.29 * n_in ** 0.5 * 2.0 ** -24
    log(f"  {law}, group {group}, {act}: {e:.2e}, bound {bound:.2e}")
    assert e <= bound
