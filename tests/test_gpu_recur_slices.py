"""The recurrence with everything a column slice of one matrix: inputs, output and
gradients side by side, rows behind the last sequence left as they were, and
single rows and short batches of slices."""
import pytest
import torch

import ternary_weight_linear_tern_amd as tl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    tl.lib()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,C,lens", [(1, 8, [1]), (2, 72, [1, 1]), (300, 136, [100, 0, 190]), (1000, 264, [1000])])
def test_slices_of_one_matrix_equal_separate_ones(T, C, lens, dt):
    g = torch.Generator(device="cuda").manual_seed(T)
    N = lambda *s: torch.randn(*s, generator=g, device="cuda")
    off = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist()).cuda()
    h0, dhT = N(len(lens), C), N(len(lens), C)
    K, V, R, dY = (N(T, C).to(dt) for _ in range(4))
    new = lambda: torch.full((T, C), 7.0, dtype=dt, device="cuda")
    st, ws = tl.empty_recur_states(T, C), tl.empty_recur_workspace(T, C)

    def run(K, V, R, Y, dY, dK, dV, dR):
        hT, dh0 = torch.empty_like(h0), torch.empty_like(h0)
        tl.tern_recur_fwd(K, V, R, Y, ws, h0=h0, offsets=off, hT=hT, states=st)
        tl.tern_recur_bwd(K, V, R, dY, st, dK, dV, dR, ws, h0=h0, offsets=off, dhT=dhT, dh0=dh0)
        torch.cuda.synchronize()
        return [Y.clone(), hT, dK.clone(), dV.clone(), dR.clone(), dh0]

    want = run(K, V, R, new(), dY, new(), new(), new())
    # R, K, V, Y, dR, dK, dV, dY and a column block that belongs to none of them
    m = torch.full((T, 9 * C), 7.0, dtype=dt, device="cuda")
    s = [m[:, i * C:(i + 1) * C] for i in range(9)]
    for d, x in ((s[0], R), (s[1], K), (s[2], V), (s[7], dY)):
        d.copy_(x)
    got = run(s[1], s[2], s[0], s[3], s[7], s[5], s[6], s[4])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(s[0], R) and torch.equal(s[1], K) and torch.equal(s[2], V) and torch.equal(s[7], dY)
    assert bool((s[8] == 7.0).all())
    for x in (s[3], s[4], s[5], s[6]):
        assert bool((x[int(off[-1]):] == 7.0).all())
    # overlapping by 8 columns: refused
    if C > 8:
        with pytest.raises(tl.TernError):
            tl.tern_recur_fwd(s[1], s[2], s[0], m[:, 3 * C - 8:4 * C - 8], ws, h0=h0, offsets=off)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B", [1, 2, 33])
def test_one_token_of_slices(B, dt):
    C = 72
    g = torch.Generator(device="cuda").manual_seed(B)
    N = lambda *s: torch.randn(*s, generator=g, device="cuda")
    m = N(B, 5 * C).to(dt)
    s = [m[:, i * C:(i + 1) * C] for i in range(5)]
    keep, h = m.clone(), N(B, C)
    Y, out = torch.empty((B, C), dtype=dt, device="cuda"), torch.empty_like(h)
    tl.tern_recur_step(s[1].contiguous(), s[2].contiguous(), s[0].contiguous(), h, Y, out)
    tl.tern_recur_step(s[1], s[2], s[0], h, s[3])
    torch.cuda.synchronize()
    assert torch.equal(h, out) and torch.equal(s[3], Y)
    for i in (0, 1, 2, 4):
        assert torch.equal(s[i], keep[:, i * C:(i + 1) * C])
