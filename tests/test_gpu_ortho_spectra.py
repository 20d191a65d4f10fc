"""The orthogonalisation of matrices whose singular values are not of like size:
decaying spectra, low rank, gradients over few tokens.

Bound.  O is rounded to bf16 once, which moves an element by at most 2^-8 of
itself and so O by at most 2^-8 of its Frobenius norm.  The result before that
rounding is asked to be near enough that the whole distance to the 64-bit
definition stays within this, whatever the kernel holds X in: an rms rounding
error of bf16 is 0.0017 of the norm, which leaves sqrt(2^-16 - 0.0017^2) = 0.0035
for everything else.  (An fp32 evaluation leaves 0.00002 in 5 steps and 0.0027 in 8 steps on
rank one, its worst here.)  With X in fp16 alone the distance is 0.007 to 0.15.
"""
import pytest
import torch

import ortho_ref as ref
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


SPECTRA = {
    "1/k": lambda k: 1.0 / k,
    "1/k^2": lambda k: 1.0 / k ** 2,
    "exp(-k/50)": lambda k: torch.exp(-k / 50),
    "exp(-k/20)": lambda k: torch.exp(-k / 20),
    "rank 64": lambda k: (k <= 64).double(),
    "rank 1": lambda k: (k <= 1).double(),
}


def with_spectrum(rows, cols, law, seed):
    """U diag(law(1), law(2), ...) V^T with random orthogonal U, V, in fp32."""
    g = torch.Generator().manual_seed(seed)
    m = min(rows, cols)
    basis = lambda n: torch.linalg.qr(torch.randn(n, m, dtype=torch.float64, generator=g))[0]
    return ((basis(rows) * law(torch.arange(1, m + 1, dtype=torch.float64))) @ basis(cols).t()).float().cuda()


def check(G, steps, tag):
    O = torch.full(G.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    tl.tern_orthogonalize(G, O, tl.empty_ortho_workspace([G.shape]), steps)
    torch.cuda.synchronize()
    E = ref.exact(G, steps)
    e = float((O.double() - E).norm() / E.norm())
    log(f"  {tag}: relative error {e:.5f}, bound {2.0 ** -8:.5f}")
    assert e <= 2.0 ** -8, (tag, e)


@pytest.mark.parametrize("steps", [5, 8])
@pytest.mark.parametrize("law", sorted(SPECTRA))
def test_decaying_spectra(law, steps):
    check(with_spectrum(512, 1024, SPECTRA[law], 1), steps, f"{law}, {steps} steps")


@pytest.mark.parametrize("law", ["exp(-k/20)", "rank 64"])
@pytest.mark.parametrize("rows,cols", [(264, 264), (1000, 264), (136, 2056), (1544, 1544)])
def test_decaying_spectra_odd_sizes(rows, cols, law):
    check(with_spectrum(rows, cols, SPECTRA[law], 2), 5, f"{law}, {rows} x {cols}")


@pytest.mark.parametrize("rows,cols,T", [(520, 1032, 24), (2048, 2048, 128), (2600, 1000, 100), (4096, 4096, 256)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_gradient_of_few_tokens(rows, cols, T, dt):
    """X^T . dY over fewer tokens than either side: its rank is T (in bf16 its
    rounding fills the other directions 0.002 of the way)."""
    g = torch.Generator(device="cuda").manual_seed(T)
    N = lambda *s: torch.randn(*s, generator=g, device="cuda")
    check((N(rows, T) @ (N(T, cols) * 0.01)).to(dt), 5, f"{rows} x {cols}, {T} tokens, {dt}")


def test_layer_of_mixed_spectra():
    """Matrices of different laws in one call, each as if alone."""
    shapes = [(512, 512), (512, 2048), (2048, 512), (264, 520)]
    laws = ["rank 1", "1/k^2", "exp(-k/20)", "rank 64"]
    mats = [dict(G=with_spectrum(r, c, SPECTRA[l], i), O=torch.empty(r, c, dtype=torch.bfloat16, device="cuda"))
            for i, ((r, c), l) in enumerate(zip(shapes, laws))]
    tl.tern_layer_orthogonalize(mats, tl.empty_ortho_workspace(shapes))
    for m, l in zip(mats, laws):
        E = ref.exact(m["G"])
        e = float((m["O"].double() - E).norm() / E.norm())
        log(f"  {l}: {e:.5f}")
        assert e <= 2.0 ** -8, (l, e)


@pytest.mark.parametrize("norm", [1e-13, 1e-10, 1e-7, 1e-3, 1e30, 1e38])
def test_norms_far_from_one(norm):
    """The 1e-7 beside |G|_F makes X small as G is; large norms are taken out before
    X is rounded."""
    g = torch.Generator(device="cuda").manual_seed(5)
    G = torch.randn(264, 520, generator=g, device="cuda", dtype=torch.float64)
    check((G * (norm / G.norm())).float(), 5, f"norm {norm}")
