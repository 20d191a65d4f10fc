"""The Newton-Schulz orthogonalisation (tern_orthogonalize,
tern_layer_orthogonalize) on the GPU against its definition in 64 bits, within
the bounds ortho_ref derives."""
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


def gradient(rows, cols, dt, seed, T=None):
    """X^T . dY * scale over T tokens, the law of the library's inputs."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = T or 2 * max(rows, cols)
    N = lambda *s: torch.randn(*s, generator=g, device="cuda")
    G = N(rows, T) @ (N(T, cols) * 0.01) * (torch.rand(cols, generator=g, device="cuda") * 0.09 + 0.01)
    return G.to(dt)


def run(G, steps=5, gain=1.0):
    O = torch.full(G.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    tl.tern_orthogonalize(G, O, tl.empty_ortho_workspace([G.shape]), steps, gain)
    return O


def check(G, O, steps=5, gain=1.0, tag=""):
    torch.cuda.synchronize()
    E, fro, elem = ref.bounds(G, steps)
    d = O.double() / gain - E
    assert float(d.norm()) <= fro, f"{tag}: {float(d.norm()):.3e} > {fro:.3e}"
    bad = d.abs() > elem
    assert not bool(bad.any()), f"{tag}: {int(bad.sum())} elements, first {bad.nonzero()[0].tolist()}"
    log(f"  {tag}: worst element {float((d.abs() / elem).max()):.2f} of its bound, error {float(d.norm()) / max(float(E.norm()), 1e-30):.4f} relative, bound "
        f"{fro / max(float(E.norm()), 1e-30):.4f}")


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(8, 8), (8, 520), (520, 8), (64, 64), (72, 136), (136, 72), (264, 264),
                                       (1000, 264), (512, 2048), (264, 4104), (1032, 1160)])
def test_ortho_matches_definition(rows, cols, dt):
    log(f"ortho {rows} x {cols} {dt}")
    G = gradient(rows, cols, dt, rows + cols)
    check(G, run(G), tag="5 steps")


@pytest.mark.parametrize("rows,cols", [(2600, 1000), (2048, 8192), (4096, 4096)])
def test_ortho_large_tiles(rows, cols):
    log(f"ortho {rows} x {cols}")
    G = gradient(rows, cols, torch.float32, 3, T=4096)
    check(G, run(G), tag="5 steps")


@pytest.mark.parametrize("steps", [1, 2, 3, 8])
def test_ortho_steps(steps):
    G = gradient(136, 200, torch.float32, steps)
    check(G, run(G, steps), steps, tag=f"{steps} steps")


def test_ortho_of_an_orthogonal_matrix():
    """G = c Q: every singular value follows the scalar polynomial from
    1 / sqrt(m); gain multiplies the result."""
    m = 256
    Q = torch.linalg.qr(torch.randn(m, m, dtype=torch.float64, generator=torch.Generator().manual_seed(1)))[0].cuda()
    for c in (1e-3, 1.0, 1e15):
        G = (Q * c).float().contiguous()
        x = 1.0 / m ** 0.5
        for _ in range(5):
            x = ref.A * x + ref.B * x ** 3 + ref.C * x ** 5
        O = run(G, gain=0.25)
        check(G, O, gain=0.25, tag=f"c={c}")
        assert float((O.double() - 0.25 * x * Q).norm()) <= 0.01 * float((0.25 * x * Q).norm())


def test_ortho_zero_and_rank_one():
    for shape in ((64, 200), (200, 64)):
        assert bool((run(torch.zeros(shape, device="cuda")) == 0).all())
    u, v = torch.randn(72, 1, device="cuda"), torch.randn(1, 264, device="cuda")
    G = u @ v
    check(G, run(G), tag="rank one")


def test_ortho_rows_apart_from_the_padding():
    """Outputs next to their neighbours in one buffer: nothing outside O is
    written, nothing of the workspace's old contents is read."""
    G = gradient(72, 200, torch.float32, 5)
    buf = torch.full((3, 72, 200), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = tl.empty_ortho_workspace([(72, 200)])
    ws.fill_(255)
    tl.tern_orthogonalize(G, buf[1], ws)
    torch.cuda.synchronize()
    assert bool((buf[0] == 7).all()) and bool((buf[2] == 7).all())
    first = buf[1].clone()
    ws.fill_(0)
    tl.tern_orthogonalize(G, buf[1], ws)
    torch.cuda.synchronize()
    assert torch.equal(first, buf[1])
    check(G, buf[1], tag="padding")


@pytest.mark.parametrize("d,f", [(64, 256), (512, 2048), (1024, 2048)])
def test_ortho_layer(d, f):
    """A layer's six gradients in one call, each with its own gain."""
    shapes = [(d, d)] * 4 + [(d, f), (f, d)]
    mats = [dict(G=gradient(r, c, torch.float32, i), O=torch.empty(r, c, dtype=torch.bfloat16, device="cuda"),
                 gain=0.5 + i) for i, (r, c) in enumerate(shapes)]
    tl.tern_layer_orthogonalize(mats, tl.empty_ortho_workspace(shapes))
    for i, x in enumerate(mats):
        check(x["G"], x["O"], gain=x["gain"], tag=f"matrix {i}")


def test_ortho_empty():
    ws = tl.empty_ortho_workspace([(0, 64), (64, 64)])
    G = gradient(64, 64, torch.float32, 1)
    mats = [dict(G=torch.empty(0, 64, device="cuda"), O=torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")),
            dict(G=G, O=torch.empty(64, 64, dtype=torch.bfloat16, device="cuda"))]
    tl.tern_layer_orthogonalize(mats, ws)
    check(G, mats[1]["O"], tag="beside an empty matrix")


def test_ortho_repeats_on_streams_and_in_graphs():
    G = gradient(264, 520, torch.float32, 9)
    O = torch.empty(264, 520, dtype=torch.bfloat16, device="cuda")
    ws = tl.empty_ortho_workspace([G.shape])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    tl.tern_graph_begin(s)
    tl.tern_orthogonalize(G, O, ws, stream=s)
    g = tl.tern_graph_end(s)
    keep = G.clone()
    for rep in range(4):
        G.copy_(keep.roll(rep, 0) + rep)
        want = run(G)
        O.fill_(7.0)
        ws.fill_(255)
        torch.cuda.synchronize()
        tl.tern_graph_launch(g, s)
        s.synchronize()
        assert torch.equal(want, O), rep
    tl.tern_graph_destroy(g)
