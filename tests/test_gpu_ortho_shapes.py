"""The orthogonalisation at the sizes where the larger tiles are chosen for each of
its products, on and off their multiples, single and in layers of either type.

Bounds: the whole result within half a step of bf16 of its norm, as
test_gpu_ortho_spectra derives it, and every element within ortho_ref's bound,
whose emulation rounds more than the kernel does."""
import pytest
import torch

import ortho_ref as ref
import ternary_weight_linear_tern_amd as tl
from gpu_util import log
from test_gpu_ortho import gradient

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    tl.lib()
    yield
    torch.cuda.synchronize()


def check(G, O, tag):
    torch.cuda.synchronize()
    E, _, elem = ref.bounds(G)
    d = O.double() - E
    e = float(d.norm() / E.norm())
    log(f"  {tag}: error {e:.5f} relative, worst element {float((d.abs() / elem).max()):.2f} of its bound")
    assert e <= 2.0 ** -8, tag
    assert not bool((d.abs() > elem).any()), tag


# the first product takes tiles of 256 x 256 at 4256 x 5416, the polynomial at 4880 x
# 4880, the last product at 1448 x 8408 (and of 192 x 192 at 928 x 8352), each with rows
# and columns that fill their last tile in part
@pytest.mark.parametrize("rows,cols", [(4256, 5416), (5416, 4256), (4880, 4880), (1448, 8408), (8408, 1448),
                                       (928, 8352), (2080, 2072)])
def test_ortho_large_odd_sizes(rows, cols):
    G = gradient(rows, cols, torch.float32, rows, T=6000)
    O = torch.full((rows, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    tl.tern_orthogonalize(G, O, tl.empty_ortho_workspace([(rows, cols)]))
    check(G, O, f"{rows} x {cols}")


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d,f", [(264, 1032), (1032, 4104), (2048, 8192), (2056, 8200)])
def test_ortho_layer_of_either_type(d, f, dt):
    shapes = [(d, d)] * 4 + [(d, f), (f, d)]
    mats = [dict(G=gradient(r, c, dt, i, T=4096), O=torch.full((r, c), 7.0, dtype=torch.bfloat16, device="cuda"))
            for i, (r, c) in enumerate(shapes)]
    tl.tern_layer_orthogonalize(mats, tl.empty_ortho_workspace(shapes))
    for i in (0, 3, 4, 5):
        check(mats[i]["G"], mats[i]["O"], f"matrix {i} of the layer of {d}, {dt}")


def test_ortho_large_layer_repeats_in_a_graph():
    d, f = 2056, 4104
    shapes = [(d, d)] * 4 + [(d, f), (f, d)]
    mats = [dict(G=gradient(r, c, torch.float32, i, T=4096), O=torch.empty(r, c, dtype=torch.bfloat16, device="cuda"))
            for i, (r, c) in enumerate(shapes)]
    ws = tl.empty_ortho_workspace(shapes)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    tl.tern_graph_begin(s)
    tl.tern_layer_orthogonalize(mats, ws, stream=s)
    g = tl.tern_graph_end(s)
    for rep in range(3):
        for m in mats:
            m["G"].mul_(-1.5)
        ws.fill_(255)
        tl.tern_layer_orthogonalize(mats, ws)
        torch.cuda.synchronize()
        want = [m["O"].clone() for m in mats]
        ws.fill_(255)
        for m in mats:
            m["O"].fill_(7.0)
        torch.cuda.synchronize()
        tl.tern_graph_launch(g, s)
        s.synchronize()
        assert all(torch.equal(m["O"], w) for m, w in zip(mats, want)), rep
    tl.tern_graph_destroy(g)
