"""A projection of a 4-bit layer call is computed as in a call of its own, bit for
bit, whatever else the call holds, and each kernel of the products against the
definition."""
import pytest
import torch

import ternary_weight_linear_tern_amd as tl
from gpu_util import log
from test_gpu_q4 import check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    tl.lib()
    yield
    torch.cuda.synchronize()


# (in, out, group) of the call's projections
COMPANY = {
    "short and long sums": [(512, 512, 32), (8192, 128, 128), (136, 264, 64), (2600, 72, 64), (8, 8, 32)],
    # 1024 column blocks and more: two a wave, four waves, which share out the long
    # projections' runs of rows
    "many columns": [(2048, 8200, 64), (8192, 2048, 128), (4096, 6152, 32), (2600, 40, 64), (16392, 16, 128)],
    "one wide": [(256, 16392, 128), (4104, 24, 64), (200, 8, 32)],
    "nothing beside something": [(0, 64, 32), (1024, 520, 64), (264, 0, 32)],
}


@pytest.mark.parametrize("act,sc,y", [("bf16", "f32", "bf16"), ("bf16", "bf16", "f32"), ("f32", "f32", "f32"),
                                      ("f32", "bf16", "f32")])
@pytest.mark.parametrize("T", [1, 5, 16, 19])
@pytest.mark.parametrize("company", sorted(COMPANY))
def test_company_changes_no_bit(company, T, act, sc, y):
    log(f"q4 layer: {company}, T={T}, {act}, scales {sc}, Y {y}")
    ds = [make(T, n_in, n_out, g, act, sc, y, i) for i, (n_in, n_out, g) in enumerate(COMPANY[company])]
    tl.tern_layer_q4_matvec(ds)
    torch.cuda.synchronize()
    for i, d in enumerate(ds):
        check(d, (company, i))
        alone = torch.full_like(d["Y"], 7.0)
        tl.tern_q4_matvec(d["X"], d["packed"], d["gscale"], d["group"], alone)
        assert torch.equal(d["Y"], alone), (company, i)


@pytest.mark.parametrize("act,sc,y", [("bf16", "f32", "bf16"), ("bf16", "bf16", "f32"), ("f32", "f32", "f32"),
                                      ("f32", "bf16", "f32")])
@pytest.mark.parametrize("T,n_in,n_out", [(1, 264, 16384), (1, 2048, 16400), (3, 136, 16392), (16, 520, 16384),
                                          (17, 1032, 16408), (2, 8, 16392), (1, 16384, 512), (13, 16392, 264)])
def test_wide_and_tall(T, n_in, n_out, act, sc, y):
    """The widths from which a wave takes two column blocks, with an odd number of
    them and a last one half full; the longest sums."""
    for group in (32, 64, 128):
        log(f"q4 T={T} in={n_in} out={n_out} group={group} {act} scale={sc} y={y}")
        d = make(T, n_in, n_out, group, act, sc, y, T + n_in + group)
        tl.tern_q4_matvec(d["X"], d["packed"], d["gscale"], group, d["Y"])
        check(d, group)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("n_in,n_out", [(1032, 520), (4096, 16408)])
def test_a_token_does_not_depend_on_the_others(n_in, n_out, act):
    d = make(19, n_in, n_out, 64, act, "f32", "f32", 1)
    tl.tern_q4_matvec(d["X"], d["packed"], d["gscale"], 64, d["Y"])
    for t in (0, 7, 15, 16, 18):
        Y = torch.full((1, n_out), 7.0, device="cuda")
        tl.tern_q4_matvec(d["X"][t:t + 1].contiguous(), d["packed"], d["gscale"], 64, Y)
        torch.cuda.synchronize()
        assert torch.equal(Y[0], d["Y"][t]), t


def test_layer_call_of_fp32_activations_in_a_graph():
    ds = [make(3, n_in, n_out, 64, "f32", "f32", "f32", i) for i, (n_in, n_out) in
          enumerate([(2048, 8200), (8192, 2048), (1000, 8192)])]
    tl.tern_layer_q4_matvec(ds)
    torch.cuda.synchronize()
    first = [d["Y"].clone() for d in ds]
    s = torch.cuda.Stream()
    tl.tern_graph_begin(s)
    tl.tern_layer_q4_matvec(ds, stream=s)
    g = tl.tern_graph_end(s)
    for rep in range(3):
        for d in ds:
            d["Y"].fill_(7.0)
        torch.cuda.synchronize()
        tl.tern_graph_launch(g, s)
        s.synchronize()
        assert all(torch.equal(d["Y"], f) for d, f in zip(ds, first)), rep
    tl.tern_graph_destroy(g)
