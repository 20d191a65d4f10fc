"""Products with 4-bit weights and group scales (tern_q4_*) on the GPU against
the definition in 64 bits, element by element.

The integer codes are exact and so are their products with the activations
(bf16, or the three bf16 terms of an fp32 value).  What rounds are the fp32
sums: each of the at most 6 n_in additions of an output by 2^-24 of the partial
sum, whose terms are at most 31 |x s| (a code is multiplied as 24 + q and the 24
taken off again) and which is then about 31 sqrt(sum_r x^2 s^2).  Roundings of
either sign add up as sqrt(n_in); the bound takes 8 times that,
    8 sqrt(n_in) 2^-24 31 sqrt(sum_r x^2 s^2),
and half a step of Y's type relative to y.  A wrong, missing or misplaced weight
is off by |x s|, thousands of times more.
"""
import numpy as np
import pytest
import torch

import ternary_weight_linear_tern_amd as tl
from gpu_util import log

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    tl.lib()
    yield
    torch.cuda.synchronize()


def make(T, n_in, n_out, group, act, sc, y, seed, lo=-8, hi=8):
    rng = np.random.default_rng(seed)
    q = rng.integers(lo, hi, (n_in, n_out)).astype(np.int8)
    X = torch.from_numpy(rng.normal(0, 1, (T, n_in))).to(DT[act]).cuda()
    s = torch.from_numpy(rng.uniform(0.01, 0.1, (-(-n_in // group), n_out))).to(DT[sc]).cuda()
    pk = tl.empty_q4_packed(n_in, n_out)
    tl.tern_q4_pack(torch.from_numpy(q).cuda(), pk)
    return dict(n_in=n_in, n_out=n_out, group=group, packed=pk, gscale=s, X=X, q=np.clip(q, -8, 7),
                Y=torch.full((T, n_out), 7.0, dtype=DT[y], device="cuda"))


def check(d, what=""):
    torch.cuda.synchronize()
    X = d["X"].double().cpu().numpy()
    s = np.repeat(d["gscale"].double().cpu().numpy(), d["group"], axis=0)[: d["n_in"]]
    want = X @ (d["q"].astype(np.float64) * s)
    size = np.sqrt((X * X) @ (s * s))
    half = 2.0 ** -8 if d["Y"].dtype == torch.bfloat16 else 2.0 ** -24
    bound = 8 * 2.0 ** -24 * np.sqrt(max(d["n_in"], 1)) * 31 * size + half * np.abs(want) + 1e-30
    err = np.abs(d["Y"].double().cpu().numpy() - want)
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size}, first {np.argwhere(bad)[0]}"
    if err.size:
        log(f"  worst error {float((err / bound).max()):.3f} of its bound")


SHAPES = [(1, 8, 8), (1, 32, 16), (1, 40, 24), (2, 128, 128), (1, 136, 264), (16, 512, 72), (17, 200, 1000),
          (5, 1000, 40), (33, 264, 136), (1, 2048, 2048), (3, 4104, 520), (1, 16392, 64), (70, 2056, 48)]


@pytest.mark.parametrize("act,sc,y", [("bf16", "f32", "bf16"), ("bf16", "bf16", "f32"), ("bf16", "f32", "f32"),
                                      ("bf16", "bf16", "bf16"), ("f32", "f32", "f32"), ("f32", "bf16", "f32")])
@pytest.mark.parametrize("T,n_in,n_out", SHAPES)
def test_q4_matches_definition(T, n_in, n_out, act, sc, y):
    for group in (32, 64, 128):
        log(f"q4 T={T} in={n_in} out={n_out} group={group} {act} scale={sc} y={y}")
        d = make(T, n_in, n_out, group, act, sc, y, T + n_in + group)
        tl.tern_q4_matvec(d["X"], d["packed"], d["gscale"], group, d["Y"])
        check(d, group)


def test_q4_pack_clamps():
    d = make(2, 136, 40, 64, "bf16", "f32", "f32", 5, lo=-128, hi=128)
    tl.tern_q4_matvec(d["X"], d["packed"], d["gscale"], 64, d["Y"])
    check(d)


def test_q4_single_weights():
    """One nonzero weight at a time, a unit activation: Y is the scale times
    the code exactly, at every position of a block and its neighbours."""
    n_in, n_out, group = 264, 40, 32
    g = torch.Generator().manual_seed(3)
    rows = torch.randint(0, n_in, (60,), generator=g).tolist() + [0, 7, 8, 31, 32, 127, 128, 255, 256, 263]
    cols = torch.randint(0, n_out, (60,), generator=g).tolist() + [0, 15, 16, 31, 32, 39, 7, 8, 3, 39]
    s = torch.linspace(0.5, 1.5, -(-n_in // group) * n_out).reshape(-1, n_out).cuda()
    X = torch.eye(n_in, dtype=torch.bfloat16, device="cuda")
    for i, (r, c) in enumerate(zip(rows, cols)):
        q = torch.zeros((n_in, n_out), dtype=torch.int8)
        q[r, c] = i % 16 - 8 or 3
        pk = tl.empty_q4_packed(n_in, n_out)
        tl.tern_q4_pack(q.cuda(), pk)
        Y = torch.full((n_in, n_out), 7.0, device="cuda")
        tl.tern_q4_matvec(X, pk, s, group, Y)
        want = torch.zeros_like(Y)
        want[r, c] = float(q[r, c]) * s[r // group, c]
        assert torch.equal(Y, want), (r, c)


def test_q4_wide_fp32_activations():
    """fp32 activations with 24 significant bits and a wide range: the three
    terms lose nothing."""
    d = make(3, 512, 64, 32, "f32", "f32", "f32", 8)
    d["X"].copy_(torch.from_numpy(np.random.default_rng(1).normal(0, 1, (3, 512)) *
                                  10.0 ** np.random.default_rng(2).uniform(-6, 6, (3, 512))))
    tl.tern_q4_matvec(d["X"], d["packed"], d["gscale"], 32, d["Y"])
    check(d)


@pytest.mark.parametrize("T", [1, 4, 20])
def test_q4_layer_equals_single_calls(T):
    """Projections of different sizes and groups in one call, sharing X where
    they can: each as its own call, bit for bit."""
    ds = [make(T, 512, 2048, 32, "bf16", "f32", "bf16", 1), make(T, 2048, 520, 128, "bf16", "f32", "bf16", 2),
          make(T, 512, 8, 64, "bf16", "f32", "bf16", 3), make(T, 8, 512, 64, "bf16", "f32", "bf16", 4)]
    ds[2]["X"] = ds[0]["X"]
    tl.tern_layer_q4_matvec(ds)
    for i, d in enumerate(ds):
        check(d, i)


def test_q4_bad_rows_stay_apart():
    """A row of X with NaN or infinities spoils its own row of Y only."""
    for act in ("bf16", "f32"):
        d = make(6, 264, 72, 64, act, "f32", "f32", 4)
        tl.tern_q4_matvec(d["X"], d["packed"], d["gscale"], 64, d["Y"])
        good = d["Y"].clone()
        d["X"][1, 5], d["X"][4] = float("nan"), float("inf")
        tl.tern_q4_matvec(d["X"], d["packed"], d["gscale"], 64, d["Y"])
        for t in (0, 2, 3, 5):
            assert torch.equal(d["Y"][t], good[t])
        assert bool(d["Y"][1].isnan().all())


def test_q4_empty_sizes():
    X = torch.empty((3, 0), dtype=torch.bfloat16, device="cuda")
    Y = torch.full((3, 16), 7.0, device="cuda")
    tl.tern_q4_matvec(X, tl.empty_q4_packed(0, 16), torch.empty((0, 16), device="cuda"), 32, Y)
    assert bool((Y == 0).all())
    X = torch.empty((0, 32), dtype=torch.bfloat16, device="cuda")
    tl.tern_q4_matvec(X, tl.empty_q4_packed(32, 16), torch.ones((1, 16), device="cuda"), 32,
                      torch.empty((0, 16), device="cuda"))


def test_q4_repeats_on_streams_and_in_graphs():
    ds = [make(2, 2048, 1024, 64, "bf16", "bf16", "f32", i) for i in range(3)]
    tl.tern_layer_q4_matvec(ds)
    torch.cuda.synchronize()
    first = [d["Y"].clone() for d in ds]
    s = torch.cuda.Stream()
    tl.tern_graph_begin(s)
    tl.tern_layer_q4_matvec(ds, stream=s)
    g = tl.tern_graph_end(s)
    for rep in range(4):
        for d in ds:
            d["Y"].fill_(7.0)
        torch.cuda.synchronize()
        tl.tern_graph_launch(g, s)
        s.synchronize()
        assert all(torch.equal(d["Y"], f) for d, f in zip(ds, first)), rep
    tl.tern_graph_destroy(g)
