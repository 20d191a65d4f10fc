"""The gated linear recurrence (tern_recur_*) on the GPU against its definition
in 64 bits, element by element, within the bounds recur_ref derives."""
import numpy as np
import pytest
import torch

import recur_ref as ref
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


def lengths_to_offsets(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)


class Case:
    """Inputs on the device (K, V, R column slices of one matrix if grouped)
    and as f64 on the host; outputs filled with a marker."""

    def __init__(self, T, C, act, lens=None, grouped=False, dy="f32", seed=1, gate=(-6.0, 3.0), state=True):
        rng = np.random.default_rng(seed)
        self.T, self.C, self.act = T, C, act
        dt = DT[act]
        self.offsets = None if lens is None else lengths_to_offsets(lens)
        self.S = 1 if lens is None else len(lens)
        bias = rng.uniform(*gate, C)
        host = [rng.normal(0, 1, (T, C)), rng.normal(0, 1, (T, C)) + bias, rng.normal(0, 1, (T, C))]
        self.buf = torch.empty((T, 3 * C), dtype=dt, device="cuda")
        sl = [self.buf[:, i * C:(i + 1) * C] for i in range(3)]
        if not grouped:
            sl = [torch.empty((T, C), dtype=dt, device="cuda") for _ in range(3)]
        for d, x in zip(sl, host):
            d.copy_(torch.from_numpy(x))
        self.R, self.K, self.V = sl
        new = lambda *s, t=torch.float32: torch.full(s, 7.0, dtype=t, device="cuda")
        f = lambda *s: torch.from_numpy(rng.normal(0, 0.5, s).astype(np.float32)).cuda()
        self.h0 = f(self.S, C) if state else None
        self.dhT = f(self.S, C) if state else None
        self.dY = f(T, C).to(DT[dy])
        self.off = None if lens is None else torch.from_numpy(self.offsets).cuda()
        self.Y, self.hT = new(T, C, t=dt), new(self.S, C)
        self.states = tl.empty_recur_states(T, C)
        self.ws = tl.empty_recur_workspace(T, C)
        gb = new(T, 3 * C, t=dt)
        g = [gb[:, i * C:(i + 1) * C] for i in range(3)] if grouped else [new(T, C, t=dt) for _ in range(3)]
        self.dR, self.dK, self.dV = g
        self.dh0 = new(self.S, C)

    def fwd(self, stream=None):
        tl.tern_recur_fwd(self.K, self.V, self.R, self.Y, self.ws, h0=self.h0, offsets=self.off, hT=self.hT,
                          states=self.states, stream=stream)

    def bwd(self, stream=None):
        tl.tern_recur_bwd(self.K, self.V, self.R, self.dY, self.states, self.dK, self.dV, self.dR, self.ws,
                          h0=self.h0, offsets=self.off, dhT=self.dhT, dh0=self.dh0, stream=stream)

    def host(self):
        n = lambda t: t.double().cpu().numpy()
        z = np.zeros((self.S, self.C))
        return dict(K=n(self.K), V=n(self.V), R=n(self.R), h0=z if self.h0 is None else n(self.h0),
                    offsets=self.offsets), n(self.dY), z if self.dhT is None else n(self.dhT)

    def outputs(self):
        return [self.Y, self.hT, self.dK, self.dV, self.dR, self.dh0]

    def check(self):
        torch.cuda.synchronize()
        i, dY, dhT = self.host()
        u = HALF[self.act]
        Y, hT, _, _ = ref.forward(**i)
        tY, th = ref.tol_fwd(**i, u=u)
        want = [Y, hT] + list(ref.backward(**i, dY=dY, dhT=dhT)[:4])
        tols = [tY, th] + list(ref.tol_bwd(**i, dY=dY, dhT=dhT, u=u))
        for name, got, w, tol in zip(("Y", "hT", "dK", "dV", "dR", "dh0"), self.outputs(), want, tols):
            got = got.double().cpu().numpy()
            dead = np.isnan(w)
            assert np.all(got[dead] == 7.0), f"{name}: rows of no sequence were written"
            err = np.where(dead, 0.0, np.abs(got - np.where(dead, 0.0, w)))
            bad = ~(err <= np.broadcast_to(tol, err.shape)) & ~dead
            assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.size} out of bound, first {np.argwhere(bad)[0]}"
            if w.size and not dead.all():
                worst = np.nanmax(err / np.where(dead, 1.0, np.broadcast_to(tol, err.shape)))
                log(f"  {name}: worst error {worst:.3f} of its bound")


SHAPES = [
    # T, C, lengths
    (1, 8, None), (2, 64, None), (15, 136, None), (16, 8, None), (17, 520, None), (33, 64, [10, 0, 23]),
    (0, 64, [0, 0, 0]), (0, 64, None), (64, 128, [16, 16, 16, 16]), (70, 72, [0, 1, 0, 30, 31, 1, 0, 0]),
    (100, 128, [20, 40]),                 # 40 rows behind the last sequence
    (300, 264, [1] * 100 + [0] * 70 + [150, 50]),
    (4100, 24, [4000, 1, 99]),
]


@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("act,dy", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("T,C,lens", SHAPES)
def test_recur_matches_definition(T, C, lens, act, dy, grouped):
    log(f"recur T={T} C={C} {act} dy={dy} grouped={grouped} sequences={None if lens is None else len(lens)}")
    c = Case(T, C, act, lens, grouped, dy, seed=T + C)
    c.fwd()
    c.bwd()
    c.check()


@pytest.mark.parametrize("act,C,lens", [("bf16", 2056, [3000, 0, 17, 5183]), ("f32", 1032, None),
                                        ("bf16", 4096, [1] * 64 + [2000] * 3 + [0])])
def test_recur_many_chunks(act, C, lens):
    """Chunks of several checkpoint blocks, chained through the carry."""
    T = 8200 if lens is None or sum(lens) > 8000 else sum(lens) + 30
    log(f"recur chunks T={T} C={C} {act}")
    c = Case(T, C, act, lens, grouped=act == "bf16", seed=5)
    c.fwd()
    c.bwd()
    c.check()


def test_recur_without_states_and_gradients():
    """No h0, dhT, hT, dh0 and no checkpoints asked for: the same Y."""
    c = Case(200, 64, "f32", [120, 80], state=False)
    c.fwd()
    c.bwd()
    c.check()
    Y = torch.empty_like(c.Y)
    tl.tern_recur_fwd(c.K, c.V, c.R, Y, c.ws, offsets=c.off)
    dK, dV, dR = (torch.empty_like(c.dK) for _ in range(3))
    tl.tern_recur_bwd(c.K, c.V, c.R, c.dY, c.states, dK, dV, dR, c.ws, offsets=c.off)
    torch.cuda.synchronize()
    assert torch.equal(Y, c.Y) and torch.equal(dK, c.dK) and torch.equal(dV, c.dV) and torch.equal(dR, c.dR)


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_recur_saturated_gates(act):
    """Gates far on either side: w to 1 (the state replaced) and to 1e-30."""
    for gate in ((20.0, 60.0), (-70.0, -20.0)):
        c = Case(150, 64, act, [100, 50], gate=gate, seed=3)
        c.fwd()
        c.bwd()
        c.check()


@pytest.mark.parametrize("act,dy", [("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("lens", [[16, 32, 0, 128, 64, 16, 0, 240], [8, 8, 112, 1, 15, 144], [512], [500]])
def test_recur_borders_on_and_off_the_blocks(lens, state, act, dy):
    """Sequences that start or end with a block of 16 rows or a chunk, next to
    ones that do not, with and without states to start from; up to 12 rows behind."""
    log(f"recur borders {lens} state={state} {act}")
    c = Case(512 if sum(lens) > 300 else 300, 72, act, lens, False, dy, seed=sum(lens), state=state)
    c.fwd()
    c.bwd()
    c.check()


@pytest.mark.parametrize("gate", [(-3.0, 3.0), (3.0, 6.0), (22.0, 25.0)])
@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("where", ["V", "K", "h0", "dY", "dhT"])
def test_non_finite_value_lasts_to_its_sequences_end(where, act, gate):
    """However little of a state the gates keep (with gates near 1 the product of
    the kept shares underflows within a few rows), a NaN stays in the state, token
    by token, and the outputs are finite exactly where the definition's are."""
    log(f"recur NaN in {where}, {act}, gates {gate}")
    c = Case(1003, 136, act, [900, 0, 103], gate=gate, seed=5)
    bad = getattr(c, where)
    row = {"V": 37, "K": 37, "h0": 0, "dY": 850, "dhT": 0}[where]
    bad[row, 3] = float("nan")
    bad[row, 135] = float("inf") if where in ("V", "h0") else float("nan")
    c.fwd()
    c.bwd()
    torch.cuda.synchronize()
    i, dY, dhT = c.host()
    with np.errstate(all="ignore"):
        want = list(ref.forward(**i)[:2]) + list(ref.backward(**i, dY=dY, dhT=dhT)[:4])
    for name, got, w in zip(("Y", "hT", "dK", "dV", "dR", "dh0"), c.outputs(), want):
        got = np.isfinite(got.double().cpu().numpy())
        assert np.array_equal(got, np.isfinite(w)), f"{name}: first {np.argwhere(got != np.isfinite(w))[0]}"


@pytest.mark.parametrize("C", [40, 2056])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_recur_sequences_are_apart(bad, C):
    """Non-finite values in some sequences leave the others' outputs as they
    were, bit for bit."""
    lens = [100, 37, 0, 63, 1, 400, 3000, 16]
    T = sum(lens)
    runs = []
    for poison in (False, True):
        c = Case(T, C, "f32", lens, seed=9)
        o = c.offsets
        if poison:
            for s in (1, 4, 6):
                c.K[o[s]] = bad
                c.V[o[s]:o[s + 1]] = bad
                c.h0[s] = bad
                c.dhT[s] = bad
                c.dY[o[s]:o[s + 1]] = bad
        c.fwd()
        c.bwd()
        torch.cuda.synchronize()
        runs.append(c)
    for s in (0, 2, 3, 5, 7):
        rows = slice(int(o[s]), int(o[s + 1]))
        for name in ("Y", "dK", "dV", "dR"):
            assert torch.equal(getattr(runs[0], name)[rows], getattr(runs[1], name)[rows]), (name, s)
        assert torch.equal(runs[0].hT[s], runs[1].hT[s]) and torch.equal(runs[0].dh0[s], runs[1].dh0[s]), s


def test_recur_bad_offsets_stay_inside():
    """Offsets that break the rules: no write outside the outputs' rows, and
    the next good call is right."""
    T, C = 500, 64
    c = Case(T, C, "f32", [100, 200, 200])
    guard = torch.full((T + 64, C), 3.0, device="cuda")
    for off in ([0, 10 ** 12, -5, 500], [400, 300, 200, 100], [-7, -7, -7, -7], [501, 502, 503, 504]):
        o = torch.tensor(off, dtype=torch.int64).cuda()
        tl.tern_recur_fwd(c.K, c.V, c.R, guard[32:32 + T], c.ws, h0=c.h0, offsets=o, hT=c.hT, states=c.states)
        tl.tern_recur_bwd(c.K, c.V, c.R, c.dY, c.states, c.dK, c.dV, c.dR, c.ws, h0=c.h0, offsets=o, dhT=c.dhT,
                          dh0=c.dh0)
        torch.cuda.synchronize()
        assert bool((guard[:32] == 3.0).all()) and bool((guard[32 + T:] == 3.0).all())
    c.fwd()
    c.bwd()
    c.check()


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_recur_step_is_the_recurrence(act):
    """Token by token through tern_recur_step: the forward's outputs bit for
    bit, in place and into another state buffer, on column slices."""
    B, n, C = 5, 16, 136
    c = Case(B * n, C, act, [n] * B, grouped=True, seed=11)
    c.fwd()
    torch.cuda.synchronize()
    h, h2 = c.h0.clone(), torch.empty_like(c.h0)
    Y = torch.empty((B, C), dtype=DT[act], device="cuda")
    rows = torch.from_numpy(c.offsets[:-1]).cuda()
    for t in range(n):
        step = c.buf[rows + t]            # [B, 3 C]
        args = step[:, C:2 * C], step[:, 2 * C:], step[:, :C]
        tl.tern_recur_step(*args, h, Y, h2)
        tl.tern_recur_step(*args, h, Y)
        assert torch.equal(h, h2)
        assert torch.equal(Y, c.Y[rows + t]), t
    # chunks compose exactly only within one checkpoint block; here each
    # sequence is one
    assert torch.allclose(h, c.hT, rtol=0, atol=float(np.max(ref.tol_h(**{k: v for k, v in c.host()[0].items()
                                                                         if k != "R"}))))


@pytest.mark.parametrize("B", [1, 3, 300])
def test_recur_step_definition(B):
    c = Case(B, 72, "f32", [1] * B, seed=B)
    i, _, _ = c.host()
    tl.tern_recur_step(c.K, c.V, c.R, c.h0, c.Y, c.hT)
    torch.cuda.synchronize()
    Y, hT, _, _ = ref.forward(**i)
    tY, th = ref.tol_fwd(**i, u=2.0 ** -24)
    assert (np.abs(c.Y.double().cpu().numpy() - Y) <= tY).all()
    assert (np.abs(c.hT.double().cpu().numpy() - hT) <= th).all()


def test_recur_gradient_against_differences():
    """The kernel's gradients against central differences of the 64-bit
    forward, along random directions of every input.  The difference of step
    e has an error of order e^2 times third derivatives (at most about 1 here,
    times the norm of the direction cubed) and 2^-52 / e of rounding: 1e-6 of
    the terms' size covers both at e = 1e-4."""
    T, C = 60, 24
    c = Case(T, C, "f32", [20, 0, 40], seed=21, gate=(-2.0, 2.0))
    c.fwd()
    c.bwd()
    torch.cuda.synchronize()
    i, dY, dhT = c.host()
    loss = lambda d: float(np.sum(ref.forward(**d)[0] * dY) + np.sum(ref.forward(**d)[1] * dhT))
    rng = np.random.default_rng(0)
    tK, tV, tR, tg = ref.tol_bwd(**i, dY=dY, dhT=dhT, u=2.0 ** -24)
    e = 1e-4
    for name, grad, tol in (("K", c.dK, tK), ("V", c.dV, tV), ("R", c.dR, tR), ("h0", c.dh0, tg)):
        g = grad.double().cpu().numpy()
        for _ in range(4):
            d = rng.choice([-1.0, 1.0], g.shape)
            hi, lo = dict(i), dict(i)
            hi[name], lo[name] = i[name] + e * d, i[name] - e * d
            num = (loss(hi) - loss(lo)) / (2 * e)
            ana = float(np.sum(g * d))
            bound = float(np.sum(np.broadcast_to(tol, g.shape))) + 1e-6 * float(np.sum(np.abs(g)))
            assert abs(num - ana) <= bound, (name, num, ana, bound)


def test_recur_repeats_bitwise_on_other_streams_and_in_graphs():
    """Eager, on a stream of its own, and replayed from a graph with other
    work between the replays and new inputs in the same buffers."""
    c = Case(3000, 2056, "bf16", [1000, 0, 1500, 500], grouped=True, seed=31)
    c.fwd()
    c.bwd()
    torch.cuda.synchronize()
    first = [t.clone() for t in c.outputs()]
    s = torch.cuda.Stream()
    for t in c.outputs():
        t.fill_(7.0)
    torch.cuda.synchronize()
    c.fwd(stream=s)
    c.bwd(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, c.outputs()))
    tl.tern_graph_begin(s)
    c.fwd(stream=s)
    c.bwd(stream=s)
    g = tl.tern_graph_end(s)
    keep = c.buf.clone()
    for rep in range(4):
        c.buf.copy_(keep * (rep + 1) / 4)
        c.fwd()
        c.bwd()
        torch.cuda.synchronize()
        want = [t.clone() for t in c.outputs()]
        for t in c.outputs():
            t.fill_(7.0)
        c.ws.fill_(255)
        torch.cuda.synchronize()
        tl.tern_graph_launch(g, s)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, c.outputs())), rep
    tl.tern_graph_destroy(g)
