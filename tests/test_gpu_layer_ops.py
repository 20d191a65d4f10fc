"""The sequence, serving and update operators in runs, as a layer uses them:
  training   grouped r/k/v projections -> recurrence -> output projection, back
             through the recurrence (whose K, V, R and their gradients are column
             slices of the group's matrices) to the group's weight gradient, and the
             weight gradient orthogonalised;
  serving    4-bit r/k/v products -> one recurrence step -> 4-bit output product,
             token after token, recorded as one graph.
Each run is compared with the same chain in 64 bits, fed the library's inputs.

Bounds.  Every activation between two operators is rounded to bf16, half a step
2^-8 of its value, so two chains that round separately differ by the sum of what
their operators pass on.  The chain is linear or smooth with slopes below 2 at
these sizes; the relative L2 distance is then at most the number of roundings on
the path times 2^-8, taken twice for the gates' slopes.
"""
import numpy as np
import pytest
import torch

import ortho_ref
import recur_ref as ref
import ternary_weight_linear_tern_amd as tl
from gpu_util import log, rel_l2

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    tl.lib()
    yield
    torch.cuda.synchronize()


def f64(t):
    return t.double().cpu().numpy()


def test_training_run():
    T, d, lens = 1000, 264, [300, 0, 700]
    rng = np.random.default_rng(1)
    dev = lambda a, dt=torch.float32: torch.from_numpy(np.ascontiguousarray(a)).to(dt).cuda()
    q = [dev(rng.integers(-7, 8, (d, d)), torch.int8) for _ in range(4)]        # r, k, v, output
    sc = [dev(rng.uniform(0.01, 0.1, d)) for _ in range(4)]
    X, dOut = dev(rng.normal(0, 1, (T, d)), torch.bfloat16), dev(rng.normal(0, 0.01, (T, d)), torch.bfloat16)
    off = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int64).cuda()

    # the group of r, k, v: one matrix of 3 d columns
    qg = torch.empty((d, 3 * d), dtype=torch.int8, device="cuda")
    sg = torch.empty(3 * d, device="cuda")
    tl.tern_group_gather(q[:3], sc[:3], qg, sg)
    pg, po = tl.empty_packed(d, 3 * d), tl.empty_packed(d, d)
    tl.tern_materialize(qg, 2, pg)
    tl.tern_materialize(q[3], 2, po)
    new = lambda *s, dt=torch.float32: torch.empty(s, dtype=dt, device="cuda")
    G, Y, out = new(T, 3 * d, dt=torch.bfloat16), new(T, d, dt=torch.bfloat16), new(T, d)
    rkv = lambda g: (g[:, :d], g[:, d:2 * d], g[:, 2 * d:])
    R, K, V = rkv(G)
    states, ws = tl.empty_recur_states(T, d), tl.empty_recur_workspace(T, d)
    tl.tern_linear_fwd(X, pg, sg, G)
    tl.tern_recur_fwd(K, V, R, Y, ws, offsets=off, states=states)
    tl.tern_linear_fwd(Y, po, sc[3], out)
    dY, dG, dX = new(T, d), new(T, 3 * d, dt=torch.bfloat16), new(T, d)
    dR, dK, dV = rkv(dG)
    gq, sgrad = new(d, 3 * d), new(3 * d)
    tl.tern_linear_bwd_dx(dOut, po, sc[3], dY)
    tl.tern_recur_bwd(K, V, R, dY, states, dK, dV, dR, ws, offsets=off)
    tl.tern_linear_bwd(X, dG, pg, sg, dX, gq, sgrad, tl.empty_workspace(T, d, 3 * d))
    O = new(d, 3 * d, dt=torch.bfloat16)
    tl.tern_orthogonalize(gq, O, tl.empty_ortho_workspace([(d, 3 * d)]), gain=0.1)
    torch.cuda.synchronize()

    tern = [np.sign(x) * (np.abs(x) >= 2) for x in (f64(t) for t in q)]
    W = [t * f64(s) for t, s in zip(tern, sc)]
    x, do = f64(X), f64(dOut)
    r, k, v = (x @ w for w in W[:3])
    i = dict(K=k, V=v, R=r, h0=np.zeros((3, d)), offsets=off.tolist())
    y = ref.forward(**i)[0]
    g = ref.backward(**i, dY=do @ W[3].T, dhT=np.zeros((3, d)))
    dg = np.concatenate([g[2], g[0], g[1]], axis=1)
    wg = np.concatenate(W[:3], axis=1)
    u = 2.0 ** -8
    for name, got, want, rounds in (("out", out, y @ W[3], 2), ("dG", dG, dg, 4), ("dX", dX, dg @ wg.T, 5),
                                    ("gq", gq, x.T @ dg * np.concatenate([f64(s) for s in sc[:3]]), 4)):
        e = rel_l2(f64(got), want)
        log(f"  {name}: relL2 {e:.2e}, bound {2 * rounds * u:.2e}")
        assert e <= 2 * rounds * u, name
    E, fro, _ = ortho_ref.bounds(gq)
    assert float((O.double() / 0.1 - E).norm()) <= fro


@pytest.mark.parametrize("B", [1, 5])
def test_serving_run(B):
    d, n = 512, 6
    rng = np.random.default_rng(B)
    qs = [rng.integers(-7, 8, (d, d)).astype(np.int8) for _ in range(4)]
    ss = [rng.uniform(0.01, 0.1, (d // 64, d)).astype(np.float32) for _ in range(4)]
    X = torch.empty((B, d), dtype=torch.bfloat16, device="cuda")
    r, k, v, y = (torch.empty_like(X) for _ in range(4))
    out, h = torch.empty((B, d), device="cuda"), torch.zeros((B, d), device="cuda")
    projs = []
    for q, s, x, o in zip(qs, ss, (X, X, X, y), (r, k, v, out)):
        pk = tl.empty_q4_packed(d, d)
        tl.tern_q4_pack(torch.from_numpy(q).cuda(), pk)
        projs.append(dict(n_in=d, n_out=d, group=64, packed=pk, gscale=torch.from_numpy(s).cuda(), X=x, Y=o))

    def token(stream):
        tl.tern_layer_q4_matvec(projs[:3], stream=stream)
        tl.tern_recur_step(k, v, r, h, y, stream=stream)
        tl.tern_layer_q4_matvec(projs[3:], stream=stream)

    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    tl.tern_graph_begin(s)
    token(s)
    g = tl.tern_graph_end(s)
    W = [q.astype(np.float64) * np.repeat(sc.astype(np.float64), 64, axis=0) for q, sc in zip(qs, ss)]
    state = np.zeros((B, d))
    eager = torch.zeros_like(h)
    u = 2.0 ** -8
    for t in range(n):
        X.copy_(torch.from_numpy(rng.normal(0, 1, (B, d))))
        before = h.clone()
        torch.cuda.synchronize()
        tl.tern_graph_launch(g, s)
        s.synchronize()
        got, hg = out.clone(), h.clone()
        h.copy_(before)
        token(None)                                  # the same token, call by call
        torch.cuda.synchronize()
        assert torch.equal(got, out) and torch.equal(hg, h), t
        x = f64(X)
        rr, kk, vv = (x @ w for w in W[:3])
        state = state + ref.sig(kk) * (vv - state)
        want = (ref.sig(rr) * state) @ W[3]
        # r, k, v and y round once each; the state keeps what its steps brought in
        assert rel_l2(f64(h), state) <= 2 * 2 * u and rel_l2(f64(got), want) <= 2 * 4 * u, t
    tl.tern_graph_destroy(g)


def test_two_calls_at_once():
    """Two long chains on two streams, each with its own workspace, started
    together: both end, with the results of either alone."""
    T, C = 6000, 2056
    runs = []
    for seed in (1, 2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        N = lambda *s: torch.randn(*s, generator=g, device="cuda")
        d = dict(K=(N(T, C) - 3).bfloat16(), V=N(T, C).bfloat16(), R=N(T, C).bfloat16(), dY=N(T, C) * 0.01)
        e = lambda: torch.empty((T, C), dtype=torch.bfloat16, device="cuda")
        d.update(Y=e(), g=[e(), e(), e()], st=tl.empty_recur_states(T, C), ws=tl.empty_recur_workspace(T, C),
                 s=torch.cuda.Stream())
        runs.append(d)

    def go(d, s):
        tl.tern_recur_fwd(d["K"], d["V"], d["R"], d["Y"], d["ws"], states=d["st"], stream=s)
        tl.tern_recur_bwd(d["K"], d["V"], d["R"], d["dY"], d["st"], *d["g"], d["ws"], stream=s)
    alone = []
    for d in runs:
        go(d, None)
        torch.cuda.synchronize()
        alone.append([t.clone() for t in (d["Y"], *d["g"])])
        for t in (d["Y"], *d["g"]):
            t.fill_(7.0)
    torch.cuda.synchronize()
    for _ in range(3):
        for d in runs:
            go(d, d["s"])
    torch.cuda.synchronize()
    for d, want in zip(runs, alone):
        assert all(torch.equal(a, b) for a, b in zip(want, (d["Y"], *d["g"])))
