"""The norm, the head's projection, the teacher's alternatives and the distillation
loss as a distillation step runs them together: its gradients against autograd in 64
bits, the step recorded as one graph and replayed, two at once, another stream."""
import pytest
import torch

import ternary_weight_linear_tern_amd as tl

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
T, C, V, K, TAU, ALPHA = 70, 264, 1000, 12, 2.0, 0.25


class Step:
    """Residual add and norm, a ternary head, the loss against a teacher, back to
    the stream's gradient and the norm's weights."""

    def __init__(self, seed, act=F32):
        g = torch.Generator(device="cuda").manual_seed(seed)
        N = lambda *s: torch.randn(*s, generator=g, device="cuda")
        new = lambda *s, dt=F32: torch.zeros(*s, dtype=dt, device="cuda")
        self.X, self.A = N(T, C).to(act), N(T, C).to(act)
        self.w, self.b = N(C) * 0.2 + 1, N(C) * 0.1
        self.q = torch.randint(-7, 8, (C, V), generator=g, device="cuda", dtype=torch.int8)
        self.scale = torch.rand(V, generator=g, device="cuda") * 0.1 + 0.02
        self.teacher = (N(T, V) * 2).to(act)
        self.y = torch.randint(-1, V, (T,), generator=g, device="cuda")
        self.dloss = torch.rand(T, generator=g, device="cuda") / T
        self.dres = N(T, C) * 1e-3
        self.S, self.Y, self.stats = new(T, C, dt=act), new(T, C, dt=act), tl.empty_norm_stats(T)
        self.packed = tl.empty_packed(C, V)
        self.Z, self.dZ = new(T, V, dt=act), new(T, V, dt=act)
        self.ids, self.lp = torch.zeros(T, K, dtype=torch.int64, device="cuda"), new(T, K)
        self.logp, self.loss = new(T), new(T)
        self.dY, self.dX, self.dw, self.db = new(T, C), new(T, C), new(C), new(C)
        self.gq, self.sgrad = new(C, V), new(V)
        self.ws = dict(lin=tl.empty_workspace(T, C, V), norm=tl.empty_norm_workspace(T, C),
                       top=tl.empty_logprob_workspace(T, V, K), kd=tl.empty_distill_workspace(T, V))

    def run(self, stream=None):
        s = dict(stream=stream)
        tl.tern_logprob(self.teacher, self.ws["top"], top_ids=self.ids, top_logp=self.lp, scale=1 / TAU, **s)
        tl.tern_norm_fwd(self.X, self.Y, w=self.w, b=self.b, A=self.A, S=self.S, stats=self.stats, **s)
        tl.tern_materialize(self.q, 2, self.packed, **s)
        tl.tern_linear_fwd(self.Y, self.packed, self.scale, self.Z, **s)
        tl.tern_logprob(self.Z, self.ws["top"], tokens=self.y, logp=self.logp, **s)
        tl.tern_distill(self.Z, self.ws["kd"], targets=self.y, teacher_ids=self.ids, teacher_logp=self.lp, alpha=ALPHA,
                        tau=TAU, loss=self.loss, dloss=self.dloss, dZ=self.dZ, **s)
        tl.tern_linear_bwd(self.Y, self.dZ, self.packed, self.scale, self.dY, self.gq, self.sgrad, self.ws["lin"], **s)
        tl.tern_norm_bwd(self.S, self.stats, self.dY, self.dX, self.ws["norm"], w=self.w, dS=self.dres, dw=self.dw,
                         db=self.db, **s)

    def results(self):
        return [x.clone() for x in (self.ids, self.lp, self.S, self.Y, self.stats, self.Z, self.logp, self.loss, self.dZ,
                                    self.dX, self.dw, self.db, self.gq, self.sgrad)]


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


def test_step_against_autograd():
    st = Step(1)
    st.run()
    torch.cuda.synchronize()
    d = lambda x: x.double().requires_grad_()
    S = d(st.X + st.A)
    w, b, scale = d(st.w), d(st.b), d(st.scale)
    tern = (st.q >= 2).double() - (st.q <= -2).double()
    Y = torch.nn.functional.layer_norm(S, (C,), w, b, 1e-5)
    Z = (Y @ tern) * scale
    lt = torch.log_softmax(st.teacher.double() / TAU, 1)
    lp, ids = lt.topk(K, 1)
    assert torch.equal(ids, st.ids)
    p = torch.softmax(lp, 1)
    kl = (p * (p.log() - torch.log_softmax(Z / TAU, 1).gather(1, ids))).sum(1)
    ok = st.y >= 0
    ll = torch.log_softmax(Z, 1).gather(1, st.y.clamp(min=0)[:, None])[:, 0]
    loss = (1 - ALPHA) * TAU ** 2 * kl - torch.where(ok, ALPHA * ll, 0.0)
    ((loss * st.dloss.double()).sum() + (S * st.dres.double()).sum()).backward()
    want = dict(lp=lp, Y=Y, Z=Z, logp=torch.where(ok, ll, 0.0), loss=loss, dX=S.grad, dw=w.grad, db=b.grad,
                sgrad=scale.grad)
    # Every sum here has under 1100 terms of fp32 (2^-24 each step, so 2^-14 at the very worst, two or three
    # of them in a row); a wrong term of any of them is above a thousandth.
    for name, x in want.items():
        assert rel(getattr(st, name), x.detach()) < 2e-5, (name, rel(getattr(st, name), x.detach()))


@pytest.mark.parametrize("act", [F32, BF])
def test_step_as_a_graph(act):
    st = Step(2, act)
    other = Step(3, act)
    stream = torch.cuda.Stream()
    st.run()
    torch.cuda.synchronize()
    want = st.results()
    tl.tern_graph_begin(stream)
    st.run(stream)
    graph = tl.tern_graph_end(stream)
    try:
        for i in range(4):
            for x in (st.ids, st.lp, st.S, st.Y, st.stats, st.Z, st.logp, st.loss, st.dZ, st.dX, st.dw, st.db):
                x.zero_()
            for x in st.ws.values():
                x.fill_(255 if i % 2 else 0)          # a workspace's contents mean nothing
            torch.cuda.synchronize()
            tl.tern_graph_launch(graph, stream)
            other.run()                               # the program's own work in between
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(st.results(), want)), i
        st.X.mul_(0.5)
        st.dloss.mul_(2.0)
        torch.cuda.synchronize()
        tl.tern_graph_launch(graph, stream)
        torch.cuda.synchronize()
        got = st.results()
        st.run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, st.results()))
    finally:
        tl.tern_graph_destroy(graph)


def test_two_at_once():
    """Two steps with their own workspaces on two streams."""
    a, b = Step(4), Step(5)
    a.run()
    b.run()
    torch.cuda.synchronize()
    wa, wb = a.results(), b.results()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        a.run(sa)
        b.run(sb)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a.results(), wa))
    assert all(torch.equal(x, y) for x, y in zip(b.results(), wb))


def test_current_stream_is_taken():
    st = Step(6)
    st.run()
    torch.cuda.synchronize()
    want = st.results()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        st.X.mul_(2.0)
        st.X.mul_(0.5)
        st.run()
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(st.results(), want))
