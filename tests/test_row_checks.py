"""Refusals of the layer norm, the log probabilities and the distillation loss,
through the C ABI and the binding, and the references of their tests, on the CPU:
nothing here launches a kernel."""
import ctypes
import math

import pytest
import torch

import rows_ref as ref
import ternary_weight_linear_tern_amd as tl

OK, NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, ALIAS, VALUE = 0, -1, -2, -4, -5, -6, -7, -9
F32, BF16 = 0, 1
P = ctypes.c_void_p
A = lambda i: i << 40


@pytest.fixture(scope="module")
def L():
    return tl.lib()


def nfwd(L, **kw):
    a = dict(X=A(1), ldx=64, x=BF16, A=A(2), lda=64, a=F32, w=A(3), b=A(4), eps=1e-5, T=100, C=64, S=A(5), lds=64, Y=A(6),
             ldy=64, y=BF16, st=A(7))
    a.update(kw)
    return L.tern_norm_fwd(P(a["X"]), a["ldx"], a["x"], P(a["A"]), a["lda"], a["a"], P(a["w"]), P(a["b"]), a["eps"],
                           a["T"], a["C"], P(a["S"]), a["lds"], P(a["Y"]), a["ldy"], a["y"], P(a["st"]), P(0))


def nbwd(L, **kw):
    a = dict(S=A(1), lds=64, s=BF16, st=A(2), w=A(3), dY=A(4), lddy=64, dy=F32, dS=A(5), ldds=64, T=100, C=64, dX=A(6),
             lddx=64, dx=F32, dw=A(7), db=A(8), ws=A(9), n=1 << 30)
    a.update(kw)
    return L.tern_norm_bwd(P(a["S"]), a["lds"], a["s"], P(a["st"]), P(a["w"]), P(a["dY"]), a["lddy"], a["dy"],
                           P(a["dS"]), a["ldds"], a["T"], a["C"], P(a["dX"]), a["lddx"], a["dx"], P(a["dw"]), P(a["db"]),
                           P(a["ws"]), a["n"], P(0))


def lprob(L, **kw):
    a = dict(Z=A(1), ld=1008, z=BF16, scale=1.0, T=2, V=1001, tok=A(2), logp=A(3), ent=A(4), lse=A(5), k=5, ids=A(6),
             lp=A(7), ws=A(8), n=1 << 30)
    a.update(kw)
    return L.tern_logprob(P(a["Z"]), a["ld"], a["z"], a["scale"], a["T"], a["V"], P(a["tok"]), P(a["logp"]), P(a["ent"]),
                          P(a["lse"]), a["k"], P(a["ids"]), P(a["lp"]), P(a["ws"]), a["n"], P(0))


def dist(L, **kw):
    a = dict(Z=A(1), ld=1008, z=BF16, T=2, V=1001, y=A(2), K=5, ids=A(3), lp=A(4), alpha=0.5, tau=2.0, dl=A(5), loss=A(6),
             dZ=A(7), lddz=1008, ws=A(8), n=1 << 30)
    a.update(kw)
    return L.tern_distill(P(a["Z"]), a["ld"], a["z"], a["T"], a["V"], P(a["y"]), a["K"], P(a["ids"]), P(a["lp"]),
                          a["alpha"], a["tau"], P(a["dl"]), P(a["loss"]), P(a["dZ"]), a["lddz"], P(a["ws"]), a["n"], P(0))


def test_norm_fwd_rejects(L):
    assert nfwd(L, T=-1) == SHAPE
    assert nfwd(L, C=60) == SHAPE
    assert nfwd(L, C=-8) == SHAPE
    assert nfwd(L, C=(1 << 20) + 8, ldx=1 << 21, ldy=1 << 21, lda=1 << 21, lds=1 << 21) == SHAPE
    for name in ("ldx", "lda", "lds", "ldy"):
        assert nfwd(L, **{name: 56}) == SHAPE
        assert nfwd(L, **{name: 68}) == SHAPE
    assert nfwd(L, x=2) == DTYPE
    assert nfwd(L, a=7) == DTYPE
    assert nfwd(L, y=-1) == DTYPE
    for eps in (0.0, -1e-5, math.inf, math.nan):
        assert nfwd(L, eps=eps) == VALUE
    assert nfwd(L, X=None) == NULL
    assert nfwd(L, Y=None) == NULL
    assert nfwd(L, A=None) == NULL               # S without A
    assert nfwd(L, S=None) == NULL               # A without S
    for name in ("X", "A", "w", "b", "S", "Y"):
        assert nfwd(L, **{name: A(20) + 8}) == ALIGN
    assert nfwd(L, st=A(7) + 4) == ALIGN
    assert nfwd(L, Y=A(1)) == ALIAS
    assert nfwd(L, Y=A(5)) == ALIAS
    assert nfwd(L, S=A(2)) == ALIAS              # the sum over the branch
    assert nfwd(L, S=A(1), lds=128) == ALIAS     # in place only with X's stride
    assert nfwd(L, S=A(1) + 128) == ALIAS        # rows shifted by one
    assert nfwd(L, st=A(6) + 64) == ALIAS
    assert nfwd(L, w=A(6) + 16) == ALIAS
    assert nfwd(L, T=0, X=None, Y=None, A=None, S=None, st=None) == OK
    assert nfwd(L, C=0, ldx=0, ldy=0, lda=0, lds=0) == OK


def test_norm_bwd_rejects(L):
    need = tl.tern_norm_bwd_workspace_bytes(100, 64)
    assert need > 0 and tl.tern_norm_bwd_workspace_bytes(-1, 64) == 0 and tl.tern_norm_bwd_workspace_bytes(5, 60) == 0
    assert nbwd(L, T=-1) == SHAPE
    assert nbwd(L, C=60) == SHAPE
    for name in ("lds", "lddy", "ldds", "lddx"):
        assert nbwd(L, **{name: 56}) == SHAPE
        assert nbwd(L, **{name: 68}) == SHAPE
    assert nbwd(L, s=2) == DTYPE
    assert nbwd(L, dy=3) == DTYPE
    assert nbwd(L, dx=3) == DTYPE
    assert nbwd(L, s=F32, dx=BF16) == DTYPE      # a bf16 gradient of an fp32 stream
    for name in ("S", "st", "dY", "dX"):
        assert nbwd(L, **{name: None}) == NULL
    assert nbwd(L, ws=None) == WORKSPACE
    assert nbwd(L, n=need - 1) == WORKSPACE
    for name in ("S", "w", "dY", "dS", "dX", "dw", "db", "ws"):
        assert nbwd(L, **{name: A(20) + 8}) == ALIGN
    assert nbwd(L, st=A(2) + 4) == ALIGN
    assert nbwd(L, dX=A(4)) == ALIAS
    assert nbwd(L, dX=A(5), lddx=128) == ALIAS   # in place only with dS's stride
    assert nbwd(L, dw=A(8)) == ALIAS
    assert nbwd(L, ws=A(1)) == ALIAS
    assert nbwd(L, db=A(6) + 16) == ALIAS
    assert nbwd(L, C=0, lds=0, lddy=0, ldds=0, lddx=0) == OK
    assert nbwd(L, T=0, S=None, dY=None, dX=None, st=None, dw=None, db=None, ws=None, n=0) == OK


def test_logprob_rejects(L):
    assert lprob(L, T=-1) == SHAPE
    assert lprob(L, V=0) == SHAPE
    assert lprob(L, V=(1 << 20) + 1, ld=1 << 21) == SHAPE
    assert lprob(L, ld=1000) == SHAPE
    assert lprob(L, ld=1004) == SHAPE
    assert lprob(L, z=2) == DTYPE
    for scale in (0.0, -1.0, math.inf, math.nan, 3e38):
        assert lprob(L, scale=scale) == VALUE
    assert lprob(L, k=-1) == VALUE
    assert lprob(L, k=65) == VALUE
    assert lprob(L, V=4, ld=8, k=5) == VALUE
    assert lprob(L, Z=None) == NULL
    assert lprob(L, tok=None) == NULL
    assert lprob(L, logp=None) == NULL
    assert lprob(L, ids=None) == NULL
    assert lprob(L, lp=None) == NULL
    assert lprob(L, Z=A(1) + 8) == ALIGN
    for name in ("tok", "ids"):
        assert lprob(L, **{name: A(20) + 4}) == ALIGN
    for name in ("logp", "ent", "lse", "lp"):
        assert lprob(L, **{name: A(20) + 2}) == ALIGN
    need = tl.tern_logprob_workspace_bytes(2, 1001, 5)
    if need:
        assert lprob(L, ws=None) == WORKSPACE
        assert lprob(L, n=need - 1) == WORKSPACE
    assert lprob(L, ent=A(5)) == ALIAS
    assert lprob(L, lse=A(1) + 2000) == ALIAS
    assert lprob(L, ids=A(2)) == ALIAS
    assert lprob(L, T=0, Z=None, tok=None, logp=None, ids=None, lp=None) == OK
    assert tl.tern_logprob_workspace_bytes(-1, 100, 0) == 0 and tl.tern_logprob_workspace_bytes(1, 0, 0) == 0


def test_distill_rejects(L):
    assert dist(L, T=-1) == SHAPE
    assert dist(L, V=0) == SHAPE
    assert dist(L, ld=1000) == SHAPE
    assert dist(L, lddz=1004) == SHAPE
    assert dist(L, z=4) == DTYPE
    assert dist(L, K=-1) == VALUE
    assert dist(L, K=65) == VALUE
    for alpha in (-0.1, 1.1, math.nan):
        assert dist(L, alpha=alpha) == VALUE
    for tau in (0.0, -1.0, math.inf, math.nan, 1e-39, 1e30):
        assert dist(L, tau=tau) == VALUE
    assert dist(L, Z=None) == NULL
    assert dist(L, ids=None) == NULL
    assert dist(L, lp=None) == NULL
    for name in ("Z", "dZ"):
        assert dist(L, **{name: A(20) + 8}) == ALIGN
    for name in ("y", "ids"):
        assert dist(L, **{name: A(20) + 4}) == ALIGN
    for name in ("lp", "dl", "loss"):
        assert dist(L, **{name: A(20) + 2}) == ALIGN
    need = tl.tern_distill_workspace_bytes(2, 1001)
    if need:
        assert dist(L, ws=None) == WORKSPACE
        assert dist(L, n=need - 1) == WORKSPACE
    assert dist(L, dZ=A(1), lddz=1016) == ALIAS  # in place only with Z's stride
    assert dist(L, dZ=A(1) + 2016) == ALIAS      # rows shifted by one
    assert dist(L, loss=A(5)) == ALIAS
    assert dist(L, dZ=A(1), loss=A(1) + 64) == ALIAS
    assert dist(L, loss=A(2)) == ALIAS
    assert dist(L, T=0, Z=None) == OK
    assert dist(L, loss=None, dZ=None) == OK     # nothing asked for
    assert tl.tern_distill_workspace_bytes(-1, 100) == 0 and tl.tern_distill_workspace_bytes(1, 0) == 0


def test_binding_refuses():
    """By name, before anything reaches the library: tensors of the CPU, other
    shapes and types, arrays that come in pairs."""
    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt)
    X, Y = z(4, 64), z(4, 64)
    with pytest.raises(ValueError, match="on a GPU"):
        tl.tern_norm_fwd(X, Y)
    with pytest.raises(TypeError, match="X must be a tensor"):
        tl.tern_norm_fwd(None, Y)
    with pytest.raises(ValueError, match="two dimensions"):
        tl.tern_norm_fwd(z(64), Y)
    with pytest.raises(ValueError, match="Y has shape"):
        tl.tern_norm_fwd(X, z(4, 72))
    with pytest.raises(TypeError, match="X has dtype"):
        tl.tern_norm_fwd(X.half(), Y)
    with pytest.raises(ValueError, match="together"):
        tl.tern_norm_fwd(X, Y, A=X)
    with pytest.raises(ValueError, match="rows of X must be contiguous"):
        tl.tern_norm_fwd(z(64, 4).t(), Y)
    with pytest.raises(ValueError, match="w has shape"):
        tl.tern_norm_fwd(X, Y, w=z(63))
    with pytest.raises(ValueError, match="stats has shape"):
        tl.tern_norm_bwd(X, z(3, 2), Y, z(4, 64))
    with pytest.raises(TypeError, match="dX has dtype"):
        tl.tern_norm_bwd(X, z(4, 2), Y, z(4, 64, dt=torch.bfloat16))
    with pytest.raises(TypeError, match="dS has dtype"):
        tl.tern_norm_bwd(X, z(4, 2), Y, z(4, 64), dS=z(4, 64, dt=torch.bfloat16))
    with pytest.raises(TypeError, match="tokens has dtype"):
        tl.tern_logprob(X, tokens=z(4, dt=torch.int32), logp=z(4))
    with pytest.raises(ValueError, match="together"):
        tl.tern_logprob(X, top_ids=z(4, 2, dt=torch.int64))
    with pytest.raises(ValueError, match="top_logp has shape"):
        tl.tern_logprob(X, top_ids=z(4, 2, dt=torch.int64), top_logp=z(4, 3))
    with pytest.raises(ValueError, match="on a GPU"):
        tl.tern_logprob(X, lse=z(4))
    with pytest.raises(ValueError, match="together"):
        tl.tern_distill(X, teacher_ids=z(4, 2, dt=torch.int64))
    with pytest.raises(TypeError, match="dZ has dtype"):
        tl.tern_distill(X, dZ=z(4, 64, dt=torch.bfloat16))
    with pytest.raises(ValueError, match="targets has shape"):
        tl.tern_distill(X, targets=z(5, dt=torch.int64))
    with pytest.raises(ValueError, match="on a GPU"):
        tl.tern_distill(X, loss=z(4))


# ---------------------------------------------------------------------------
# the references: against autograd in 64 bits, and planted mistakes
# ---------------------------------------------------------------------------

def test_norm_reference():
    g = torch.Generator().manual_seed(1)
    R = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    S, w, b, dY, dS = R(5, 24).requires_grad_(), R(24).requires_grad_(), R(24).requires_grad_(), R(5, 24), R(5, 24)
    Y = ref.norm_fwd(S, w, b, 1e-5)[0]
    assert torch.allclose(Y, torch.nn.functional.layer_norm(S, (24,), w, b, 1e-5), atol=1e-12)
    ((Y * dY).sum() + (S * dS).sum()).backward()
    mu = S.detach().mean(1, keepdim=True)
    stats = torch.cat([mu, (((S.detach() - mu) ** 2).mean(1, keepdim=True) + 1e-5) ** -0.5], 1)
    dX, dw, db, ex, ew, eb = ref.norm_bwd(S.detach(), stats, w.detach(), dY, dS)
    for got, want in ((dX, S.grad), (dw, w.grad), (db, b.grad)):
        assert torch.allclose(got, want, atol=1e-12)
    # the bounds are tight enough to see what could go wrong: the mean of g left out, xh's, a row of dw
    r, xh = stats[:, 1:], (S.detach() - mu) * stats[:, 1:]
    gg = dY * w.detach()
    for wrong in (dX + r * gg.mean(1, keepdim=True), dX + r * xh * (gg * xh).mean(1, keepdim=True), dX - dS):
        with pytest.raises(AssertionError):
            ref.assert_within(wrong, dX, ex)
    with pytest.raises(AssertionError):
        ref.assert_within(dw - (dY * xh)[2], dw, ew)
    with pytest.raises(AssertionError):
        ref.assert_within(db - dY[4], db, eb)


def test_logprob_reference():
    g = torch.Generator().manual_seed(2)
    Z = torch.randn(6, 100, generator=g)
    Z[1, 50:] = -math.inf
    Z[2] = -math.inf
    Z[3, 7] = math.nan
    tok = torch.tensor([3, 4, 5, 6, -1, 100])
    o = ref.logprob(Z, 0.5, tok, 4)
    L = torch.log_softmax(Z.double() * 0.5, 1)
    for t in (0, 1, 4, 5):
        p = L[t].exp()
        assert torch.allclose(o["entropy"][0][t], -(p[p > 0] * L[t][p > 0]).sum())
        assert torch.allclose(o["lse"][0][t], torch.logsumexp(Z[t].double() * 0.5, 0))
    assert torch.allclose(o["logp"][0][:2], L[[0, 1], [3, 4]]) and o["logp"][0][4:].tolist() == [0.0, 0.0]
    assert o["lse"][0][2] == -math.inf and o["entropy"][0][2] == 0 and bool(torch.isnan(o["entropy"][0][3]))
    assert o["top_ids"][2].tolist() == [0, 1, 2, 3]
    # a lost token of a wide row shows in the bounds
    Z = torch.randn(1, 131072, generator=g)
    v, e = ref.logprob(Z, 1.0, None, 0)["lse"]
    Z[0, int(Z.argmax())] = -math.inf
    with pytest.raises(AssertionError):
        ref.assert_within(ref.logprob(Z, 1.0, None, 0)["lse"][0], v, e)


def test_distill_reference():
    g = torch.Generator().manual_seed(3)
    T, V, K = 5, 40, 6
    Z = torch.randn(T, V, generator=g, dtype=torch.float64).requires_grad_()
    ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(T)])
    lp = torch.log_softmax(torch.randn(T, K + 1, generator=g, dtype=torch.float64), 1)[:, :K]
    ids[1, 4] = ids[1, 2]
    ids[2, 3:] = -1
    y = torch.tensor([1, 2, -1, int(ids[3, 0]), 39])
    w = torch.rand(T, generator=g, dtype=torch.float64)
    alpha, tau = 0.3, 2.0
    want = torch.zeros(T, dtype=torch.float64)
    for t in range(T):
        p = torch.zeros(V, dtype=torch.float64)
        live = ids[t] >= 0
        pk = torch.softmax(lp[t][live], 0)
        q = torch.log_softmax(Z[t] / tau, 0)
        kl = (pk * (pk.log() - q[ids[t][live]])).sum()
        ce = -torch.log_softmax(Z[t], 0)[y[t]] if y[t] >= 0 else 0.0
        want[t] = alpha * ce + (1 - alpha) * tau ** 2 * kl
    (want * w).sum().backward()
    loss, le, G, ge = ref.distill(Z.detach(), y, ids, lp, alpha, tau, w)
    assert torch.allclose(loss, want.detach(), atol=1e-12) and torch.allclose(G, Z.grad, atol=1e-12)
    # the bounds see a teacher's token that is left out, and tau in place of tau^2
    wrong = G.clone()
    wrong[0, ids[0, 5]] += (1 - alpha) * tau * w[0] * torch.softmax(lp[0], 0)[5]
    with pytest.raises(AssertionError):
        ref.assert_within(wrong, G, ge)
    with pytest.raises(AssertionError):
        ref.assert_within(ref.distill(Z.detach(), y, ids, lp, alpha, 1.9999, w)[0], loss, le)
