"""Refusals of the 4-bit products' entry points, on the CPU: nothing here
launches a kernel."""
import ctypes

import pytest
import torch

import ternary_weight_linear_tern_amd as tl

OK, NULL, SHAPE, DTYPE, ALIGN, ALIAS, VALUE = 0, -1, -2, -4, -5, -7, -9
F32, BF16 = 0, 1
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    return tl.lib()


def test_packed_bytes(L):
    assert tl.tern_q4_packed_bytes(0, 64) == 0
    assert tl.tern_q4_packed_bytes(8, 8) == 1024
    assert tl.tern_q4_packed_bytes(4096, 16384) == 4096 * 16384 // 2
    assert tl.tern_q4_packed_bytes(136, 24) == 2 * 2 * 1024
    assert tl.tern_q4_packed_bytes(12, 8) == -1
    assert tl.tern_q4_packed_bytes(-8, 8) == -1


def test_pack_rejects(L):
    f = L.tern_q4_pack
    assert f(P(1 << 40), 12, 8, P(2 << 40), P(0)) == SHAPE
    assert f(P(1 << 40), -8, 8, P(2 << 40), P(0)) == SHAPE
    assert f(None, 8, 8, P(2 << 40), P(0)) == NULL
    assert f(P(1 << 40), 8, 8, None, P(0)) == NULL
    assert f(P(1 << 40), 8, 8, P((2 << 40) + 4), P(0)) == ALIGN
    assert f(P(1 << 40), 64, 64, P((1 << 40) + 1024), P(0)) == ALIAS
    assert f(None, 0, 8, None, P(0)) == OK


def call(L, **kw):
    a = dict(X=1 << 40, act=BF16, pk=2 << 40, s=3 << 40, sd=F32, group=64, T=4, n_in=512, n_out=256, Y=4 << 40, yd=F32)
    a.update(kw)
    return L.tern_q4_matvec(P(a["X"]), a["act"], P(a["pk"]), P(a["s"]), a["sd"], a["group"], a["T"], a["n_in"],
                            a["n_out"], P(a["Y"]), a["yd"], P(0))


def test_matvec_rejects(L):
    assert call(L, T=-1) == SHAPE
    assert call(L, T=1 << 21) == SHAPE
    assert call(L, n_in=12) == SHAPE
    assert call(L, n_out=4) == SHAPE
    assert call(L, group=0) == VALUE
    assert call(L, group=48) == VALUE
    assert call(L, group=256) == VALUE
    assert call(L, act=3) == DTYPE
    assert call(L, sd=3) == DTYPE
    assert call(L, act=F32, yd=BF16) == DTYPE
    for k in ("X", "pk", "s", "Y"):
        assert call(L, **{k: None}) == NULL
        assert call(L, **{k: (9 << 40) + 8}) == ALIGN
    assert call(L, Y=1 << 40) == ALIAS
    assert call(L, Y=(3 << 40) + 64) == ALIAS
    assert call(L, T=0, X=None, Y=None) == OK
    assert call(L, n_out=0, pk=None, s=None, Y=None) == OK


def test_layer_rejects(L):
    def projs(n):
        a = (tl.TernQ4Proj * n)()
        for i in range(n):
            a[i].in_, a[i].out, a[i].group = 512, 256, 64
            for j, f in enumerate(("packed", "gscale", "X", "Y")):
                setattr(a[i], f, (1 << 40) + ((i * 8 + j) << 30))
        return a
    f = L.tern_layer_q4_matvec
    assert f(projs(1), 0, 4, BF16, F32, F32, P(0)) == SHAPE
    assert f(projs(9), 9, 4, BF16, F32, F32, P(0)) == SHAPE
    assert f(None, 2, 4, BF16, F32, F32, P(0)) == NULL
    a = projs(2)
    a[1].Y = a[0].Y + 512
    assert f(a, 2, 4, BF16, F32, F32, P(0)) == ALIAS          # two outputs
    a = projs(2)
    a[0].Y = a[1].X
    assert f(a, 2, 4, BF16, F32, F32, P(0)) == ALIAS          # the other projection's input
    a = projs(2)
    a[1].X = a[0].X                                           # shared: not an alias
    a[1].Y = a[1].Y + 4
    assert f(a, 2, 4, BF16, F32, F32, P(0)) == ALIGN


def _t(shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def _refused(fn, *a, **k):
    with pytest.raises((TypeError, ValueError)) as e:
        fn(*a, **k)
    assert "GPU" not in str(e.value), f"mismatch not detected: {e.value}"


def test_binding_rejects(L):
    X, pk, s, Y = _t((2, 136), torch.bfloat16), _t((2 * 2 * 256,), torch.int32), _t((3, 24)), _t((2, 24))
    f = tl.tern_q4_matvec
    _refused(f, X.half(), pk, s, 64, Y)
    _refused(f, X, pk[:-1], s, 64, Y)
    _refused(f, X, pk.float(), s, 64, Y)
    _refused(f, X, pk, s, 32, Y)                       # 5 groups of 32
    _refused(f, X, pk, s, 0, Y)
    _refused(f, X, pk, s.double(), 64, Y)
    _refused(f, X, pk, s, 64, Y[:1])
    _refused(f, X.float(), pk, s, 64, Y.bfloat16())
    _refused(tl.tern_q4_pack, _t((136, 24)), pk)
    _refused(tl.tern_q4_pack, _t((136, 24), torch.int8), pk[:100])
    d = dict(n_in=136, n_out=24, group=64, packed=pk, gscale=s, X=X, Y=Y)
    g = tl.tern_layer_q4_matvec
    _refused(g, [])
    _refused(g, [d] * 9)
    _refused(g, [d, dict(d, X=X[:1])])
    _refused(g, [d, dict(d, gscale=s.bfloat16())])
    _refused(g, [d, dict(d, Y=Y.bfloat16())])
    _refused(g, [dict(d, packed=pk[:100])])
    for fn, a in ((f, (X, pk, s, 64, Y)), (g, ([d],)), (tl.tern_q4_pack, (_t((136, 24), torch.int8), pk))):
        with pytest.raises(ValueError, match="GPU"):
            fn(*a)
