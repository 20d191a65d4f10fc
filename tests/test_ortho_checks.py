"""Refusals of the orthogonalisation's entry points and its oracle, on the CPU:
nothing here launches a kernel."""
import ctypes

import pytest
import torch

import ortho_ref as ref
import ternary_weight_linear_tern_amd as tl

OK, NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, ALIAS, VALUE = 0, -1, -2, -4, -5, -6, -7, -9
F32, BF16 = 0, 1
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    return tl.lib()


def call(L, **kw):
    a = dict(G=1 << 40, dt=F32, r=512, c=256, steps=5, O=2 << 40, ws=3 << 40, n=1 << 40)
    a.update(kw)
    return L.tern_orthogonalize(P(a["G"]), a["dt"], a["r"], a["c"], a["steps"], ctypes.c_float(1.0), P(a["O"]),
                                P(a["ws"]), a["n"], P(0))


def test_rejects(L):
    need = tl.tern_orthogonalize_workspace_bytes(512, 256)
    assert need > 0 and need % 256 == 0
    assert call(L, r=-8) == SHAPE
    assert call(L, r=12) == SHAPE
    assert call(L, c=(1 << 20) + 8) == SHAPE
    assert call(L, r=1 << 20, c=1 << 20) == SHAPE
    assert call(L, dt=2) == DTYPE
    assert call(L, steps=0) == VALUE
    assert call(L, steps=65) == VALUE
    assert call(L, G=None) == NULL
    assert call(L, O=None) == NULL
    assert call(L, ws=None) == WORKSPACE
    assert call(L, n=need - 1) == WORKSPACE
    assert call(L, G=(1 << 40) + 8) == ALIGN
    assert call(L, O=(2 << 40) + 8) == ALIGN
    assert call(L, ws=(3 << 40) + 8) == ALIGN
    assert call(L, O=(1 << 40) + 512 * 256 * 4 - 16) == ALIAS     # O over G's end
    assert call(L, O=3 << 40) == ALIAS
    assert call(L, ws=1 << 40) == ALIAS
    assert call(L, r=0, G=None, O=None, ws=None, n=0) == OK


def mats(n):
    a = (tl.TernOrtho * n)()
    for i in range(n):
        a[i].rows, a[i].cols, a[i].gain = 128, 64, 1.0
        a[i].G, a[i].O = (1 << 40) + (i << 30), (2 << 40) + (i << 30)
    return a


def test_layer_rejects(L):
    f = L.tern_layer_orthogonalize
    ws, n = P(3 << 40), 1 << 40
    assert f(mats(1), 0, F32, 5, ws, n, P(0)) == SHAPE
    assert f(mats(9), 9, F32, 5, ws, n, P(0)) == SHAPE
    assert f(None, 2, F32, 5, ws, n, P(0)) == NULL
    a = mats(3)
    a[2].O = a[0].O + 1024
    assert f(a, 3, F32, 5, ws, n, P(0)) == ALIAS
    a = mats(3)
    a[2].O = a[0].G
    assert f(a, 3, F32, 5, ws, n, P(0)) == ALIAS
    a = mats(2)
    assert f(a, 2, F32, 5, ws, tl.tern_layer_orthogonalize_workspace_bytes([(128, 64)] * 2) - 1, P(0)) == WORKSPACE
    assert L.tern_layer_orthogonalize_workspace_bytes(a, 0) == 0
    assert tl.tern_layer_orthogonalize_workspace_bytes([(128, 64)] * 2) == \
        2 * tl.tern_orthogonalize_workspace_bytes(64, 128)


def _t(shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def test_binding_rejects(L):
    G, O, ws = _t((64, 128)), _t((64, 128), torch.bfloat16), _t((1 << 20,), torch.uint8)
    f = tl.tern_orthogonalize

    def refused(fn, *a, **k):
        with pytest.raises((TypeError, ValueError)) as e:
            fn(*a, **k)
        assert "GPU" not in str(e.value), f"mismatch not detected: {e.value}"
    refused(f, G.half(), O, ws)
    refused(f, G, O.float(), ws)
    refused(f, G, O[:32], ws)
    refused(f, G.t(), O.t(), ws)
    refused(f, G[0], O[0], ws)
    d = dict(G=G, O=O)
    refused(tl.tern_layer_orthogonalize, [], ws)
    refused(tl.tern_layer_orthogonalize, [d] * 9, ws)
    refused(tl.tern_layer_orthogonalize, [d, dict(G=G.bfloat16(), O=O.clone())], ws)
    with pytest.raises(ValueError, match="GPU"):
        f(G, O, ws)


def test_oracle_is_the_scalar_polynomial_on_singular_values():
    """The 64-bit oracle against its action on the singular values, for wide,
    tall and square matrices."""
    for r, c in ((20, 33), (33, 20), (24, 24)):
        G = torch.randn(r, c, dtype=torch.float64, generator=torch.Generator().manual_seed(r))
        U, S, V = torch.linalg.svd(G, full_matrices=False)
        x = S / (G.norm() + ref.EPS)
        for _ in range(5):
            x = ref.A * x + ref.B * x ** 3 + ref.C * x ** 5
        assert float((ref.exact(G) - U @ torch.diag(x) @ V).norm()) < 1e-10
        assert float((ref.rounded(G) - ref.exact(G)).norm()) < 0.02 * float(ref.exact(G).norm())
