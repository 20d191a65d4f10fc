"""Refusals of the recurrence's entry points and the oracle of its tests, on
the CPU: nothing here launches a kernel."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import recur_ref as ref
import ternary_weight_linear_tern_amd as tl

OK, NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, ALIAS = 0, -1, -2, -4, -5, -6, -7
F32, BF16 = 0, 1
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    return tl.lib()


def fwd(L, **kw):
    a = dict(K=1 << 40, V=2 << 40, R=3 << 40, ld=64, act=BF16, h0=4 << 40, off=5 << 40, S=3, T=4096, C=64, Y=6 << 40,
             ldy=64, hT=7 << 40, states=8 << 40, ws=9 << 40, n=1 << 40)
    a.update(kw)
    p = lambda k: P(a[k])
    return L.tern_recur_fwd(p("K"), p("V"), p("R"), a["ld"], a["act"], p("h0"), p("off"), a["S"], a["T"], a["C"],
                            p("Y"), a["ldy"], p("hT"), p("states"), p("ws"), a["n"], P(0))


def bwd(L, **kw):
    a = dict(K=1 << 40, V=2 << 40, R=3 << 40, ld=64, act=BF16, h0=4 << 40, off=5 << 40, S=3, T=4096, C=64,
             states=8 << 40, dY=10 << 40, lddy=64, dy=F32, dhT=11 << 40, dK=12 << 40, dV=13 << 40, dR=14 << 40,
             ldd=64, dh0=15 << 40, ws=9 << 40, n=1 << 40)
    a.update(kw)
    p = lambda k: P(a[k])
    return L.tern_recur_bwd(p("K"), p("V"), p("R"), a["ld"], a["act"], p("h0"), p("off"), a["S"], a["T"], a["C"],
                            p("states"), p("dY"), a["lddy"], a["dy"], p("dhT"), p("dK"), p("dV"), p("dR"), a["ldd"],
                            p("dh0"), p("ws"), a["n"], P(0))


@pytest.mark.parametrize("call", [fwd, bwd])
def test_rejects_common(L, call):
    assert call(L, T=-1) == SHAPE
    assert call(L, C=60) == SHAPE
    assert call(L, C=-8) == SHAPE
    assert call(L, ld=56) == SHAPE
    assert call(L, ld=68) == SHAPE
    assert call(L, S=-1) == SHAPE
    assert call(L, off=None) == SHAPE            # several sequences need offsets
    assert call(L, act=5) == DTYPE
    assert call(L, K=None) == NULL
    assert call(L, V=None) == NULL
    assert call(L, R=None) == NULL
    assert call(L, ws=None) == WORKSPACE
    assert call(L, n=16) == WORKSPACE
    assert call(L, K=(1 << 40) + 8) == ALIGN
    assert call(L, h0=(4 << 40) + 4) == ALIGN
    assert call(L, off=(5 << 40) + 4) == ALIGN
    assert call(L, ws=(9 << 40) + 8) == ALIGN
    assert call(L, ws=1 << 40) == ALIAS          # workspace over K


def test_fwd_rejects(L):
    assert fwd(L, Y=None) == NULL
    assert fwd(L, ldy=56) == SHAPE
    assert fwd(L, Y=1 << 40) == ALIAS
    assert fwd(L, hT=4 << 40) == ALIAS           # hT over h0
    assert fwd(L, hT=(6 << 40) + 128) == ALIAS   # hT inside Y
    assert fwd(L, states=2 << 40) == ALIAS
    # nothing to do
    assert fwd(L, T=0, S=0, hT=None, K=None, V=None, R=None, Y=None) == OK
    assert fwd(L, T=0, C=0, ld=0, ldy=0) == OK


def test_bwd_rejects(L):
    assert bwd(L, states=None) == NULL
    assert bwd(L, dY=None) == NULL
    assert bwd(L, dK=None) == NULL
    assert bwd(L, dR=None) == NULL
    assert bwd(L, act=F32, dy=BF16) == DTYPE     # dY fp32 or the activations' type
    assert bwd(L, dV=12 << 40) == ALIAS
    assert bwd(L, dK=10 << 40) == ALIAS          # dK over dY
    assert bwd(L, dh0=11 << 40) == ALIAS         # dh0 over dhT
    assert bwd(L, lddy=60) == SHAPE
    assert bwd(L, ldd=60) == SHAPE


def test_column_slices_are_apart(L):
    """Slices of one matrix interleave without sharing an element; a misplaced
    workspace pointer ends the checks (WORKSPACE comes before ALIGN and ALIAS,
    so ALIGN from a later pointer shows the aliasing was not the reason)."""
    w = 3 * 64
    base = 12 << 40
    sl = dict(ldd=w, dR=base, dK=base + 128, dV=base + 256)
    assert bwd(L, **sl, dh0=(15 << 40) + 4) == ALIGN
    assert bwd(L, **{**sl, "dV": base + 192}) == ALIAS                # 32 columns shared with dK
    assert bwd(L, **{**sl, "dV": base + 2 * w * 2 + 128}) == ALIAS    # dK's columns, two rows on
    assert bwd(L, **{**sl, "dV": base + w * 2 - 64}) == ALIAS         # wraps into the next row's dR


def test_step_rejects(L):
    f = L.tern_recur_step
    K, V, R, h, ho, Y = (P(i << 40) for i in range(1, 7))
    assert f(K, V, R, 64, BF16, -1, 64, h, ho, Y, 64, P(0)) == SHAPE
    assert f(K, V, R, 56, BF16, 4, 64, h, ho, Y, 64, P(0)) == SHAPE
    assert f(K, V, R, 64, BF16, 4, 64, h, ho, Y, 60, P(0)) == SHAPE
    assert f(K, V, R, 64, 9, 4, 64, h, ho, Y, 64, P(0)) == DTYPE
    assert f(K, V, R, 64, BF16, 4, 64, None, ho, Y, 64, P(0)) == NULL
    assert f(K, V, R, 64, BF16, 4, 64, h, P((5 << 40) + 4), Y, 64, P(0)) == ALIGN
    assert f(K, V, R, 64, BF16, 4, 64, h, P((4 << 40) + 256), Y, 64, P(0)) == ALIAS   # rows shifted by one
    assert f(K, V, R, 64, BF16, 4, 64, h, h, K, 64, P(0)) == ALIAS
    assert f(None, None, None, 64, BF16, 0, 64, None, None, None, 64, P(0)) == OK


def test_sizes(L):
    assert tl.tern_recur_states_bytes(33, 64) == 3 * 64 * 4
    assert tl.tern_recur_states_bytes(0, 64) == 0
    assert tl.tern_recur_states_bytes(33, 60) == 0
    assert tl.tern_recur_workspace_bytes(-1, 64) == 0
    assert tl.tern_recur_workspace_bytes(16, 64) == 0          # one chunk
    for T, C in ((1000, 64), (16384, 2048), (32768, 4096)):
        assert tl.tern_recur_workspace_bytes(T, C) % 256 == 0 and tl.tern_recur_workspace_bytes(T, C) > 0


def test_cursor(tmp_path):
    """The walk over the offsets stays inside them, whatever they hold."""
    if not shutil.which("g++"):
        pytest.skip("g++ not available")
    exe = str(tmp_path / "cursor_check")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                        os.path.join(os.path.dirname(__file__), "csrc", "cursor_check.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120,
                       env=dict(os.environ, ASAN_OPTIONS="verify_asan_link_order=0"))
    assert r.returncode == 0, r.stdout + r.stderr


def _t(shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def _refused(fn, *a, **k):
    with pytest.raises((TypeError, ValueError)) as e:
        fn(*a, **k)
    assert "GPU" not in str(e.value), f"mismatch not detected: {e.value}"


def test_binding_rejects(L):
    T, C = 40, 64
    K, V, R, Y = (_t((T, C)) for _ in range(4))
    ws, st = _t((1 << 16,), torch.uint8), _t((3, C))
    f = tl.tern_recur_fwd
    _refused(f, K.half(), V, R, Y, ws)
    _refused(f, K, V[:39], R, Y, ws)
    _refused(f, K, V.bfloat16(), R, Y, ws)
    _refused(f, K, V, R, Y.bfloat16(), ws)
    _refused(f, K, V, R, Y, ws, h0=_t((2, C)))
    _refused(f, K, V, R, Y, ws, offsets=_t((3,), torch.int32))
    _refused(f, K, V, R, Y, ws, offsets=_t((3,), torch.int64), h0=_t((1, C)))
    _refused(f, K, V, R, Y, ws, states=_t((2, C)))
    _refused(f, K.t(), V.t(), R.t(), Y.t(), ws)                 # rows not contiguous
    _refused(f, _t((T, 2 * C))[:, :C], V, R, Y, ws)             # two strides among K, V, R
    b = tl.tern_recur_bwd
    g = [_t((T, C)) for _ in range(3)]
    _refused(b, K, V, R, Y.bfloat16(), st, *g, ws)              # a bf16 dY needs bf16 activations
    _refused(b, K, V, R, Y, _t((2, C)), *g, ws)
    _refused(b, K, V, R, Y, st, g[0], g[1].bfloat16(), g[2], ws)
    _refused(b, K, V, R, Y, st, *g, ws, dh0=_t((1, C - 8)))
    _refused(tl.tern_recur_step, K, V, R, _t((T, C), torch.float64), Y)
    _refused(tl.tern_recur_step, K, V, R, _t((T - 1, C)), Y)
    for fn, a in ((f, (K, V, R, Y, ws)), (b, (K, V, R, Y, st, *g, ws)), (tl.tern_recur_step, (K, V, R, Y, Y.clone()))):
        with pytest.raises(ValueError, match="GPU"):
            fn(*a)


def test_oracle_gradient_against_differences():
    """The oracle's own backward against central differences of its forward."""
    rng = np.random.default_rng(3)
    T, C, off = 23, 5, [0, 7, 7, 20]
    i = dict(K=rng.normal(size=(T, C)), V=rng.normal(size=(T, C)), R=rng.normal(size=(T, C)),
             h0=rng.normal(size=(3, C)), offsets=off)
    dY, dhT = rng.normal(size=(T, C)), rng.normal(size=(3, C))
    dY[20:] = 0
    grads = dict(zip(("K", "V", "R", "h0"), ref.backward(**i, dY=dY, dhT=dhT)[:4]))
    loss = lambda d: np.nansum(ref.forward(**d)[0] * dY) + np.sum(ref.forward(**d)[1] * dhT)
    for name, g in grads.items():
        g = np.nan_to_num(g)
        for idx in [tuple(x) for x in rng.integers(0, [g.shape[0], g.shape[1]], (12, 2))]:
            hi, lo = dict(i), dict(i)
            hi[name], lo[name] = i[name].copy(), i[name].copy()
            hi[name][idx] += 1e-5
            lo[name][idx] -= 1e-5
            assert abs((loss(hi) - loss(lo)) / 2e-5 - g[idx]) < 1e-7, (name, idx)
