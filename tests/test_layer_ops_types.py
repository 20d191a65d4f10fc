"""Arguments of the operators around the projections that are no tensors: a
TypeError or ValueError that names the call, on the CPU, before anything runs."""
import numpy as np
import pytest
import torch

import ternary_weight_linear_tern_amd as tl

T, C = 40, 64


def _t(shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def calls():
    a = lambda: _t((T, C))
    ws, st = _t((1 << 16,), torch.uint8), _t((3, C))
    off = torch.tensor([0, T])
    q4 = dict(X=_t((2, 136), torch.bfloat16), packed=_t((2 * 2 * 256,), torch.int32), gscale=_t((3, 24)), group=64,
              Y=_t((2, 24)))
    G = _t((64, 128))
    return {
        "tern_recur_fwd": dict(K=a(), V=a(), R=a(), Y=a(), workspace=ws, h0=_t((1, C)), offsets=off, hT=_t((1, C)),
                               states=st),
        "tern_recur_bwd": dict(K=a(), V=a(), R=a(), dY=a(), states=st, dK=a(), dV=a(), dR=a(), workspace=ws,
                               h0=_t((1, C)), offsets=off, dhT=_t((1, C)), dh0=_t((1, C))),
        "tern_recur_step": dict(K=a(), V=a(), R=a(), h=a(), Y=a(), h_out=a()),
        "tern_q4_pack": dict(q=_t((136, 24), torch.int8), packed=q4["packed"]),
        "tern_q4_matvec": q4,
        "tern_orthogonalize": dict(G=G, O=G.bfloat16(), workspace=ws),
    }


CASES = [(fn, k) for fn, a in calls().items() for k in a if k != "group"]


@pytest.mark.parametrize("bad", [np.zeros((T, C), dtype=np.float32), 7])
@pytest.mark.parametrize("fn,name", CASES)
def test_no_tensor(fn, name, bad):
    args = calls()[fn]
    args[name] = bad
    with pytest.raises((TypeError, ValueError), match=fn):
        getattr(tl, fn)(**args)


@pytest.mark.parametrize("fn,name", [c for c in CASES if c[1] not in ("h0", "hT", "offsets", "dhT", "dh0", "h_out",
                                                                      "workspace")
                                     and c != ("tern_recur_fwd", "states")])
def test_required_tensor_missing(fn, name):
    args = calls()[fn]
    args[name] = None
    with pytest.raises((TypeError, ValueError), match=fn):
        getattr(tl, fn)(**args)


@pytest.mark.parametrize("bad", [None, 7, np.zeros((2, 24), dtype=np.float32)])
@pytest.mark.parametrize("name", ["X", "packed", "gscale", "Y"])
def test_layer_q4_no_tensor(name, bad):
    for at in (0, 1):
        ds = [dict(calls()["tern_q4_matvec"], n_in=136, n_out=24) for _ in range(2)]
        ds[at][name] = bad
        with pytest.raises((TypeError, ValueError), match="tern_layer_q4_matvec"):
            tl.tern_layer_q4_matvec(ds)


@pytest.mark.parametrize("bad", [None, 7, np.zeros((64, 128), dtype=np.float32)])
@pytest.mark.parametrize("name", ["G", "O"])
def test_layer_ortho_no_tensor(name, bad):
    for at in (0, 1):
        G = _t((64, 128))
        ms = [dict(G=G, O=G.bfloat16()) for _ in range(2)]
        ms[at][name] = bad
        with pytest.raises((TypeError, ValueError), match="tern_layer_orthogonalize"):
            tl.tern_layer_orthogonalize(ms, _t((1 << 20,), torch.uint8))


def test_errors_name_the_call():
    G = _t((64, 128))
    with pytest.raises(ValueError, match="^tern_orthogonalize"):
        tl.tern_orthogonalize(G, G.bfloat16()[:32], None)
