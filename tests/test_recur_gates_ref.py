"""The per-element bounds of recur_gates_ref on the CPU: an fp32 evaluation that
multiplies by the smaller gate keeps them, and one that takes w where it is
near 1 does not."""
import numpy as np
import pytest

import recur_gates_ref as gr

LENS = [30, 0, 1, 69]


def excess(d, **how):
    i = {k: v.astype(np.float64) if k != "offsets" else v for k, v in d.items()}
    want, tol = gr.definition(**i), gr.bounds(**i, u=2.0 ** -24)
    with np.errstate(all="ignore"):
        got = gr.evaluate(**d, **how)
        return {n: float(np.nanmax(np.abs(g - w) / t)) for n, g, w, t in zip(gr.NAMES, got, want, tol)}


@pytest.mark.parametrize("what", ["late", "reset", "still"])
@pytest.mark.parametrize("gate", gr.GATES)
def test_bounds_hold_for_the_smaller_gate(gate, what):
    e = excess(gr.inputs(104, 40, LENS, gate, 1, what))
    assert max(e.values()) <= 1, e


@pytest.mark.parametrize("gate", gr.GATES[1:])
def test_bounds_see_a_lost_gradient(gate):
    e = excess(gr.inputs(104, 40, LENS, gate, 1, "late"), backward_from_w=True)
    assert e["dh0"] > 10 and e["dV"] > 10 and e["dK"] > 10, e


@pytest.mark.parametrize("what", ["reset", "still"])
@pytest.mark.parametrize("gate", gr.GATES[1:])
def test_bounds_see_a_lost_state(gate, what):
    e = excess(gr.inputs(104, 40, LENS, gate, 1, what), forward_from_w=True)
    assert e["Y"] > 10 and (what == "still" or e["hT"] > 10), e   # nothing is left at the end of 69 still tokens


def test_definitions_agree():
    """With gates that 64 bits hold from either end, this definition is the other
    tests' one."""
    import recur_ref as ref
    d = gr.inputs(104, 40, LENS, (-4.0, 4.0), 2, "late")
    i = {k: v.astype(np.float64) if k != "offsets" else v for k, v in d.items()}
    dY, dhT = i.pop("dY"), i.pop("dhT")
    want = list(ref.forward(**i)[:2]) + list(ref.backward(**i, dY=dY, dhT=dhT)[:4])
    for a, b in zip(gr.definition(**i, dY=dY, dhT=dhT), want):
        assert np.allclose(a, b, rtol=1e-12, atol=1e-14, equal_nan=True)
