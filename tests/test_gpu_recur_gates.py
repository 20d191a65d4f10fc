"""The gated linear recurrence on the GPU where its gates are wide open, within
the per-element bounds of recur_gates_ref."""
import numpy as np
import pytest
import torch

import recur_gates_ref as gr
import ternary_weight_linear_tern_amd as tl
from gpu_util import log

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
LENS = [[100, 0, 1, 16, 33, 150], [700, 400], [1, 2, 128, 64, 5]]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    tl.lib()
    yield
    torch.cuda.synchronize()


def run(lens, C, gate, what, act, dy):
    """The library's outputs, the definition's and the bounds, by name."""
    T = sum(lens)
    d = gr.inputs(T, C, lens, gate, T + C, what)
    dev = {k: torch.from_numpy(v).cuda() for k, v in d.items()}
    for k in ("K", "V", "R"):
        dev[k] = dev[k].to(DT[act])
    dev["dY"] = dev["dY"].to(DT[dy])
    new = lambda t: torch.full(t.shape, 7.0, dtype=t.dtype, device="cuda")
    o = dict(Y=new(dev["K"]), hT=new(dev["h0"]), dK=new(dev["K"]), dV=new(dev["K"]), dR=new(dev["K"]),
             dh0=new(dev["h0"]))
    st, ws = tl.empty_recur_states(T, C), tl.empty_recur_workspace(T, C)
    kvr, seq = (dev["K"], dev["V"], dev["R"]), dict(h0=dev["h0"], offsets=dev["offsets"])
    tl.tern_recur_fwd(*kvr, o["Y"], ws, hT=o["hT"], states=st, **seq)
    tl.tern_recur_bwd(*kvr, dev["dY"], st, o["dK"], o["dV"], o["dR"], ws, dhT=dev["dhT"], dh0=o["dh0"], **seq)
    torch.cuda.synchronize()
    i = {k: v.double().cpu().numpy() if k != "offsets" else d[k] for k, v in dev.items()}
    return dev, o, dict(zip(gr.NAMES, gr.definition(**i))), dict(zip(gr.NAMES, gr.bounds(**i, u=HALF[act])))


def check(got, want, tol, names):
    for n in names:
        err = np.abs(got[n].double().cpu().numpy() - want[n])
        bad = ~(err <= tol[n])
        log(f"  {n}: worst error {float(np.max(err / tol[n])):.3f} of its bound")
        assert not bad.any(), f"{n}: {int(bad.sum())} of {bad.size}, first {np.argwhere(bad)[0]}"


ACTS = [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")]


@pytest.mark.parametrize("act,dy", ACTS)
@pytest.mark.parametrize("what", ["late", "reset", "still"])
@pytest.mark.parametrize("gate", gr.GATES)
def test_states_through_open_gates(gate, what, act, dy):
    """What is left of a state, however little, and what replaces it, however
    small next to it."""
    for lens in LENS:
        log(f"recur states, gates {gate}, {what}, {act}, lengths {lens}")
        _, o, want, tol = run(lens, 136, gate, what, act, dy)
        check(o, want, tol, ("Y", "hT"))


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("gate", gr.GATES)
def test_one_token_through_open_gates(gate, act):
    """tern_recur_step: one token of each of 40 sequences."""
    for what in ("reset", "late"):
        d, o, want, tol = run([1] * 40, 72, gate, what, act, "f32")
        tl.tern_recur_step(d["K"], d["V"], d["R"], d["h0"], o["Y"], o["hT"])
        torch.cuda.synchronize()
        check(o, want, tol, ("Y", "hT"))


@pytest.mark.parametrize("act,dy", ACTS)
@pytest.mark.parametrize("what", ["late", "reset", "still"])
@pytest.mark.parametrize("gate", gr.GATES)
def test_gradients_through_open_gates(gate, what, act, dy):
    """What is left of a gradient behind open gates: with 'late', tokens that have
    none of their own receive only that."""
    for lens in LENS:
        log(f"recur gradients, gates {gate}, {what}, {act}, dY {dy}, lengths {lens}")
        _, o, want, tol = run(lens, 136, gate, what, act, dy)
        check(o, want, tol, gr.NAMES)
