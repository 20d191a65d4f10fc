"""Python binding of libtern, the MI355X forward and backward of the SR4
ternary projection, with the recurrence, the 4-bit products and the
orthogonalisation that stand around it in a layer (C ABI in include/tern.h).

The functions below carry the C entry points' names and only marshal
arguments: torch tensors (device memory) become raw pointers, the current HIP
stream becomes the stream handle, and a nonzero status becomes a ``TernError``.
Every computation runs in the HIP kernels of libtern.so; there is no fallback.
If the library has not been built, the first call raises.

Build it in-tree with ``python -m ternary_weight_linear_tern_amd.build``.
"""
from __future__ import annotations

import ctypes
import os
from array import array

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libtern.so")

TERN_F32 = 0
TERN_BF16 = 1

STATUS = {
    0: "TERN_OK", -1: "TERN_ERR_NULL", -2: "TERN_ERR_SHAPE", -3: "TERN_ERR_THETA",
    -4: "TERN_ERR_DTYPE", -5: "TERN_ERR_ALIGN", -6: "TERN_ERR_WORKSPACE", -7: "TERN_ERR_ALIAS",
    -8: "TERN_ERR_HIP", -9: "TERN_ERR_VALUE", -10: "TERN_ERR_SCRATCH",
}

# Every symbol include/tern.h declares: name -> (restype, argtypes)
_vp, _i64, _i32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
SIGNATURES = {
    "tern_packed_words": (_i64, [_i64, _i64]),
    "tern_materialize": (ctypes.c_int, [_vp, _i64, _i64, _i32, _vp, _vp]),
    "tern_linear_fwd": (ctypes.c_int, [_vp, _i32, _vp, _vp, _i64, _i64, _i64, _vp, _i32, _vp]),
    "tern_linear_bwd_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "tern_linear_bwd": (ctypes.c_int, [_vp, _vp, _i32, _vp, _vp, _i64, _i64, _i64, _vp, _i32, _vp,
                                       _vp, _vp, _sz, _vp]),
    "tern_linear_bwd_noalloc": (ctypes.c_int, [_vp, _vp, _i32, _vp, _vp, _i64, _i64, _i64, _vp, _i32, _vp,
                                               _vp, _vp]),
    "tern_linear_bwd_dx": (ctypes.c_int, [_vp, _i32, _vp, _vp, _i64, _i64, _i64, _vp, _i32, _vp]),
    "tern_linear_bwd_dw": (ctypes.c_int, [_vp, _vp, _i32, _vp, _vp, _i64, _i64, _i64, _vp, _vp,
                                          _vp, _sz, _vp]),
    "tern_linear_bwd_dx_acc": (ctypes.c_int, [_vp, _i32, _vp, _vp, _i64, _i64, _i64, _vp, _vp]),
    "tern_linear_bwd_acc_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "tern_linear_bwd_dw_acc": (ctypes.c_int, [_vp, _vp, _i32, _vp, _vp, _i64, _i64, _i64, ctypes.c_float,
                                              _vp, _vp, _vp, _sz, _vp]),
    "tern_group_gather": (ctypes.c_int, [_vp, _vp, _vp, _i32, _i64, _vp, _vp, _vp]),
    "tern_scale_adamw": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i32] + [ctypes.c_float] * 6 + [_vp]),
    "tern_panel_reset": (ctypes.c_int, [_vp, _vp]),
    "tern_panel_add": (ctypes.c_int, [_vp, _i64, _i64, _i32, _i32, _vp, _vp, _vp, _vp]),
    "tern_panel_fractions": (ctypes.c_int, [_vp, _vp]),
    "tern_layer_materialize": (ctypes.c_int, [_vp, _i32, _i32, _vp]),
    "tern_layer_fwd": (ctypes.c_int, [_vp, _i32, _i64, _i32, _i32, _vp]),
    "tern_layer_bwd_dx": (ctypes.c_int, [_vp, _i32, _i64, _i32, _vp]),
    "tern_layer_bwd_dw_workspace_bytes": (_sz, [_vp, _i32, _i64]),
    "tern_layer_bwd_dw": (ctypes.c_int, [_vp, _i32, _i64, _i32, _vp, _sz, _vp]),
    "tern_recur_states_bytes": (_sz, [_i64, _i64]),
    "tern_recur_workspace_bytes": (_sz, [_i64, _i64]),
    "tern_recur_fwd": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i32, _vp, _vp, _i64, _i64, _i64, _vp, _i64, _vp, _vp,
                                      _vp, _sz, _vp]),
    "tern_recur_bwd": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i32, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _i64, _i32,
                                      _vp, _vp, _vp, _vp, _i64, _vp, _vp, _sz, _vp]),
    "tern_recur_step": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i32, _i64, _i64, _vp, _vp, _vp, _i64, _vp]),
    "tern_q4_packed_bytes": (_i64, [_i64, _i64]),
    "tern_q4_pack": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp]),
    "tern_q4_matvec": (ctypes.c_int, [_vp, _i32, _vp, _vp, _i32, _i64, _i64, _i64, _i64, _vp, _i32, _vp]),
    "tern_layer_q4_matvec": (ctypes.c_int, [_vp, _i32, _i64, _i32, _i32, _i32, _vp]),
    "tern_orthogonalize_workspace_bytes": (_sz, [_i64, _i64]),
    "tern_orthogonalize": (ctypes.c_int, [_vp, _i32, _i64, _i64, _i32, ctypes.c_float, _vp, _vp, _sz, _vp]),
    "tern_layer_orthogonalize_workspace_bytes": (_sz, [_vp, _i32]),
    "tern_layer_orthogonalize": (ctypes.c_int, [_vp, _i32, _i32, _i32, _vp, _sz, _vp]),
    "tern_norm_bwd_workspace_bytes": (_sz, [_i64, _i64]),
    "tern_norm_fwd": (ctypes.c_int, [_vp, _i64, _i32, _vp, _i64, _i32, _vp, _vp, ctypes.c_float, _i64, _i64, _vp, _i64,
                                     _vp, _i64, _i32, _vp, _vp]),
    "tern_norm_bwd": (ctypes.c_int, [_vp, _i64, _i32, _vp, _vp, _vp, _i64, _i32, _vp, _i64, _i64, _i64, _vp, _i64, _i32,
                                     _vp, _vp, _vp, _sz, _vp]),
    "tern_logprob_workspace_bytes": (_sz, [_i64, _i64, _i32]),
    "tern_logprob": (ctypes.c_int, [_vp, _i64, _i32, ctypes.c_float, _i64, _i64, _vp, _vp, _vp, _vp, _i32, _vp, _vp,
                                    _vp, _sz, _vp]),
    "tern_distill_workspace_bytes": (_sz, [_i64, _i64]),
    "tern_distill": (ctypes.c_int, [_vp, _i64, _i32, _i64, _i64, _vp, _i32, _vp, _vp, ctypes.c_float, ctypes.c_float,
                                    _vp, _vp, _vp, _i64, _vp, _sz, _vp]),
    "tern_graph_begin": (ctypes.c_int, [_vp]),
    "tern_graph_end": (ctypes.c_int, [_vp, ctypes.POINTER(_vp)]),
    "tern_graph_launch": (ctypes.c_int, [_vp, _vp]),
    "tern_graph_destroy": (ctypes.c_int, [_vp]),
    "tern_status_str": (ctypes.c_char_p, [ctypes.c_int]),
    "tern_version": (ctypes.c_char_p, []),
}


class TernError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {STATUS.get(status, status)} ({tern_status_str(status)})")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libtern.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -m ternary_weight_linear_tern_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------

def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libtern must be contiguous")
    return ctypes.c_void_p(t.data_ptr()) if t.numel() else None


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _act_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return TERN_BF16
    if t.dtype == torch.float32:
        return TERN_F32
    raise TypeError(f"activation dtype must be bfloat16 or float32, got {t.dtype}")


def _check(fn: str, rc: int):
    if rc != 0:
        raise TernError(fn, rc)


_F32 = (torch.float32,)
_ACT = (torch.bfloat16, torch.float32)


def _need(fn: str, name: str, t, shape, dtypes) -> None:
    """t must be a tensor of this shape and one of these dtypes."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{fn}: {name} must be a tensor")
    if tuple(t.shape) != tuple(int(x) for x in shape):
        raise ValueError(f"{fn}: {name} has shape {tuple(t.shape)}, expected {tuple(int(x) for x in shape)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{fn}: {name} has dtype {t.dtype}, expected one of {dtypes}")


def _need_bytes(fn: str, name: str, t, nbytes: int) -> None:
    """t must hold at least nbytes (a packed handle, a workspace, a panel)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{fn}: {name} must be a tensor")
    have = t.numel() * t.element_size()
    if have < nbytes:
        raise ValueError(f"{fn}: {name} holds {have} bytes, needs {nbytes}")


def _need_packed(fn: str, t, n_in: int, n_out: int) -> None:
    if not isinstance(t, torch.Tensor) or t.dtype not in (torch.int32, torch.uint32):
        raise TypeError(f"{fn}: tern_packed must be an int32 tensor (see empty_packed)")
    _need_bytes(fn, "tern_packed", t, 4 * max(tern_packed_words(n_in, n_out), 0))


def _need_device(fn: str, *ts) -> None:
    """Every tensor passed to the library lives on one GPU."""
    devs = {t.device for t in ts if isinstance(t, torch.Tensor)}
    if any(d.type != "cuda" for d in devs):
        raise ValueError(f"{fn}: every tensor must be on a GPU (got {sorted(map(str, devs))})")
    if len(devs) > 1:
        raise ValueError(f"{fn}: tensors on several devices {sorted(map(str, devs))}")


# ---------------------------------------------------------------------------
# entry points (same names as the C ABI)
# ---------------------------------------------------------------------------

def tern_status_str(status: int) -> str:
    return lib().tern_status_str(int(status)).decode()


def tern_version() -> str:
    return lib().tern_version().decode()


def tern_packed_words(n_in: int, n_out: int) -> int:
    return int(lib().tern_packed_words(n_in, n_out))


def tern_linear_bwd_workspace_bytes(T: int, n_in: int, n_out: int) -> int:
    return int(lib().tern_linear_bwd_workspace_bytes(T, n_in, n_out))


def tern_materialize(q: torch.Tensor, theta: int, tern_packed: torch.Tensor, stream=None) -> None:
    """q int8 [in, out] -> packed ternary handle (see empty_packed)."""
    fn = "tern_materialize"
    if q.dim() != 2:
        raise ValueError(f"{fn}: q must be [in, out]")
    n_in, n_out = q.shape
    _need(fn, "q", q, (n_in, n_out), (torch.int8,))
    _need_packed(fn, tern_packed, n_in, n_out)
    _need_device(fn, q, tern_packed)
    rc = lib().tern_materialize(_ptr(q), n_in, n_out, int(theta), _ptr(tern_packed), _stream(stream))
    _check("tern_materialize", rc)


def tern_linear_fwd(X: torch.Tensor, tern_packed: torch.Tensor, scale: torch.Tensor, Y: torch.Tensor,
                    stream=None) -> None:
    """Y [T, out] (fp32 or bf16) = X [T, in] . (scale * tern)."""
    fn = "tern_linear_fwd"
    if X.dim() != 2 or scale.dim() != 1:
        raise ValueError(f"{fn}: X must be [T, in] and scale [out]")
    T, n_in = X.shape
    n_out = scale.shape[0]
    _need(fn, "X", X, (T, n_in), _ACT)
    _need(fn, "scale", scale, (n_out,), _F32)
    _need(fn, "Y", Y, (T, n_out), (torch.float32, X.dtype))
    _need_packed(fn, tern_packed, n_in, n_out)
    _need_device(fn, X, tern_packed, scale, Y)
    rc = lib().tern_linear_fwd(_ptr(X), _act_code(X), _ptr(tern_packed), _ptr(scale), T, n_in, n_out,
                               _ptr(Y), _act_code(Y), _stream(stream))
    _check("tern_linear_fwd", rc)


def _bwd_dw_checks(fn, X, dY, tern_packed, scale, gq, sgrad, workspace):
    if X.dim() != 2 or scale.dim() != 1:
        raise ValueError(f"{fn}: X must be [T, in] and scale [out]")
    T, n_in = X.shape
    n_out = scale.shape[0]
    _need(fn, "X", X, (T, n_in), _ACT)
    _need(fn, "dY", dY, (T, n_out), (X.dtype,))
    _need(fn, "scale", scale, (n_out,), _F32)
    _need(fn, "gq", gq, (n_in, n_out), _F32)
    _need(fn, "sgrad", sgrad, (n_out,), _F32)
    _need_packed(fn, tern_packed, n_in, n_out)
    if workspace is not None:
        _need_bytes(fn, "workspace", workspace, 0)
    return T, n_in, n_out


def tern_linear_bwd(X, dY, tern_packed, scale, dX, gq, sgrad, workspace, stream=None) -> None:
    fn = "tern_linear_bwd"
    T, n_in, n_out = _bwd_dw_checks(fn, X, dY, tern_packed, scale, gq, sgrad, workspace)
    _need(fn, "dX", dX, (T, n_in), _F32)
    _need_device(fn, X, dY, tern_packed, scale, dX, gq, sgrad, workspace)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = lib().tern_linear_bwd(_ptr(X), _ptr(dY), _act_code(X), _ptr(tern_packed), _ptr(scale), T,
                               n_in, n_out, _ptr(dX), _act_code(dX), _ptr(gq), _ptr(sgrad),
                               _ptr(workspace), ws_bytes, _stream(stream))
    _check("tern_linear_bwd", rc)


def tern_linear_bwd_noalloc(X, dY, tern_packed, scale, dX, gq, sgrad, stream=None) -> None:
    """tern_linear_bwd without a workspace: the library's static scratch is
    used (calls that overlap on one GPU race)."""
    fn = "tern_linear_bwd_noalloc"
    T, n_in, n_out = _bwd_dw_checks(fn, X, dY, tern_packed, scale, gq, sgrad, None)
    _need(fn, "dX", dX, (T, n_in), _F32)
    _need_device(fn, X, dY, tern_packed, scale, dX, gq, sgrad)
    rc = lib().tern_linear_bwd_noalloc(_ptr(X), _ptr(dY), _act_code(X), _ptr(tern_packed), _ptr(scale), T,
                                       n_in, n_out, _ptr(dX), _act_code(dX), _ptr(gq), _ptr(sgrad),
                                       _stream(stream))
    _check(fn, rc)


def _bwd_dx_checks(fn, dY, tern_packed, scale, dX, n_in):
    if dY.dim() != 2 or scale.dim() != 1 or dX.dim() != 2:
        raise ValueError(f"{fn}: dY must be [T, out], scale [out] and dX [T, in]")
    T, n_out = dY.shape
    n_in = dX.shape[1] if n_in is None else n_in
    _need(fn, "dY", dY, (T, n_out), _ACT)
    _need(fn, "scale", scale, (n_out,), _F32)
    _need(fn, "dX", dX, (T, n_in), _F32)
    _need_packed(fn, tern_packed, n_in, n_out)
    _need_device(fn, dY, tern_packed, scale, dX)
    return T, n_in, n_out


def tern_linear_bwd_dx(dY, tern_packed, scale, dX, n_in: int | None = None, stream=None) -> None:
    T, n_in, n_out = _bwd_dx_checks("tern_linear_bwd_dx", dY, tern_packed, scale, dX, n_in)
    rc = lib().tern_linear_bwd_dx(_ptr(dY), _act_code(dY), _ptr(tern_packed), _ptr(scale), T, n_in,
                                  n_out, _ptr(dX), _act_code(dX), _stream(stream))
    _check("tern_linear_bwd_dx", rc)


def tern_linear_bwd_dw(X, dY, tern_packed, scale, gq, sgrad, workspace, stream=None) -> None:
    fn = "tern_linear_bwd_dw"
    T, n_in, n_out = _bwd_dw_checks(fn, X, dY, tern_packed, scale, gq, sgrad, workspace)
    _need_device(fn, X, dY, tern_packed, scale, gq, sgrad, workspace)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = lib().tern_linear_bwd_dw(_ptr(X), _ptr(dY), _act_code(X), _ptr(tern_packed), _ptr(scale), T,
                                  n_in, n_out, _ptr(gq), _ptr(sgrad), _ptr(workspace), ws_bytes,
                                  _stream(stream))
    _check("tern_linear_bwd_dw", rc)


def tern_linear_bwd_dx_acc(dY, tern_packed, scale, dX, n_in: int | None = None, stream=None) -> None:
    """dX (fp32) += dY . (scale * tern)^T."""
    T, n_in, n_out = _bwd_dx_checks("tern_linear_bwd_dx_acc", dY, tern_packed, scale, dX, n_in)
    rc = lib().tern_linear_bwd_dx_acc(_ptr(dY), _act_code(dY), _ptr(tern_packed), _ptr(scale), T, n_in, n_out,
                                      _ptr(dX), _stream(stream))
    _check("tern_linear_bwd_dx_acc", rc)


def tern_linear_bwd_acc_workspace_bytes(T: int, n_in: int, n_out: int) -> int:
    return int(lib().tern_linear_bwd_acc_workspace_bytes(T, n_in, n_out))


def tern_linear_bwd_dw_acc(X, dY, tern_packed, scale, gq, sgrad, workspace, alpha: float = 1.0,
                           stream=None) -> None:
    """gq += alpha * G * scale, sgrad += alpha * sum_r G * tern (G = X^T . dY)."""
    fn = "tern_linear_bwd_dw_acc"
    T, n_in, n_out = _bwd_dw_checks(fn, X, dY, tern_packed, scale, gq, sgrad, workspace)
    _need_device(fn, X, dY, tern_packed, scale, gq, sgrad, workspace)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = lib().tern_linear_bwd_dw_acc(_ptr(X), _ptr(dY), _act_code(X), _ptr(tern_packed), _ptr(scale), T,
                                      n_in, n_out, float(alpha), _ptr(gq), _ptr(sgrad), _ptr(workspace),
                                      ws_bytes, _stream(stream))
    _check("tern_linear_bwd_dw_acc", rc)


def tern_group_gather(qs, scales, q_group: torch.Tensor, scale_group: torch.Tensor, stream=None) -> None:
    """q_group [in, sum out] and scale_group [sum out] from the members' q
    [in, out_i] and scale [out_i] (projections that read one input)."""
    fn = "tern_group_gather"
    n = len(qs)
    if n != len(scales):
        raise ValueError(f"{fn}: {n} q matrices but {len(scales)} scales")
    n_in = qs[0].shape[0] if n else 0
    for i, (qi, si) in enumerate(zip(qs, scales)):
        if qi.dim() != 2:
            raise ValueError(f"{fn}: q[{i}] must be [in, out_i]")
        _need(fn, f"q[{i}]", qi, (n_in, qi.shape[1]), (torch.int8,))
        _need(fn, f"scale[{i}]", si, (qi.shape[1],), _F32)
    tot = sum(int(t.shape[1]) for t in qs)
    _need(fn, "q_group", q_group, (n_in, tot), (torch.int8,))
    _need(fn, "scale_group", scale_group, (tot,), _F32)
    _need_device(fn, *qs, *scales, q_group, scale_group)
    qa = (_vp * max(n, 1))(*[_ptr(t) for t in qs])
    sa = (_vp * max(n, 1))(*[_ptr(t) for t in scales])
    oa = (_i64 * max(n, 1))(*[int(t.shape[1]) for t in qs])
    rc = lib().tern_group_gather(qa, sa, oa, n, n_in, _ptr(q_group), _ptr(scale_group), _stream(stream))
    _check("tern_group_gather", rc)


def tern_scale_adamw(sgrad, scale, m, v, step: int, lr: float, scale_lr: float | None = None, b1: float = 0.9,
                     b2: float = 0.999, eps: float = 1e-8, wd: float = 0.0, stream=None) -> None:
    """AdamW step of the per-column scale from its gradient (in place on
    scale, m, v; scale_lr defaults to lr)."""
    fn = "tern_scale_adamw"
    if scale.dim() != 1:
        raise ValueError(f"{fn}: scale must be [out]")
    for name, t in (("sgrad", sgrad), ("scale", scale), ("m", m), ("v", v)):
        _need(fn, name, t, scale.shape, _F32)
    _need_device(fn, sgrad, scale, m, v)
    sl = lr if scale_lr is None else scale_lr
    rc = lib().tern_scale_adamw(_ptr(sgrad), _ptr(scale), _ptr(m), _ptr(v), int(scale.shape[0]), int(step),
                                float(lr), float(sl), float(b1), float(b2), float(eps), float(wd),
                                _stream(stream))
    _check("tern_scale_adamw", rc)


PANEL_COUNTS = ("total", "neg", "zero", "pos", "rail", "dead", "churn", "churn_total", "scale_count")
PANEL_STATS = ("scale_sum", "scale_min", "scale_max")


def empty_panel(device="cuda") -> torch.Tensor:
    """Device storage of one tern_panel_t (9 uint64 counts, then 3 doubles)."""
    return torch.empty((len(PANEL_COUNTS) + len(PANEL_STATS),), dtype=torch.float64, device=device)


def _need_panel(fn, panel):
    _need(fn, "panel", panel, (len(PANEL_COUNTS) + len(PANEL_STATS),), (torch.float64,))


def tern_panel_reset(panel: torch.Tensor, stream=None) -> None:
    _need_panel("tern_panel_reset", panel)
    _need_device("tern_panel_reset", panel)
    _check("tern_panel_reset", lib().tern_panel_reset(_ptr(panel), _stream(stream)))


def tern_panel_add(q: torch.Tensor, theta: int, scale: torch.Tensor, panel: torch.Tensor, prev_packed=None,
                   q_clamp: int = 7, stream=None) -> None:
    """Add one ternary matrix (q int8 [in, out], scale [out]) to the panel;
    prev_packed: the previous step's handle for churn, or None."""
    fn = "tern_panel_add"
    if q.dim() != 2:
        raise ValueError(f"{fn}: q must be [in, out]")
    n_in, n_out = q.shape
    _need(fn, "q", q, (n_in, n_out), (torch.int8,))
    _need(fn, "scale", scale, (n_out,), _F32)
    _need_panel(fn, panel)
    if prev_packed is not None:
        _need_packed(fn, prev_packed, n_in, n_out)
    _need_device(fn, q, scale, panel, prev_packed)
    rc = lib().tern_panel_add(_ptr(q), n_in, n_out, int(theta), int(q_clamp), _ptr(prev_packed), _ptr(scale),
                              _ptr(panel), _stream(stream))
    _check("tern_panel_add", rc)


PANEL_FRACTIONS = ("pct_neg", "pct_zero", "pct_pos", "rail_pct", "dead_pct", "churn_frac", "scale_mean")


def tern_panel_fractions(panel_host: torch.Tensor) -> dict:
    """The page's fractions of an accumulator (host copy), computed by the
    library's tern_panel_fractions."""
    h = panel_host.contiguous()
    if h.device.type != "cpu" or h.numel() != len(PANEL_COUNTS) + len(PANEL_STATS) or h.dtype != torch.float64:
        raise ValueError("tern_panel_fractions needs a host copy of one panel (12 x 8 bytes)")
    out = (ctypes.c_double * len(PANEL_FRACTIONS))()
    _check("tern_panel_fractions", lib().tern_panel_fractions(ctypes.c_void_p(h.data_ptr()), out))
    return dict(zip(PANEL_FRACTIONS, list(out)))


def panel_values(panel: torch.Tensor) -> dict:
    """The accumulator's fields (copied to the host) and the page's fractions
    of them from tern_panel_fractions."""
    h = panel.cpu()
    n = len(PANEL_COUNTS)
    r = dict(zip(PANEL_COUNTS, h[:n].view(torch.int64).tolist()))
    r.update(zip(PANEL_STATS, h[n:].tolist()))
    r.update(tern_panel_fractions(h))
    return r


class TernProj(ctypes.Structure):
    """tern_proj_t: one projection of a layer call."""
    _fields_ = [("in_", _i64), ("out", _i64), ("q", _vp), ("tern_packed", _vp), ("scale", _vp), ("X", _vp),
                ("dY", _vp), ("Y", _vp), ("dX", _vp), ("gq", _vp), ("sgrad", _vp)]


LAYER_MEMBERS = ("q", "packed", "scale", "X", "dY", "Y", "dX", "gq", "sgrad")


def _layer(fn: str, projs, T: int | None, need, act=None):
    """Marshal a list of projections (dicts with n_in, n_out and the device
    tensors the call uses: q, packed, scale, X, dY, Y, dX, gq, sgrad) into a
    tern_proj_t array, checking every tensor the call uses."""
    n = len(projs)
    if not 1 <= n <= 8:
        raise ValueError(f"{fn}: 1 to 8 projections, got {n}")
    arr = (TernProj * n)()
    used = []
    for i, d in enumerate(projs):
        ni, no = int(d["n_in"]), int(d["n_out"])
        shapes = {"q": ((ni, no), (torch.int8,)), "scale": ((no,), _F32), "X": ((T, ni), act),
                  "dY": ((T, no), act), "Y": ((T, no), (torch.float32, act[0] if act else None)),
                  "dX": ((T, ni), _F32), "gq": ((ni, no), _F32), "sgrad": ((no,), _F32)}
        for k in need:
            if k == "packed":
                _need_packed(fn, d.get("packed"), ni, no)
            else:
                shape, dts = shapes[k]
                _need(fn, f"{k}[{i}]", d.get(k), shape, dts)
            used.append(d.get(k))
        arr[i].in_, arr[i].out = ni, no
        for k, field in (("q", "q"), ("packed", "tern_packed"), ("scale", "scale"), ("X", "X"), ("dY", "dY"),
                         ("Y", "Y"), ("dX", "dX"), ("gq", "gq"), ("sgrad", "sgrad")):
            if k in need:
                p = _ptr(d[k])
                setattr(arr[i], field, p.value if p is not None else None)
    _need_device(fn, *used)
    return arr


def tern_layer_materialize(projs, theta: int, stream=None) -> None:
    """tern_materialize of every projection (q -> packed), one launch."""
    arr = _layer("tern_layer_materialize", projs, None, ("q", "packed"))
    _check("tern_layer_materialize", lib().tern_layer_materialize(arr, len(projs), int(theta), _stream(stream)))


def tern_layer_fwd(projs, stream=None) -> None:
    """tern_linear_fwd of every projection (they share T and X's dtype)."""
    X0 = projs[0]["X"]
    act = (X0.dtype,)
    arr = _layer("tern_layer_fwd", projs, X0.shape[0], ("packed", "scale", "X", "Y"), act)
    ydt = _act_code(projs[0]["Y"])
    if any(_act_code(d["Y"]) != ydt for d in projs):
        raise TypeError("tern_layer_fwd: every Y must have the same dtype")
    _check("tern_layer_fwd", lib().tern_layer_fwd(arr, len(projs), X0.shape[0], _act_code(X0), ydt, _stream(stream)))


def tern_layer_bwd_dx(projs, stream=None) -> None:
    """tern_linear_bwd_dx of every projection."""
    dY0 = projs[0]["dY"]
    arr = _layer("tern_layer_bwd_dx", projs, dY0.shape[0], ("packed", "scale", "dY", "dX"), (dY0.dtype,))
    _check("tern_layer_bwd_dx", lib().tern_layer_bwd_dx(arr, len(projs), dY0.shape[0], _act_code(dY0),
                                                       _stream(stream)))


def tern_layer_bwd_dw_workspace_bytes(shapes, T: int) -> int:
    """Workspace of tern_layer_bwd_dw for projections of these (n_in, n_out)."""
    n = len(shapes)
    arr = (TernProj * max(n, 1))()
    for i, (ni, no) in enumerate(shapes):
        arr[i].in_, arr[i].out = int(ni), int(no)
    return int(lib().tern_layer_bwd_dw_workspace_bytes(arr, n, int(T)))


def empty_layer_workspace(shapes, T: int, device="cuda") -> torch.Tensor:
    nbytes = tern_layer_bwd_dw_workspace_bytes(shapes, T)
    return torch.empty((max(nbytes, 16) // 16, 16), dtype=torch.uint8, device=device)


def tern_layer_bwd_dw(projs, workspace, stream=None) -> None:
    """tern_linear_bwd_dw of every projection (gq, sgrad)."""
    X0 = projs[0]["X"]
    arr = _layer("tern_layer_bwd_dw", projs, X0.shape[0], ("packed", "scale", "X", "dY", "gq", "sgrad"),
                 (X0.dtype,))
    _need_device("tern_layer_bwd_dw", workspace)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("tern_layer_bwd_dw", lib().tern_layer_bwd_dw(arr, len(projs), X0.shape[0], _act_code(X0),
                                                       _ptr(workspace), ws_bytes, _stream(stream)))


RECUR_BLOCK = 16


def tern_recur_states_bytes(T: int, C: int) -> int:
    return int(lib().tern_recur_states_bytes(int(T), int(C)))


def tern_recur_workspace_bytes(T: int, C: int) -> int:
    return int(lib().tern_recur_workspace_bytes(int(T), int(C)))


# The calls below run once per generated token, where the host's share of a
# call is most of its time: each check is first made in its cheapest form, and
# only a mismatch goes through the helpers above, which word the error.

def _shaped(fn, name, t, shape, dtypes) -> None:
    if not isinstance(t, torch.Tensor) or t.shape != shape or t.dtype not in dtypes:
        _need(fn, name, t, shape, dtypes)


def _tensors(fn, **ts) -> None:
    """Words the error for an argument that is no tensor."""
    for name, t in ts.items():
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{fn}: {name} must be a tensor")


def _device_of(fn, t0, *ts) -> int:
    """Index of the one GPU every tensor (None: not given) lives on."""
    if not all(t is None or isinstance(t, torch.Tensor) for t in ts):
        raise TypeError(f"{fn}: an array must be a tensor or None")
    d = t0.get_device()
    for t in ts:
        if t is not None and t.get_device() != d:
            _need_device(fn, t0, *ts)
    if d < 0:
        _need_device(fn, t0, *ts)
    return d


def _addr(t):
    """Address of a contiguous tensor (None: not given)."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libtern must be contiguous")
    return t.data_ptr()


def _call(fn: str, dev: int, stream, *args) -> None:
    """Run an entry point on `stream` (None: the current stream of GPU dev),
    with dev the current device."""
    # the raw handle of torch.cuda.current_stream(dev), without building the object
    s = torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)
    f = getattr(_lib or lib(), fn)
    if torch._C._cuda_getDevice() == dev:
        rc = f(*args, s)
    else:
        with torch.cuda.device(dev):
            rc = f(*args, s)
    if rc:
        raise TernError(fn, rc)


def _row_stride(fn: str, name: str, t) -> int:
    """Row stride (elements) of a [rows, cols] tensor whose rows are
    contiguous: a matrix, or a column slice of a wider one."""
    rows, cols = t.shape
    if rows <= 1:
        ld = cols          # the stride of a single row means nothing
    else:
        ld = t.stride(0)
    if cols > 1 and rows and t.stride(1) != 1:
        raise ValueError(f"{fn}: the rows of {name} must be contiguous")
    return ld


def _row_strides(fn: str, names, a, b, c) -> int:
    """The row stride three [rows, cols] tensors share."""
    ld = _row_stride(fn, names[0], a)
    if _row_stride(fn, names[1], b) != ld or _row_stride(fn, names[2], c) != ld:
        raise ValueError(f"{fn}: {', '.join(names)} must share one row stride")
    return ld


def _recur_inputs(fn, K, V, R):
    """Shape of K, V and R, and the row stride they share."""
    if not isinstance(K, torch.Tensor):
        raise TypeError(f"{fn}: K must be a tensor")
    shape, dt = K.shape, K.dtype
    if len(shape) != 2:
        raise ValueError(f"{fn}: K must be [T, C]")
    if not isinstance(V, torch.Tensor) or not isinstance(R, torch.Tensor) or dt not in _ACT or V.shape != shape \
            or R.shape != shape or V.dtype is not dt or R.dtype is not dt:
        _need(fn, "K", K, shape, _ACT)
        _need(fn, "V", V, shape, (dt,))
        _need(fn, "R", R, shape, (dt,))
    strides = K.stride()
    if strides[1] == 1 and shape[0] > 1 and V.stride() == strides and R.stride() == strides:
        return shape, strides[0]
    return shape, _row_strides(fn, ("K", "V", "R"), K, V, R)


def _recur_sequences(fn, C, h0, offsets) -> int:
    S = 1
    if offsets is not None:
        if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.shape[0] < 1:
            raise ValueError(f"{fn}: offsets must be a tensor [n_seq + 1]")
        S = offsets.shape[0] - 1
        _shaped(fn, "offsets", offsets, (S + 1,), (torch.int64,))
    if h0 is not None:
        _shaped(fn, "h0", h0, (S, C), _F32)
    return S


def _bytes_of(t) -> int:
    return t.numel() * t.element_size() if t is not None else 0


def tern_recur_fwd(K, V, R, Y, workspace, h0=None, offsets=None, hT=None, states=None, stream=None) -> None:
    """Y = sigmoid(R) h with h_t = h_{t-1} + sigmoid(K_t) (V_t - h_{t-1}), over
    the packed sequences `offsets` cuts [T, C] into (int64 [n_seq + 1] on the
    device; None: one sequence).  K, V, R may be column slices of one matrix;
    hT receives the final states, states the backward's checkpoints."""
    fn = "tern_recur_fwd"
    (T, C), ld = _recur_inputs(fn, K, V, R)
    S = _recur_sequences(fn, C, h0, offsets)
    _shaped(fn, "Y", Y, (T, C), (K.dtype,))
    if hT is not None:
        _shaped(fn, "hT", hT, (S, C), _F32)
    if states is not None:
        _need_bytes(fn, "states", states, tern_recur_states_bytes(T, C))
    dev = _device_of(fn, K, V, R, Y, workspace, h0, offsets, hT, states)
    _call(fn, dev, stream, K.data_ptr(), V.data_ptr(), R.data_ptr(), ld, _act_code(K), _addr(h0), _addr(offsets), S,
          T, C, Y.data_ptr(), _row_stride(fn, "Y", Y), _addr(hT), _addr(states), _addr(workspace),
          _bytes_of(workspace))


def tern_recur_bwd(K, V, R, dY, states, dK, dV, dR, workspace, h0=None, offsets=None, dhT=None, dh0=None,
                   stream=None) -> None:
    """Gradients of tern_recur_fwd from dY (fp32 or K's dtype) and dhT (the
    gradient of hT); states as the forward wrote them."""
    fn = "tern_recur_bwd"
    (T, C), ld = _recur_inputs(fn, K, V, R)
    S = _recur_sequences(fn, C, h0, offsets)
    _shaped(fn, "dY", dY, (T, C), (torch.float32, K.dtype))
    for name, t in (("dK", dK), ("dV", dV), ("dR", dR)):
        _shaped(fn, name, t, (T, C), (K.dtype,))
    for name, t in (("dhT", dhT), ("dh0", dh0)):
        if t is not None:
            _shaped(fn, name, t, (S, C), _F32)
    _need_bytes(fn, "states", states, tern_recur_states_bytes(T, C))
    dev = _device_of(fn, K, V, R, dY, states, dK, dV, dR, workspace, h0, offsets, dhT, dh0)
    _call(fn, dev, stream, K.data_ptr(), V.data_ptr(), R.data_ptr(), ld, _act_code(K), _addr(h0), _addr(offsets), S,
          T, C, _addr(states), dY.data_ptr(), _row_stride(fn, "dY", dY), _act_code(dY), _addr(dhT), dK.data_ptr(),
          dV.data_ptr(), dR.data_ptr(), _row_strides(fn, ("dK", "dV", "dR"), dK, dV, dR), _addr(dh0),
          _addr(workspace), _bytes_of(workspace))


def tern_recur_step(K, V, R, h, Y, h_out=None, stream=None) -> None:
    """One token of each sequence (rows of K, V, R): the state moves from h to
    h_out (None: in place) and Y = sigmoid(R) h_out."""
    fn = "tern_recur_step"
    shape, ld = _recur_inputs(fn, K, V, R)
    if h_out is None:
        h_out = h
    dt, f32 = K.dtype, torch.float32
    if not (isinstance(h, torch.Tensor) and isinstance(h_out, torch.Tensor) and isinstance(Y, torch.Tensor)):
        _tensors(fn, h=h, h_out=h_out, Y=Y)
    if h.shape != shape or h.dtype is not f32 or h_out.shape != shape or h_out.dtype is not f32 \
            or Y.shape != shape or Y.dtype is not dt:
        _need(fn, "h", h, shape, _F32)
        _need(fn, "h_out", h_out, shape, _F32)
        _need(fn, "Y", Y, shape, (dt,))
    dev = K.get_device()
    if dev < 0 or V.get_device() != dev or R.get_device() != dev or h.get_device() != dev \
            or h_out.get_device() != dev or Y.get_device() != dev:
        _need_device(fn, K, V, R, h, h_out, Y)
    _call(fn, dev, stream, K.data_ptr(), V.data_ptr(), R.data_ptr(), ld, TERN_BF16 if dt is torch.bfloat16 else
          TERN_F32, shape[0], shape[1], _addr(h), _addr(h_out), Y.data_ptr(), _row_stride(fn, "Y", Y))


def empty_recur_states(T: int, C: int, device="cuda") -> torch.Tensor:
    """Checkpoints of tern_recur_fwd for tern_recur_bwd: one state row every
    RECUR_BLOCK tokens."""
    return torch.empty((-(-T // RECUR_BLOCK), C), dtype=torch.float32, device=device)


def empty_recur_workspace(T: int, C: int, device="cuda") -> torch.Tensor:
    """Workspace of tern_recur_fwd and tern_recur_bwd, either activation type."""
    return torch.empty((max(tern_recur_workspace_bytes(T, C), 16),), dtype=torch.uint8, device=device)


class TernQ4Proj(ctypes.Structure):
    """tern_q4_proj_t: one projection of a 4-bit layer call."""
    _fields_ = [("in_", _i64), ("out", _i64), ("group", _i64), ("packed", _vp), ("gscale", _vp), ("X", _vp),
                ("Y", _vp)]


def tern_q4_packed_bytes(n_in: int, n_out: int) -> int:
    return int(lib().tern_q4_packed_bytes(int(n_in), int(n_out)))


def empty_q4_packed(n_in: int, n_out: int, device="cuda") -> torch.Tensor:
    """Handle of tern_q4_pack for an [n_in, n_out] matrix."""
    return torch.empty((max(tern_q4_packed_bytes(n_in, n_out), 16) // 4,), dtype=torch.int32, device=device)


def tern_q4_pack(q: torch.Tensor, packed: torch.Tensor, stream=None) -> None:
    """q int8 [in, out] (clamped to [-8, 7]) -> 4-bit handle (see empty_q4_packed).
    For a ternary projection q is its ternary matrix (-1, 0, 1), not the accumulator."""
    fn = "tern_q4_pack"
    if not isinstance(q, torch.Tensor) or q.dim() != 2:
        raise ValueError(f"{fn}: q must be a tensor [in, out]")
    n_in, n_out = q.shape
    _need(fn, "q", q, (n_in, n_out), (torch.int8,))
    _need_bytes(fn, "packed", packed, max(tern_q4_packed_bytes(n_in, n_out), 0))
    _call(fn, _device_of(fn, q, packed), stream, _addr(q), n_in, n_out, _addr(packed))


def _q4_packed(fn, packed, n_in: int, n_out: int) -> None:
    if not isinstance(packed, torch.Tensor) or packed.dtype != torch.int32:
        raise TypeError(f"{fn}: packed must be an int32 tensor (see empty_q4_packed)")
    # 16 columns x 128 rows a block of 256 words
    if packed.numel() < -(-n_out // 16) * -(-n_in // 128) * 256:
        _need_bytes(fn, "packed", packed, tern_q4_packed_bytes(n_in, n_out))


def tern_q4_matvec(X, packed, gscale, group: int, Y, stream=None) -> None:
    """Y [T, out] = X [T, in] . (q * scale of the group), with q as packed by
    tern_q4_pack and gscale [ceil(in / group), out] (fp32 or bf16)."""
    fn = "tern_q4_matvec"
    if not isinstance(X, torch.Tensor) or not isinstance(Y, torch.Tensor):
        _tensors(fn, X=X, Y=Y)
    if X.dim() != 2 or Y.dim() != 2:
        raise ValueError(f"{fn}: X must be [T, in] and Y [T, out]")
    T, n_in = X.shape
    n_out = Y.shape[1]
    _shaped(fn, "X", X, (T, n_in), _ACT)
    _shaped(fn, "Y", Y, (T, n_out), (torch.float32, X.dtype))
    group = int(group)
    _shaped(fn, "gscale", gscale, (-(-n_in // group) if group > 0 else 0, n_out), _ACT)
    _q4_packed(fn, packed, n_in, n_out)
    dev = _device_of(fn, X, packed, gscale, Y)
    _call(fn, dev, stream, _addr(X), _act_code(X), _addr(packed), _addr(gscale), _act_code(gscale), group, T, n_in,
          n_out, _addr(Y), _act_code(Y))


def tern_layer_q4_matvec(projs, stream=None) -> None:
    """tern_q4_matvec of 1 to 8 projections in one launch.  projs: dicts with
    n_in, n_out, group and the tensors packed, gscale, X, Y; they share T and
    the types of X, gscale and Y."""
    fn = "tern_layer_q4_matvec"
    n = len(projs)
    if not 1 <= n <= 8:
        raise ValueError(f"{fn}: 1 to 8 projections, got {n}")
    first = projs[0]
    X0, s0, Y0 = first["X"], first["gscale"], first["Y"]
    tensor = torch.Tensor
    if not (isinstance(X0, tensor) and isinstance(s0, tensor) and isinstance(Y0, tensor)):
        _tensors(fn, X=X0, gscale=s0, Y=Y0)
    if X0.dim() != 2:
        raise ValueError(f"{fn}: X must be [T, in]")
    T = X0.shape[0]
    act, sdt, ydt = X0.dtype, s0.dtype, Y0.dtype
    if act not in _ACT or sdt not in _ACT or ydt not in (torch.float32, act):
        raise TypeError(f"{fn}: X and gscale must be bfloat16 or float32, Y float32 or X's dtype")
    dev = X0.get_device()
    words = []   # the tern_q4_proj_t array: seven 64-bit members each
    int32 = torch.int32
    for d in projs:
        n_in, n_out, group = d["n_in"], d["n_out"], d["group"]
        X, s, Y, pk = d["X"], d["gscale"], d["Y"], d["packed"]
        if not (isinstance(X, tensor) and isinstance(s, tensor) and isinstance(Y, tensor) and isinstance(pk, tensor)):
            _tensors(fn, X=X, gscale=s, Y=Y, packed=pk)
        if X.shape != (T, n_in) or X.dtype is not act:
            _need(fn, "X", X, (T, n_in), (act,))
        groups = -(-n_in // group) if group > 0 else 0
        if s.shape != (groups, n_out) or s.dtype is not sdt:
            _need(fn, "gscale", s, (groups, n_out), (sdt,))
        if Y.shape != (T, n_out) or Y.dtype is not ydt:
            _need(fn, "Y", Y, (T, n_out), (ydt,))
        if pk.dtype is not int32 or pk.numel() < -(-n_out // 16) * -(-n_in // 128) * 256:
            _q4_packed(fn, pk, n_in, n_out)
        if X.get_device() != dev or s.get_device() != dev or Y.get_device() != dev \
                or pk.get_device() != dev:
            _need_device(fn, X0, X, s, Y, pk)
        if not (X.is_contiguous() and s.is_contiguous() and Y.is_contiguous() and pk.is_contiguous()):
            raise ValueError("tensors passed to libtern must be contiguous")
        words += (n_in, n_out, group, pk.data_ptr(), s.data_ptr(), X.data_ptr(), Y.data_ptr())
    if dev < 0:
        _need_device(fn, X0)
    arr = array("q", words)   # alive for the call
    _call(fn, dev, stream, arr.buffer_info()[0], n, T, _act_code(X0), _act_code(s0), _act_code(Y0))


class TernOrtho(ctypes.Structure):
    """tern_ortho_t: one matrix of a layer's orthogonalisation."""
    _fields_ = [("rows", _i64), ("cols", _i64), ("G", _vp), ("O", _vp), ("gain", ctypes.c_float)]


def tern_orthogonalize_workspace_bytes(rows: int, cols: int) -> int:
    return int(lib().tern_orthogonalize_workspace_bytes(int(rows), int(cols)))


def tern_layer_orthogonalize_workspace_bytes(shapes) -> int:
    """Workspace of tern_layer_orthogonalize for matrices of these (rows, cols)."""
    arr = (TernOrtho * max(len(shapes), 1))()
    for a, (r, c) in zip(arr, shapes):
        a.rows, a.cols = int(r), int(c)
    return int(lib().tern_layer_orthogonalize_workspace_bytes(arr, len(shapes)))


def empty_ortho_workspace(shapes, device="cuda") -> torch.Tensor:
    """Workspace for matrices of these (rows, cols): one pair for
    tern_orthogonalize, a layer's for tern_layer_orthogonalize."""
    return torch.empty((max(tern_layer_orthogonalize_workspace_bytes(shapes), 16),), dtype=torch.uint8, device=device)


def tern_orthogonalize(G, O, workspace, steps: int = 5, gain: float = 1.0, stream=None) -> None:
    """O (bf16) = gain * the Newton-Schulz orthogonalisation of G (fp32 or bf16)."""
    fn = "tern_orthogonalize"
    g, o = _ortho_matrix(fn, G, O, _ACT)
    rows, cols = G.shape
    dev = _device_of(fn, G, O, workspace)
    _call(fn, dev, stream, g, _act_code(G), rows, cols, int(steps), float(gain), o, _addr(workspace),
          _bytes_of(workspace))


def _ortho_matrix(fn, G, O, dtypes):
    """Addresses of a matrix and of its result."""
    if not isinstance(G, torch.Tensor) or G.dim() != 2:
        raise ValueError(f"{fn}: G must be a tensor [rows, cols]")
    _shaped(fn, "G", G, G.shape, dtypes)
    _shaped(fn, "O", O, G.shape, (torch.bfloat16,))
    return _addr(G), _addr(O)


def tern_layer_orthogonalize(mats, workspace, steps: int = 5, stream=None) -> None:
    """tern_orthogonalize of 1 to 8 matrices together.  mats: dicts with G and O
    [rows, cols] and, if not 1, gain; the G share one dtype."""
    fn = "tern_layer_orthogonalize"
    n = len(mats)
    if not 1 <= n <= 8:
        raise ValueError(f"{fn}: 1 to 8 matrices, got {n}")
    arr = (TernOrtho * n)()
    G0 = mats[0]["G"]
    used = []
    for a, d in zip(arr, mats):
        G, O = d["G"], d["O"]
        a.G, a.O = _ortho_matrix(fn, G, O, _ACT if G is G0 else (G0.dtype,))
        a.rows, a.cols = G.shape
        a.gain = float(d.get("gain", 1.0))
        used += (G, O)
    dev = _device_of(fn, *used, workspace)
    _call(fn, dev, stream, arr, n, _act_code(G0), int(steps), _addr(workspace), _bytes_of(workspace))


def tern_norm_bwd_workspace_bytes(T: int, C: int) -> int:
    return int(lib().tern_norm_bwd_workspace_bytes(int(T), int(C)))


def empty_norm_stats(T: int, device="cuda") -> torch.Tensor:
    """Row statistics of tern_norm_fwd for tern_norm_bwd: mean and 1 / deviation."""
    return torch.empty((T, 2), dtype=torch.float32, device=device)


def empty_norm_workspace(T: int, C: int, device="cuda") -> torch.Tensor:
    """Workspace of tern_norm_bwd where it computes dw or db."""
    return torch.empty((max(tern_norm_bwd_workspace_bytes(T, C), 16),), dtype=torch.uint8, device=device)


# As for the calls above: what is wrong is worded by the helpers, what is right takes
# the fewest steps.  `dev` is the device of the call's first array.

def _elsewhere(fn, t) -> None:
    raise ValueError(f"{fn}: tensors on several devices (one on {t.device})")


def _first(fn, name, t) -> int:
    """Device index of the call's first array, a matrix (-1: not on a GPU)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{fn}: {name} must be a tensor")
    if t.dim() != 2:
        raise ValueError(f"{fn}: {name} must have two dimensions")
    return t.get_device()


def _bad(fn, name, t, shape, dtypes, dev):
    """Words what is wrong with an array that is not [shape], of these dtypes, on dev."""
    _need(fn, name, t, shape, dtypes)
    _elsewhere(fn, t)


def _matrix(fn, name, t, shape, dtypes, dev) -> tuple:
    """Address, row stride and type code of a matrix whose rows are contiguous."""
    try:
        dt = t.dtype
        if dt not in dtypes or t.shape != shape or t.get_device() != dev:
            _bad(fn, name, t, shape, dtypes, dev)
        ld, one = t.stride()
    except AttributeError:
        raise TypeError(f"{fn}: {name} must be a tensor") from None
    if one != 1 or shape[0] <= 1 or shape[1] == 0:
        ld = _row_stride(fn, name, t) if shape[1] else 0   # (the stride of rows without elements means nothing)
    return t.data_ptr(), ld, TERN_BF16 if dt is torch.bfloat16 else TERN_F32


def _vector(fn, name, t, shape, dtype, dev):
    """Address of a contiguous array (None: not given)."""
    if t is None:
        return None
    try:
        if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
            _bad(fn, name, t, shape, (dtype,), dev)
        if t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        raise TypeError(f"{fn}: {name} must be a tensor") from None
    raise ValueError("tensors passed to libtern must be contiguous")


def _work(fn, t, dev) -> tuple:
    """Address and bytes of a workspace (None: not given)."""
    # (its contents mean nothing, so its type and shape do not either)
    if t is None:
        return None, 0
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{fn}: workspace must be a tensor or None")
    if t.get_device() != dev:
        _elsewhere(fn, t)
    if not t.is_contiguous():
        raise ValueError("tensors passed to libtern must be contiguous")
    return t.data_ptr(), t.nbytes


def _on_gpu(fn, dev, t) -> None:
    if dev < 0:
        _need_device(fn, t)


def tern_norm_fwd(X, Y, w=None, b=None, A=None, S=None, stats=None, eps: float = 1e-5, stream=None) -> None:
    """Y = layer norm of S = X + A (of X without A), times w, plus b.  S, given
    with A, receives the sum (it may be X: in place); stats [T, 2] the rows'
    mean and 1 / deviation for tern_norm_bwd."""
    fn = "tern_norm_fwd"
    dev = _first(fn, "X", X)
    shape = X.shape
    T, C = shape
    x, ldx, xd = _matrix(fn, "X", X, shape, _ACT, dev)
    y, ldy, yd = _matrix(fn, "Y", Y, shape, _ACT, dev)
    a, lda, ad, s, lds = None, 0, 0, None, 0
    if A is not None or S is not None:
        if A is None or S is None:
            raise ValueError(f"{fn}: A and S are given together")
        a, lda, ad = _matrix(fn, "A", A, shape, _ACT, dev)
        s, lds, _ = _matrix(fn, "S", S, shape, (X.dtype,), dev)
    wp, bp = _vector(fn, "w", w, (C,), torch.float32, dev), _vector(fn, "b", b, (C,), torch.float32, dev)
    st = _vector(fn, "stats", stats, (T, 2), torch.float32, dev)
    _on_gpu(fn, dev, X)
    _call(fn, dev, stream, x, ldx, xd, a, lda, ad, wp, bp, float(eps), T, C, s, lds, y, ldy, yd, st)


def tern_norm_bwd(S, stats, dY, dX, workspace=None, w=None, dS=None, dw=None, db=None, stream=None) -> None:
    """Gradients of tern_norm_fwd: dX (= the gradient of X and of A) from dY and
    dS, the gradient that reaches S besides the norm (None: zeros; dX may be dS);
    dw and db [C] where given, which need the workspace (empty_norm_workspace)."""
    fn = "tern_norm_bwd"
    dev = _first(fn, "S", S)
    shape = S.shape
    T, C = shape
    s, lds, sd = _matrix(fn, "S", S, shape, _ACT, dev)
    dy, lddy, dyd = _matrix(fn, "dY", dY, shape, _ACT, dev)
    dx, lddx, dxd = _matrix(fn, "dX", dX, shape, (torch.float32, S.dtype), dev)
    ds, ldds = None, 0
    if dS is not None:
        ds, ldds, _ = _matrix(fn, "dS", dS, shape, (dX.dtype,), dev)
    if stats is None:
        raise TypeError(f"{fn}: stats must be a tensor")
    st, wp = _vector(fn, "stats", stats, (T, 2), torch.float32, dev), _vector(fn, "w", w, (C,), torch.float32, dev)
    dwp, dbp = _vector(fn, "dw", dw, (C,), torch.float32, dev), _vector(fn, "db", db, (C,), torch.float32, dev)
    ws, n = _work(fn, workspace, dev)
    _on_gpu(fn, dev, S)
    _call(fn, dev, stream, s, lds, sd, st, wp, dy, lddy, dyd, ds, ldds, T, C, dx, lddx, dxd, dwp, dbp, ws, n)


def tern_logprob_workspace_bytes(T: int, V: int, k: int = 0) -> int:
    return int(lib().tern_logprob_workspace_bytes(int(T), int(V), int(k)))


def empty_logprob_workspace(T: int, V: int, k: int = 0, device="cuda") -> torch.Tensor:
    """Workspace of tern_logprob, either type of logits."""
    return torch.empty((max(tern_logprob_workspace_bytes(T, V, k), 16),), dtype=torch.uint8, device=device)


def _logits(fn, name, t, shape, dtypes, dev) -> tuple:
    """As _matrix, for rows of any length: a single row's stride is what it would be."""
    p, ld, dt = _matrix(fn, name, t, shape, dtypes, dev)
    return p, (ld if shape[0] > 1 else -(-shape[1] // 8) * 8), dt


def _pair(fn, ids_name, ids, lp_name, lp, T, dev) -> tuple:
    """Number of entries a row and addresses of two [T, k] arrays that come together."""
    if ids is None and lp is None:
        return 0, None, None
    if ids is None or lp is None:
        raise ValueError(f"{fn}: {ids_name} and {lp_name} are given together")
    _first(fn, ids_name, ids)
    k = ids.shape[1]
    return k, _vector(fn, ids_name, ids, (T, k), torch.int64, dev), _vector(fn, lp_name, lp, (T, k), torch.float32, dev)


def tern_logprob(Z, workspace=None, tokens=None, logp=None, entropy=None, lse=None, top_ids=None, top_logp=None,
                 scale: float = 1.0, stream=None) -> None:
    """Of each row of logits Z [T, V], times scale: logp [T] of the given tokens
    (int64 [T]; 0 for one outside [0, V)), the entropy [T], the log-sum-exp lse
    [T], and the k most probable tokens, top_ids (int64) and top_logp [T, k], ties
    by rising index.  Rows start on 16 bytes: for a V that is no multiple of 8,
    Z is a column slice of a wider matrix."""
    fn = "tern_logprob"
    dev = _first(fn, "Z", Z)
    shape = Z.shape
    T, V = shape
    z, ld, zd = _logits(fn, "Z", Z, shape, _ACT, dev)
    k, ids, lp = _pair(fn, "top_ids", top_ids, "top_logp", top_logp, T, dev)
    tok, lt = _vector(fn, "tokens", tokens, (T,), torch.int64, dev), _vector(fn, "logp", logp, (T,), torch.float32, dev)
    en, ls = _vector(fn, "entropy", entropy, (T,), torch.float32, dev), _vector(fn, "lse", lse, (T,), torch.float32, dev)
    ws, n = _work(fn, workspace, dev)
    _on_gpu(fn, dev, Z)
    _call(fn, dev, stream, z, ld, zd, float(scale), T, V, tok, lt, en, ls, k, ids, lp, ws, n)


def tern_distill_workspace_bytes(T: int, V: int) -> int:
    return int(lib().tern_distill_workspace_bytes(int(T), int(V)))


def empty_distill_workspace(T: int, V: int, device="cuda") -> torch.Tensor:
    """Workspace of tern_distill, either type of logits."""
    return torch.empty((max(tern_distill_workspace_bytes(T, V), 16),), dtype=torch.uint8, device=device)


def tern_distill(Z, workspace=None, targets=None, teacher_ids=None, teacher_logp=None, alpha: float = 0.0,
                 tau: float = 1.0, loss=None, dloss=None, dZ=None, stream=None) -> None:
    """loss [T] = alpha CE(targets) + (1 - alpha) tau^2 KL(teacher || softmax(Z / tau)) of
    each row of logits Z [T, V], and where dZ is given its gradient times dloss [T]
    (None: ones); dZ may be Z.  The teacher's entries teacher_ids (int64) and
    teacher_logp [T, K] are what tern_logprob with scale = 1 / tau writes; their
    probabilities are made to sum to one."""
    fn = "tern_distill"
    dev = _first(fn, "Z", Z)
    shape = Z.shape
    T, V = shape
    z, ld, zd = _logits(fn, "Z", Z, shape, _ACT, dev)
    dz, lddz = None, 0
    if dZ is not None:
        dz, lddz, _ = _logits(fn, "dZ", dZ, shape, (Z.dtype,), dev)
    K, ids, lp = _pair(fn, "teacher_ids", teacher_ids, "teacher_logp", teacher_logp, T, dev)
    y, dl = _vector(fn, "targets", targets, (T,), torch.int64, dev), _vector(fn, "dloss", dloss, (T,), torch.float32, dev)
    lo = _vector(fn, "loss", loss, (T,), torch.float32, dev)
    ws, n = _work(fn, workspace, dev)
    _on_gpu(fn, dev, Z)
    _call(fn, dev, stream, z, ld, zd, T, V, y, K, ids, lp, float(alpha), float(tau), dl, lo, dz, lddz, ws, n)


def tern_graph_begin(stream) -> None:
    """Start recording the library calls enqueued on `stream` (a created
    torch.cuda.Stream or raw handle, not the legacy default stream)."""
    _check("tern_graph_begin", lib().tern_graph_begin(_stream(stream)))


def tern_graph_end(stream) -> ctypes.c_void_p:
    """Stop recording on `stream`; returns the instantiated graph's handle
    (release it with tern_graph_destroy)."""
    h = _vp()
    _check("tern_graph_end", lib().tern_graph_end(_stream(stream), ctypes.byref(h)))
    return h


def tern_graph_launch(graph, stream=None) -> None:
    _check("tern_graph_launch", lib().tern_graph_launch(graph, _stream(stream)))


def tern_graph_destroy(graph) -> None:
    _check("tern_graph_destroy", lib().tern_graph_destroy(graph))


# ---------------------------------------------------------------------------
# allocation helpers (torch owns the memory; the library never allocates)
# ---------------------------------------------------------------------------

def empty_packed(n_in: int, n_out: int, device="cuda") -> torch.Tensor:
    """A packed ternary handle: tern_packed_words(n_in, n_out) int32 words."""
    return torch.empty((max(tern_packed_words(n_in, n_out), 1),), dtype=torch.int32, device=device)


def packed_canonical(tern_packed: torch.Tensor, n_in: int, n_out: int) -> torch.Tensor:
    """View of the canonical 2-bit matrix at the start of a packed handle:
    [n_in, ceil(n_out / 16)] words, code of (r, c) at bits 2 (c % 16) of word
    (r, c / 16)."""
    wpr = (n_out + 15) // 16
    return tern_packed.reshape(-1)[: n_in * wpr].view(n_in, wpr)


def empty_workspace(T: int, n_in: int, n_out: int, device="cuda", acc: bool = False) -> torch.Tensor:
    """Workspace of tern_linear_bwd / tern_linear_bwd_dw (acc: of
    tern_linear_bwd_dw_acc), for either activation type."""
    q = tern_linear_bwd_acc_workspace_bytes if acc else tern_linear_bwd_workspace_bytes
    nbytes = q(T, n_in, n_out)
    return torch.empty((max(nbytes, 16) // 16, 16), dtype=torch.uint8, device=device)
