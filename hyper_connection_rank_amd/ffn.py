"""Binding of the feed-forward operators: the norms around a block
(residual_norm), the gated product (glu) and the matrix product with its
epilogue (linear), each with its gradients.

Functions with the C names (``include/hclrmix.h``) marshal tensors and a
problem struct; residual_norm(), linear(), glu() and their ``*_backward``
take torch tensors alone, check them and allocate the outputs. A call is
enqueued on the current stream of its tensors' device. Autograd records none
of them: while it records, tensors that require gradients are refused.
"""
from __future__ import annotations

import ctypes

import torch

GATE_NONE, GATE_ROW, GATE_ELEMENT = 0, 1, 2
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4, "sigmoid": 5}
NORM_MAX_HIDDEN = 32768
MAX_ROWS = 1 << 21
PRODUCT_MAX_WIDTH = 1 << 21
COUNTER_BYTES = 4096

EXPORTED = ("hclrmix_residual_norm", "hclrmix_residual_norm_workspace_size", "hclrmix_residual_norm_backward",
            "hclrmix_linear", "hclrmix_linear_backward", "hclrmix_glu", "hclrmix_glu_backward",
            "hclrmix_linear_workspace_size", "hclrmix_linear_backward_workspace_size", "hclrmix_glu_workspace_size",
            "hclrmix_glu_backward_workspace_size")

_CODES = {torch.float32: 1, torch.float16: 10, torch.bfloat16: 16}
_INVALID, _UNSUPPORTED = 1, 2


class NormProblem(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("hidden", ctypes.c_int64), ("gate_stride", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("gate", ctypes.c_int32), ("post_norm", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("alpha", ctypes.c_float), ("epsilon", ctypes.c_float)]


class Product(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("in_", ctypes.c_int64), ("out", ctypes.c_int64),
                ("x_stride", ctypes.c_int64), ("weight_stride", ctypes.c_int64), ("residual_stride", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("activation", ctypes.c_int32), ("reserved", ctypes.c_int32 * 2)]


def declare(lib) -> None:
    """Argument types of this module's entry points."""
    P, N = ctypes.c_void_p, ctypes.c_size_t
    # Problem structs go by address (c_void_p takes byref() objects).
    sig = {"hclrmix_residual_norm": [P] * 9,
           "hclrmix_residual_norm_workspace_size": [P, P],
           "hclrmix_residual_norm_backward": [P] * 13 + [N, P, P],
           "hclrmix_linear": [P] * 7 + [N, P, P],
           "hclrmix_linear_backward": [P] * 8 + [N, P, P],
           "hclrmix_glu": [P] * 9 + [N, P, P],
           "hclrmix_glu_backward": [P] * 12 + [N, P, P]}
    for name in EXPORTED:
        f = getattr(lib, name)
        f.restype = ctypes.c_int
        f.argtypes = sig.get(name, [P, P])


_fn = {}   # entry points by name, from the loaded library
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _pkg():
    import hyper_connection_rank_amd as hc
    return hc


def _refuse(detail: str, status: int = _INVALID):
    raise _pkg().HclrmixError(status, detail)


def _p(t):
    return None if t is None else t.data_ptr()


def _entry(name):
    f = _fn.get(name)
    if f is None:
        f = _fn[name] = getattr(_pkg().library(), name)
    return f


def _stream(device):
    if _raw_stream is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _call(name, device, *args):
    """Calls an entry point on the current stream of ``device``, with that device current."""
    f = _fn.get(name) or _entry(name)
    if device.type != "cuda":
        _refuse("tensors must be on a GPU", _UNSUPPORTED)
    if device.index == torch.cuda.current_device():
        status = f(*args, _stream(device))
    else:
        with torch.cuda.device(device):
            status = f(*args, _stream(device))
    if status:
        _pkg()._check(status)


def _size(name, problem) -> int:
    n = ctypes.c_size_t()
    status = _entry(name)(ctypes.byref(problem), ctypes.byref(n))
    if status:
        _pkg()._check(status)
    return n.value


# ---------------------------------------------------------------- the C names

def hclrmix_residual_norm(y, residual, gate, post_scale, pre_scale, residual_out, normed, problem: NormProblem) -> None:
    _call("hclrmix_residual_norm", y.device, _p(y), _p(residual), _p(gate), _p(post_scale), _p(pre_scale),
          _p(residual_out), _p(normed), ctypes.byref(problem))


def hclrmix_residual_norm_workspace_size(problem: NormProblem) -> int:
    return _size("hclrmix_residual_norm_workspace_size", problem)


def _ws(workspace):
    return (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())


def hclrmix_residual_norm_backward(y, residual_out, gate, post_scale, pre_scale, d_residual_out, d_normed, dy,
                                   d_residual, d_gate, d_post_scale, d_pre_scale, workspace,
                                   problem: NormProblem) -> None:
    _call("hclrmix_residual_norm_backward", y.device, _p(y), _p(residual_out), _p(gate), _p(post_scale), _p(pre_scale),
          _p(d_residual_out), _p(d_normed), _p(dy), _p(d_residual), _p(d_gate), _p(d_post_scale), _p(d_pre_scale),
          *_ws(workspace), ctypes.byref(problem))


def hclrmix_linear(x, weight, bias, residual, y, preact, workspace, problem: Product) -> None:
    _call("hclrmix_linear", x.device, _p(x), _p(weight), _p(bias), _p(residual), _p(y), _p(preact), *_ws(workspace),
          ctypes.byref(problem))


def hclrmix_linear_backward(x, weight, preact, dy, dx, d_weight, d_bias, workspace, problem: Product) -> None:
    _call("hclrmix_linear_backward", dy.device, _p(x), _p(weight), _p(preact), _p(dy), _p(dx), _p(d_weight), _p(d_bias),
          *_ws(workspace), ctypes.byref(problem))


def hclrmix_glu(x, gate_weight, up_weight, gate_bias, up_bias, h, g_out, u_out, workspace, problem: Product) -> None:
    _call("hclrmix_glu", x.device, _p(x), _p(gate_weight), _p(up_weight), _p(gate_bias), _p(up_bias), _p(h), _p(g_out),
          _p(u_out), *_ws(workspace), ctypes.byref(problem))


def hclrmix_glu_backward(x, gate_weight, up_weight, g, u, dh, dx, d_gate_weight, d_up_weight, d_gate_bias, d_up_bias,
                         workspace, problem: Product) -> None:
    _call("hclrmix_glu_backward", dh.device, _p(x), _p(gate_weight), _p(up_weight), _p(g), _p(u), _p(dh), _p(dx),
          _p(d_gate_weight), _p(d_up_weight), _p(d_gate_bias), _p(d_up_bias), *_ws(workspace), ctypes.byref(problem))


def hclrmix_linear_workspace_size(problem: Product) -> int:
    return _size("hclrmix_linear_workspace_size", problem)


def hclrmix_linear_backward_workspace_size(problem: Product) -> int:
    return _size("hclrmix_linear_backward_workspace_size", problem)


def hclrmix_glu_workspace_size(problem: Product) -> int:
    return _size("hclrmix_glu_workspace_size", problem)


def hclrmix_glu_backward_workspace_size(problem: Product) -> int:
    return _size("hclrmix_glu_backward_workspace_size", problem)


# ---------------------------------------------------------------- tensors in, tensors out

def _code(t, name):
    code = _CODES.get(t.dtype)
    if code is None:
        _refuse(f"{name} has an unsupported dtype {t.dtype}", _UNSUPPORTED)
    return code


def _same(t, like, name):
    if t.dtype is not like.dtype or t.device != like.device:
        _refuse(f"{name} must have the dtype and device of the other tensors")


def _matrix(t, like, rows, cols, name) -> int:
    """Checks t's leading dimensions flatten to rows of cols elements; returns the row stride."""
    if t is not like:
        _same(t, like, name)
        if t.dim() < 1 or t.shape[-1] != cols or t.numel() != rows * cols:
            _refuse(f"{name} must be [..., {cols}] with {rows} rows, got {tuple(t.shape)}")
    if t.is_contiguous():
        return cols
    if t.stride(-1) != 1 and cols > 1:
        _refuse(f"{name}'s last dimension must be contiguous")
    try:
        stride = t.view(rows, cols).stride(0) if t.dim() != 2 else t.stride(0)
    except RuntimeError:
        _refuse(f"{name}'s leading dimensions do not flatten into rows at one stride")
    if rows <= 1:
        return cols
    if stride < cols:
        _refuse(f"{name}'s rows overlap (stride {stride}, length {cols})")
    return stride


def _dense(t, like, shape, name):
    """Checks an optional contiguous tensor of the given shape (leading dimensions may differ)."""
    if t is None:
        return
    _same(t, like, name)
    if t.shape == shape and t.is_contiguous():
        return
    n = 1
    for d in shape:
        n *= d
    if t.numel() != n or t.dim() < 1 or t.shape[-1] != shape[-1] or not t.is_contiguous():
        _refuse(f"{name} must be contiguous {tuple(shape)}, got {tuple(t.shape)}")


def _unrecorded(*tensors):
    """Refuses tensors that require gradients while autograd records: the outputs would come back detached."""
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                _refuse("autograd does not record this call: make it under torch.no_grad() (or in a "
                        "torch.autograd.Function) and take the gradients from the *_backward function")


def _scratch(workspace, need, device):
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
        workspace[:COUNTER_BYTES].zero_()  # the arrival counters; the rest may hold anything
        return workspace
    if workspace.device != device or not workspace.is_contiguous():
        _refuse("workspace must be contiguous and on the tensors' device")
    return workspace


def _norm_problem(y, gate, post_norm, alpha, epsilon):
    code = _code(y, "y")
    if y.dim() < 1 or not y.is_contiguous():
        _refuse("y must be contiguous [..., hidden]")
    hidden = y.shape[-1]
    rows = y.numel() // hidden if hidden else 0
    kind = stride = 0
    if gate is not None:
        _same(gate, y, "gate")
        if gate.shape == y.shape[:-1] or (gate.dim() == 1 and gate.shape[0] == rows):
            kind, stride = GATE_ROW, 1
            if rows > 1 and not gate.is_contiguous():
                try:
                    stride = gate.view(rows).stride(0) if gate.dim() != 1 else gate.stride(0)
                except RuntimeError:
                    _refuse("gate's dimensions do not flatten into rows at one stride")
                if stride < 1:
                    _refuse("gate must have one value of its own per row; expand()ed gates are refused")
        elif gate.shape == y.shape:
            kind = GATE_ELEMENT
            if not gate.is_contiguous():
                _refuse("a gate per element must be contiguous")
        else:
            _refuse(f"gate must have y's shape or its leading dimensions, got {tuple(gate.shape)}")
    return NormProblem(rows, hidden, stride, code, kind, 1 if post_norm else 0, 0, alpha, epsilon)


def residual_norm(y, residual=None, *, gate=None, post_scale=None, pre_scale=None, post_norm=True, want_normed=True,
                  alpha=1.0, epsilon=1e-5, out=None):
    """The norms before and after a block with its gate and residual scale:

    z = (y / rms(y) if post_norm else y) * post_scale
    residual_out = residual + alpha * gate * z
    normed = residual_out / rms(residual_out) * pre_scale

    y [..., hidden]; residual likewise or None (zeros); gate None, y's leading
    shape (one value per row, also strided as a column of post_gate) or y's
    shape; the scales [hidden] or None (ones). ``out`` may supply
    (residual_out, normed). Returns them; normed is None with
    ``want_normed=False`` (pre_scale must then be None).
    """
    _unrecorded(y, residual, gate, post_scale, pre_scale)
    p = _norm_problem(y, gate, post_norm, alpha, epsilon)
    shape = (p.rows, p.hidden)
    _dense(residual, y, shape, "residual")
    _dense(post_scale, y, shape[1:], "post_scale")
    _dense(pre_scale, y, shape[1:], "pre_scale")
    if out is None:
        res_out, normed = torch.empty_like(y), torch.empty_like(y) if want_normed else None
    else:
        res_out, normed = out
        _dense(res_out, y, shape, "residual_out")
        _dense(normed, y, shape, "normed")
    hclrmix_residual_norm(y, residual, gate, post_scale, pre_scale, res_out, normed, p)
    return res_out, normed


def residual_norm_workspace_size(rows: int, hidden: int, dtype) -> int:
    """Bytes of the workspace of residual_norm_backward with up to that many rows."""
    return hclrmix_residual_norm_workspace_size(NormProblem(rows, hidden, 0, _dtype_code(dtype), 0, 0, 0, 1.0, 0.0))


def residual_norm_backward(y, residual_out, d_residual_out=None, d_normed=None, *, gate=None, post_scale=None,
                           pre_scale=None, post_norm=True, alpha=1.0, epsilon=1e-5, workspace=None):
    """Gradients of residual_norm from y, the residual_out that it returned and
    the gradients of its outputs (either may be None: zeros). Returns
    (dy, d_residual, d_gate, d_post_scale, d_pre_scale), None for the inputs
    that were not given. ``workspace``: a uint8 device buffer, zero-filled
    before its first use, of residual_norm_workspace_size bytes.
    """
    _unrecorded(y, residual_out, d_residual_out, d_normed, gate, post_scale, pre_scale)
    p = _norm_problem(y, gate, post_norm, alpha, epsilon)
    shape = (p.rows, p.hidden)
    for t, name in ((residual_out, "residual_out"), (d_residual_out, "d_residual_out"), (d_normed, "d_normed")):
        _dense(t, y, shape, name)
    _dense(post_scale, y, shape[1:], "post_scale")
    _dense(pre_scale, y, shape[1:], "pre_scale")
    if workspace is None and (post_scale is not None or pre_scale is not None):
        workspace = _scratch(None, hclrmix_residual_norm_workspace_size(p), y.device)
    elif workspace is not None:
        _scratch(workspace, 0, y.device)
    dy, dr = torch.empty_like(y), torch.empty_like(y)
    dg = None
    if gate is not None:
        dg = torch.empty(gate.shape, dtype=gate.dtype, device=gate.device)
    dpost = None if post_scale is None else torch.empty_like(post_scale)
    dpre = None if pre_scale is None else torch.empty_like(pre_scale)
    hclrmix_residual_norm_backward(y, residual_out, gate, post_scale, pre_scale, d_residual_out, d_normed, dy, dr, dg,
                                   dpost, dpre, workspace, p)
    return dy, dr, dg, dpost, dpre


def _act(activation) -> int:
    code = ACTIVATIONS.get(activation)
    if code is None:
        _refuse(f"unknown activation {activation!r}")
    return code


def _rows_of(t, name):
    if t.dim() < 1:
        _refuse(f"{name} must be [..., columns]")
    cols = t.shape[-1]
    return (t.numel() // cols if cols else 0), cols


def _columns(w, name) -> int:
    if w.dim() != 2:
        _refuse(f"{name} must be [in, out], got {tuple(w.shape)}")
    return w.shape[1]


def _weight(w, like, k, n, name) -> int:
    _columns(w, name)
    return _matrix(w, like, k, n, name)


def _dtype_code(dtype) -> int:
    code = _CODES.get(dtype)
    if code is None:
        _refuse(f"unsupported dtype {dtype}", _UNSUPPORTED)
    return code


def linear_workspace_size(rows: int, width_in: int, width_out: int, dtype, *, backward=False) -> int:
    """Bytes of the workspace of linear (or linear_backward) with any activation and up to that many rows."""
    p = Product(rows, width_in, width_out, 0, 0, 0, _dtype_code(dtype), ACTIVATIONS["silu"])
    return hclrmix_linear_backward_workspace_size(p) if backward else hclrmix_linear_workspace_size(p)


def glu_workspace_size(rows: int, width_in: int, width_out: int, dtype, *, backward=False) -> int:
    """Bytes of the workspace of glu (or glu_backward) with up to that many rows."""
    p = Product(rows, width_in, width_out, 0, 0, 0, _dtype_code(dtype), ACTIVATIONS["silu"])
    return hclrmix_glu_backward_workspace_size(p) if backward else hclrmix_glu_workspace_size(p)


def linear(x, weight, bias=None, residual=None, *, activation="none", save=False, out=None, workspace=None):
    """residual + act(x @ weight + bias). x [..., in], weight [in, out] (row
    stride at least out), bias [out], residual [..., out]. Returns y
    [..., out]; with ``save`` (y, preact), preact = x @ weight + bias for
    linear_backward. ``out`` may supply y. ``workspace``: a uint8 device
    buffer, zero-filled before its first use, of linear_workspace_size bytes.
    """
    _unrecorded(x, weight, bias, residual)
    code = _code(x, "x")
    rows, k = _rows_of(x, "x")
    n = _columns(weight, "weight")
    p = Product(rows, k, n, _matrix(x, x, rows, k, "x"), _weight(weight, x, k, n, "weight"), 0, code, _act(activation))
    _dense(bias, x, (n,), "bias")
    if residual is not None:
        p.residual_stride = _matrix(residual, x, rows, n, "residual")
    if out is None:
        out = x.new_empty(x.shape[:-1] + (n,))
    else:
        _dense(out, x, (rows, n), "out")
    preact = x.new_empty(out.shape) if save else None
    workspace = _scratch(workspace, 0 if workspace is not None else hclrmix_linear_workspace_size(p), x.device)
    hclrmix_linear(x, weight, bias, residual, out, preact, workspace, p)
    return (out, preact) if save else out


def linear_backward(x, weight, dy, preact=None, *, activation="none", bias=False, workspace=None):
    """Gradients of linear from dy [..., out] and, with an activation, the saved
    preact. Returns (dx, d_weight, d_bias); d_bias is None without ``bias``.
    The residual's gradient is dy."""
    _unrecorded(x, weight, dy, preact)
    code = _code(x, "x")
    rows, k = _rows_of(x, "x")
    n = _columns(weight, "weight")
    p = Product(rows, k, n, _matrix(x, x, rows, k, "x"), _weight(weight, x, k, n, "weight"), 0, code, _act(activation))
    _dense(dy, x, (rows, n), "dy")
    _dense(preact, x, (rows, n), "preact")
    dx, dw = x.new_empty(x.shape), x.new_empty((k, n))
    db = x.new_empty(n) if bias else None
    workspace = _scratch(workspace, 0 if workspace is not None else hclrmix_linear_backward_workspace_size(p), x.device)
    hclrmix_linear_backward(x, weight, preact, dy, dx, dw, db, workspace, p)
    return dx, dw, db


def _glu_problem(x, gate_weight, up_weight, activation):
    code = _code(x, "x")
    rows, k = _rows_of(x, "x")
    n = _columns(gate_weight, "gate_weight")
    stride = _weight(gate_weight, x, k, n, "gate_weight")
    if _weight(up_weight, x, k, n, "up_weight") != stride:
        _refuse("gate_weight and up_weight must have the same row stride")
    return Product(rows, k, n, _matrix(x, x, rows, k, "x"), stride, 0, code, _act(activation))


def glu(x, gate_weight, up_weight, gate_bias=None, up_bias=None, *, activation="silu", save=False, out=None,
        workspace=None):
    """act(g) * u with g = x @ gate_weight + gate_bias, u = x @ up_weight +
    up_bias, in one kernel. x [..., in]; the weights [in, out] with the same
    row stride (two column ranges of one merged weight will do). Returns h
    [..., out]; with ``save`` (h, g, u) for glu_backward. ``workspace``: a
    uint8 device buffer, zero-filled before its first use, of
    glu_workspace_size bytes."""
    _unrecorded(x, gate_weight, up_weight, gate_bias, up_bias)
    p = _glu_problem(x, gate_weight, up_weight, activation)
    rows, n = p.rows, p.out
    _dense(gate_bias, x, (n,), "gate_bias")
    _dense(up_bias, x, (n,), "up_bias")
    if out is None:
        out = x.new_empty(x.shape[:-1] + (n,))
    else:
        _dense(out, x, (rows, n), "out")
    g, u = (x.new_empty(out.shape), x.new_empty(out.shape)) if save else (None, None)
    workspace = _scratch(workspace, 0 if workspace is not None else hclrmix_glu_workspace_size(p), x.device)
    hclrmix_glu(x, gate_weight, up_weight, gate_bias, up_bias, out, g, u, workspace, p)
    return (out, g, u) if save else out


def glu_backward(x, gate_weight, up_weight, g, u, dh, *, activation="silu", bias=False, workspace=None):
    """Gradients of glu from its saved g and u and dh [..., out]. Returns
    (dx, d_gate_weight, d_up_weight, d_gate_bias, d_up_bias); the last two are
    None without ``bias``."""
    _unrecorded(x, gate_weight, up_weight, g, u, dh)
    p = _glu_problem(x, gate_weight, up_weight, activation)
    rows, k, n = p.rows, p.in_, p.out
    for t, name in ((g, "g"), (u, "u"), (dh, "dh")):
        _dense(t, x, (rows, n), name)
    dx, dwg, dwu = x.new_empty(x.shape), x.new_empty((k, n)), x.new_empty((k, n))
    dbg, dbu = (x.new_empty(n), x.new_empty(n)) if bias else (None, None)
    workspace = _scratch(workspace, 0 if workspace is not None else hclrmix_glu_backward_workspace_size(p), x.device)
    hclrmix_glu_backward(x, gate_weight, up_weight, g, u, dh, dx, dwg, dwu, dbg, dbu, workspace, p)
    return dx, dwg, dwu, dbg, dbu
