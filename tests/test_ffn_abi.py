"""The feed-forward operators' boundary on the CPU: every refusal happens on
the host before any launch (fake, never-dereferenced device pointers), the
workspace sizes cover what they state, and the binding refuses tensors whose
layout the entry points cannot take."""
from __future__ import annotations

import ctypes

import pytest
import torch

import hyper_connection_rank_amd as hc

E, U, W, OK = (hc.HCLRMIX_ERR_INVALID_ARGUMENT, hc.HCLRMIX_ERR_UNSUPPORTED, hc.HCLRMIX_ERR_WORKSPACE_TOO_SMALL,
               hc.HCLRMIX_OK)
BASE = 1 << 40
BF16 = hc.HCLRMIX_BF16


def _addr(i):
    return BASE + (i << 36)


class Call:
    """One entry point's pointers by name (fake addresses) and its problem."""

    def __init__(self, name, order, problem, **given):
        self.name, self.order, self.problem = name, order, problem
        self.p = {n: _addr(i + 1) for i, n in enumerate(order)}
        self.p.update(given)
        self.ws_bytes = 1 << 35

    def run(self):
        f = getattr(hc.library(), self.name)
        args = []
        for n in self.order:
            args.append(self.p[n])
            if n == "workspace":
                args.append(self.ws_bytes)
        return f(*args, ctypes.byref(self.problem), None)


NORM = ("y", "residual", "gate", "post_scale", "pre_scale", "residual_out", "normed")
NORM_B = ("y", "residual_out", "gate", "post_scale", "pre_scale", "d_residual_out", "d_normed", "dy", "d_residual",
          "d_gate", "d_post_scale", "d_pre_scale", "workspace")
LIN = ("x", "weight", "bias", "residual", "y", "preact", "workspace")
LIN_B = ("x", "weight", "preact", "dy", "dx", "d_weight", "d_bias", "workspace")
GLU = ("x", "gate_weight", "up_weight", "gate_bias", "up_bias", "h", "g_out", "u_out", "workspace")
GLU_B = ("x", "gate_weight", "up_weight", "g", "u", "dh", "dx", "d_gate_weight", "d_up_weight", "d_gate_bias",
         "d_up_bias", "workspace")


def norm(back=False, rows=4, hidden=64, stride=1, kind=hc.GATE_ROW, dtype=BF16, **given):
    p = hc.NormProblem(rows, hidden, stride if kind == hc.GATE_ROW else 0, dtype, kind, 1, 0, 0.5, 1e-6)
    if kind == hc.GATE_NONE:
        given.setdefault("gate", None)
        given.setdefault("d_gate", None)
    return Call("hclrmix_residual_norm" + ("_backward" if back else ""), NORM_B if back else NORM, p, **given)


def product(name, rows=4, k=64, n=32, act="silu", dtype=BF16, xs=0, ws=0, rs=0, **given):
    order = {"hclrmix_linear": LIN, "hclrmix_linear_backward": LIN_B, "hclrmix_glu": GLU,
             "hclrmix_glu_backward": GLU_B}[name]
    p = hc.Product(rows, k, n, xs, ws, rs, dtype, hc.ACTIVATIONS[act])
    return Call(name, order, p, **given)


PRODUCTS = ("hclrmix_linear", "hclrmix_linear_backward", "hclrmix_glu", "hclrmix_glu_backward")


def _expect(call, status, part=""):
    assert call.run() == status, hc.hclrmix_last_error()
    assert part in hc.hclrmix_last_error()


def test_null_problem():
    for name, order in (("hclrmix_residual_norm", NORM), ("hclrmix_residual_norm_backward", NORM_B),
                        ("hclrmix_linear", LIN), ("hclrmix_linear_backward", LIN_B), ("hclrmix_glu", GLU),
                        ("hclrmix_glu_backward", GLU_B)):
        args = [None] * len(order) + ([0] if "workspace" in order else [])
        assert getattr(hc.library(), name)(*args, None, None) == E
    for name in hc.ffn.EXPORTED:
        if name.endswith("_size"):
            n = ctypes.c_size_t()
            assert getattr(hc.library(), name)(None, ctypes.byref(n)) == E


# ---------------------------------------------------------------- norms

@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("field,value,status", [
    ("rows", -1, E), ("hidden", 0, E), ("hidden", hc.NORM_MAX_HIDDEN + 1, U), ("rows", hc.MAX_ROWS + 1, U),
    ("reserved", 1, E), ("dtype", 11, U), ("gate", 3, E), ("gate", -1, E), ("gate_stride", -1, E),
    ("gate_stride", (1 << 21) + 1, U), ("post_norm", 2, E), ("alpha", float("nan"), E), ("alpha", float("inf"), E),
    ("epsilon", -1e-3, E), ("epsilon", float("nan"), E)])
def test_norm_problem_refusals(back, field, value, status):
    c = norm(back)
    setattr(c.problem, field, value)
    _expect(c, status)
    n = ctypes.c_size_t()
    assert hc.library().hclrmix_residual_norm_workspace_size(ctypes.byref(c.problem), ctypes.byref(n)) == status


@pytest.mark.parametrize("back,missing", [(False, "y"), (False, "residual_out"), (False, "gate"), (True, "y"),
                                          (True, "residual_out"), (True, "gate")])
def test_norm_required_pointers(back, missing):
    _expect(norm(back, **{missing: None}), E)


def test_norm_gate_must_match_its_kind():
    c = norm(kind=hc.GATE_NONE)
    c.p["gate"] = _addr(20)
    _expect(c, E, "gate")
    c = norm(kind=hc.GATE_ELEMENT)
    c.problem.gate_stride = 1
    _expect(c, E, "gate_stride")
    c = norm(True, kind=hc.GATE_NONE)
    c.p["d_gate"] = _addr(20)
    _expect(c, E, "d_gate")


def test_norm_scales_go_with_their_outputs():
    _expect(norm(normed=None), E, "pre_scale")
    _expect(norm(True, post_scale=None), E, "d_post_scale")
    _expect(norm(True, pre_scale=None), E, "d_pre_scale")
    _expect(norm(True, d_normed=None), E, "d_normed")
    _expect(norm(True, dy=None, d_residual=None, d_gate=None, d_post_scale=None, d_pre_scale=None), E, "wanted")


@pytest.mark.parametrize("out", ["residual_out", "normed"])
@pytest.mark.parametrize("other", ["y", "residual", "gate", "post_scale", "pre_scale", "normed"])
def test_norm_outputs_must_not_overlap(out, other):
    if out == other:
        return
    c = norm()
    c.p[out] = c.p[other] + 2
    _expect(c, E, "overlaps")


@pytest.mark.parametrize("out", ["dy", "d_residual", "d_gate", "d_post_scale", "d_pre_scale", "workspace"])
@pytest.mark.parametrize("other", ["y", "residual_out", "gate", "d_residual_out", "d_normed", "dy", "d_pre_scale"])
def test_norm_gradients_must_not_overlap(out, other):
    if out == other:
        return
    c = norm(True)
    c.p[out] = c.p[other]
    _expect(c, E, "overlaps")


def test_norm_overlap_follows_the_gate_stride():
    # rows 0..3 of a gate 4 elements apart: an output inside that range overlaps it, one behind it does not touch it
    c = norm(stride=4)
    c.p["normed"] = c.p["gate"] + 3 * 4 * 2
    _expect(c, E, "overlaps")


@pytest.mark.parametrize("name", ["y", "residual", "gate", "pre_scale", "residual_out", "normed"])
def test_norm_alignment(name):
    c = norm()
    c.p[name] += 1
    _expect(c, U, "aligned")


def test_norm_workspace():
    c = norm(True)
    need = hc.hclrmix_residual_norm_workspace_size(c.problem)
    assert need >= 4096 + 2 * 64 * 4  # the counters and, for up to 4 rows, one workgroup's two rows of fp32 sums
    c.ws_bytes = need - 1
    _expect(c, W, str(need))
    c = norm(True, workspace=None)
    _expect(c, W)
    c = norm(True)
    c.p["workspace"] += 8
    _expect(c, U, "workspace")


def test_norm_zero_rows_launches_nothing():
    c = norm(rows=0)
    for k in c.p:
        c.p[k] = None
    _expect(c, OK)
    c.p["pre_scale"] = _addr(1)  # scales have an address when empty rows have none
    _expect(c, OK)
    c = norm(True, rows=0)
    for k in c.p:
        if k not in ("dy",):
            c.p[k] = None
    _expect(c, OK)


# ---------------------------------------------------------------- products

@pytest.mark.parametrize("name", PRODUCTS)
@pytest.mark.parametrize("field,value,status", [
    ("rows", -1, E), ("in_", 0, E), ("out", 0, E), ("in_", (1 << 21) + 1, U), ("out", (1 << 21) + 1, U),
    ("rows", hc.MAX_ROWS + 1, U), ("dtype", 0, U), ("activation", 6, E), ("activation", -1, E), ("x_stride", 63, E),
    ("weight_stride", 31, E), ("x_stride", (1 << 21) + 1, U), ("weight_stride", (1 << 21) + 1, U)])
def test_product_problem_refusals(name, field, value, status):
    c = product(name)
    setattr(c.problem, field, value)
    _expect(c, status)
    n = ctypes.c_size_t()
    size = getattr(hc.library(), name + "_workspace_size")
    assert size(ctypes.byref(c.problem), ctypes.byref(n)) == status


def test_product_refusals_of_one_kind_of_call():
    for name in PRODUCTS:
        c = product(name)
        c.problem.reserved[1] = 1
        _expect(c, E, "reserved")
        c = product(name)
        c.problem.rows, c.problem.in_, c.problem.out = 1 << 12, (1 << 20) + 1, 1 << 10
        _expect(c, U)  # rows * in above 2^32
        c.problem.rows, c.problem.in_, c.problem.out = 1, (1 << 17) + 1, 1 << 15
        _expect(c, U)  # in * out above 2^32
        if name != "hclrmix_linear":
            c = product(name)
            c.problem.residual_stride = 64
            _expect(c, E, "residual_stride")
    c = product("hclrmix_linear", rs=31)
    _expect(c, E, "stride")
    for name in ("hclrmix_glu", "hclrmix_glu_backward"):
        _expect(product(name, act="none"), E, "activation")
    c = product("hclrmix_linear_backward", act="none")
    _expect(c, E, "preact")


@pytest.mark.parametrize("name,missing", [
    ("hclrmix_linear", "x"), ("hclrmix_linear", "weight"), ("hclrmix_linear", "y"), ("hclrmix_linear_backward", "dy"),
    ("hclrmix_linear_backward", "preact"), ("hclrmix_linear_backward", "weight"), ("hclrmix_linear_backward", "x"),
    ("hclrmix_glu", "x"), ("hclrmix_glu", "gate_weight"), ("hclrmix_glu", "up_weight"), ("hclrmix_glu", "h"),
    ("hclrmix_glu", "g_out"), ("hclrmix_glu", "u_out"), ("hclrmix_glu_backward", "g"), ("hclrmix_glu_backward", "u"),
    ("hclrmix_glu_backward", "dh"), ("hclrmix_glu_backward", "x"), ("hclrmix_glu_backward", "up_weight"),
    ("hclrmix_glu_backward", "d_up_weight"), ("hclrmix_glu_backward", "d_gate_bias")])
def test_product_required_pointers(name, missing):
    _expect(product(name, **{missing: None}), E)


def test_backward_wants_a_gradient():
    _expect(product("hclrmix_linear_backward", dx=None, d_weight=None, d_bias=None), E, "wanted")
    _expect(product("hclrmix_glu_backward", dx=None, d_gate_weight=None, d_up_weight=None, d_gate_bias=None,
                    d_up_bias=None), E, "wanted")


OUTPUTS = {"hclrmix_linear": ("y", "preact"), "hclrmix_linear_backward": ("dx", "d_weight", "d_bias"),
           "hclrmix_glu": ("h", "g_out", "u_out"),
           "hclrmix_glu_backward": ("dx", "d_gate_weight", "d_up_weight", "d_gate_bias", "d_up_bias")}


@pytest.mark.parametrize("name", PRODUCTS)
def test_product_outputs_must_not_overlap(name):
    order = product(name).order
    for out in OUTPUTS[name] + ("workspace",):
        for other in order:
            if other == out:
                continue
            c = product(name)
            c.p[out] = c.p[other]
            _expect(c, E, "overlaps")
            c = product(name)
            c.p[out] += 1
            assert c.run() == U, (name, out)


def test_product_overlap_follows_the_strides():
    # the last of 4 rows of x, 100 elements apart, ends 3 * 100 + 64 elements in
    c = product("hclrmix_linear", xs=100)
    c.p["y"] = c.p["x"] + 2 * (3 * 100 + 63)
    _expect(c, E, "y overlaps x")
    c = product("hclrmix_linear", ws=100)
    c.p["y"] = c.p["weight"] + 2 * (63 * 100 + 31)
    _expect(c, E, "y overlaps weight")


@pytest.mark.parametrize("name", PRODUCTS)
def test_product_workspace(name):
    for rows, k, n in ((1, 2560, 10240), (7, 33, 1), (300, 10240, 2560), (8192, 2560, 512)):
        c = product(name, rows=rows, k=k, n=n)
        need = getattr(hc, name + "_workspace_size")(c.problem)
        assert need >= 4096
        if name == "hclrmix_glu_backward":
            assert need >= 4096 + 2 * rows * n * 2
        c.ws_bytes = need - 1
        _expect(c, W, str(need))
        c = product(name, rows=rows, k=k, n=n, workspace=None)
        _expect(c, W)


def test_product_zero_rows_launches_nothing():
    for name in ("hclrmix_linear", "hclrmix_glu"):
        c = product(name, rows=0)
        for k in c.p:
            c.p[k] = None
        _expect(c, OK)
    for name in ("hclrmix_linear_backward", "hclrmix_glu_backward"):
        c = product(name, rows=0)
        for k in c.p:
            if k != "dx":
                c.p[k] = None
        _expect(c, OK)


# ---------------------------------------------------------------- the binding (CPU tensors: refused before any call)

def _refused(f, *args, part="", **kw):
    with pytest.raises(hc.HclrmixError) as e:
        f(*args, **kw)
    assert part in str(e.value), str(e.value)


def test_binding_refuses_layouts_it_cannot_pass_on():
    t = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    _refused(hc.residual_norm, t(4, 8).t(), part="contiguous")
    _refused(hc.residual_norm, t(4, 8), t(4, 9), part="residual")
    _refused(hc.residual_norm, t(4, 8), t(4, 8).float(), part="dtype")
    _refused(hc.residual_norm, t(4, 8), gate=t(5), part="gate")
    _refused(hc.residual_norm, t(4, 8), gate=t(1).expand(4), part="expand")
    _refused(hc.residual_norm, t(4, 8), pre_scale=t(7), part="pre_scale")
    _refused(hc.residual_norm, torch.zeros(4, 8, dtype=torch.float64), part="float64")
    _refused(hc.linear, t(4, 8), t(9, 3), part="weight")
    _refused(hc.linear, t(4, 8), t(3, 8).t(), part="contiguous")
    _refused(hc.linear, t(8).expand(4, 8), t(8, 3), part="overlap")
    _refused(hc.linear, t(4, 8, 2)[:, :, 0], t(8, 3), part="contiguous")
    _refused(hc.linear, t(4, 8), t(8, 3), t(4), part="bias")
    _refused(hc.linear, t(4, 8), t(8, 3), activation="tanh", part="activation")
    _refused(hc.linear, t(4, 8), t(8, 3), residual=t(4, 4), part="residual")
    _refused(hc.linear_backward, t(4, 8), t(8, 3), t(4, 6)[:, ::2], part="dy")
    _refused(hc.glu, t(4, 8), t(8, 3), t(8, 6)[:, 3:], part="stride")
    _refused(hc.glu, t(4, 8), t(8, 3), t(8, 4), part="up_weight")
    _refused(hc.glu_backward, t(4, 8), t(8, 3), t(8, 3), t(4, 3), t(4, 3), t(3, 3), part="dh")


def test_binding_refuses_cpu_tensors():
    t = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    _refused(hc.residual_norm, t(4, 8), part="GPU")
    _refused(hc.linear, t(4, 8), t(8, 3), part="GPU")
    _refused(hc.glu, t(4, 8), t(8, 3), t(8, 3), part="GPU")
