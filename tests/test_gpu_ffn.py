"""GPU tests of the feed-forward operators (residual_norm, linear, glu and
their gradients) against fp64 (tests/_ffn.py states the error bounds), at the
sizes where their kernels change: single rows, odd widths and unaligned
tensors, tile edges, split contractions, strided operands, zero rows; plus
captured graphs, side streams, shared workspaces, and the operators in a row
as a model uses them between two hyper-connection blocks."""
from __future__ import annotations

import math

import pytest
import torch

import _ffn as R
import hyper_connection_rank_amd as hc
import synth
from _ffn import T_OF, rand, within

pytestmark = pytest.mark.gpu
DTYPES = ["bf16", "f16", "f32"]


def bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)


def same(a, b, label):
    for i, (x, y) in enumerate(zip(a, b)):
        assert (x is None) == (y is None), (label, i)
        if x is not None:
            assert torch.equal(bits(x), bits(y)), (label, i)


def shifted(t):
    """The same values one element past a 16-byte boundary."""
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    v = buf[1:].view(t.shape)
    v.copy_(t)
    return v


# ---------------------------------------------------------------- norms

def norm_inputs(rows, H, dt, gate, seed):
    t = {"y": rand((rows, H), dt, seed), "residual": rand((rows, H), dt, seed + 1, 2.0),
         "post_scale": 1 + rand((H,), dt, seed + 2, 0.1), "pre_scale": 1 + rand((H,), dt, seed + 3, 0.1), "gate": None}
    if gate == "row":
        t["gate"] = (2 * torch.sigmoid(rand((rows, 4), torch.float32, seed + 4))).to(dt)[:, 2]
    elif gate == "element":
        t["gate"] = torch.sigmoid(rand((rows, H), torch.float32, seed + 4)).to(dt)
    return t


NORM_SHAPES = [(1, 1), (3, 7), (2, 64), (5, 2057), (1, 2560), (1030, 2560), (1025, 1001), (1026, 4096), (1024, 2048),
               (3, 4096), (2, 8200), (7, 12289), (2, 16384), (2, 32768), (3, 20001)]


@pytest.mark.parametrize("gate", ["none", "row", "element"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,H", NORM_SHAPES)
def test_residual_norm(rows, H, dtype, gate):
    dt = T_OF[dtype]
    t = norm_inputs(rows, H, dt, gate, 10 + rows + H)
    ref = R.norm(t["y"], t["residual"], t["gate"], t["post_scale"], t["pre_scale"], True, 0.5, 1e-6)
    out = hc.residual_norm(t["y"], t["residual"], gate=t["gate"], post_scale=t["post_scale"], pre_scale=t["pre_scale"],
                           alpha=0.5, epsilon=1e-6)
    for got, name in zip(out, ("residual_out", "normed")):
        within(got, *ref[name], (name, rows, H, dtype, gate))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H", [8, 2560, 1001])
def test_residual_norm_optional_tensors(H, dtype):
    """Without a residual, scales, the post norm or the second output; the same
    bits from tensors that are not 16-byte aligned; a row of zeros."""
    dt = T_OF[dtype]
    t = norm_inputs(9, H, dt, "row", 77 + H)
    t["y"][4] = 0
    t["residual"][4] = 0
    for res in (None, t["residual"]):
        for post in (None, t["post_scale"]):
            for post_norm in (False, True):
                ref = R.norm(t["y"], res, t["gate"], post, None, post_norm, -1.5, 1e-5)
                out = hc.residual_norm(t["y"], res, gate=t["gate"], post_scale=post, post_norm=post_norm, alpha=-1.5)
                for got, name in zip(out, ("residual_out", "normed")):
                    within(got, *ref[name], (name, H, dtype, res is None, post is None, post_norm))
                one, none = hc.residual_norm(t["y"], res, gate=t["gate"], post_scale=post, post_norm=post_norm,
                                             alpha=-1.5, want_normed=False)
                assert none is None
                same([one], out[:1], "residual_out alone")
    a = hc.residual_norm(t["y"], t["residual"], gate=t["gate"], post_scale=t["post_scale"], pre_scale=t["pre_scale"])
    b = hc.residual_norm(shifted(t["y"]), shifted(t["residual"]), gate=t["gate"].contiguous(),
                         post_scale=shifted(t["post_scale"]), pre_scale=shifted(t["pre_scale"]))
    same(a, b, "unaligned")


def _norm_back(t, r, dres, dn, post_norm=True, alpha=0.5, eps=1e-6, **kw):
    return hc.residual_norm_backward(t["y"], r, dres, dn, gate=t["gate"], post_scale=t["post_scale"],
                                     pre_scale=t["pre_scale"], post_norm=post_norm, alpha=alpha, epsilon=eps, **kw)


NAMES = ("dy", "d_residual", "d_gate", "d_post_scale", "d_pre_scale")


@pytest.mark.parametrize("gate", ["none", "row", "element"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,H", NORM_SHAPES + [(1541, 264)])
def test_residual_norm_backward(rows, H, dtype, gate):
    dt = T_OF[dtype]
    t = norm_inputs(rows, H, dt, gate, 20 + rows + H)
    dres, dn = rand((rows, H), dt, 5), rand((rows, H), dt, 6)
    ref = R.norm_backward(t["y"], t["residual"], dres, dn, t["gate"], t["post_scale"], t["pre_scale"], True, 0.5, 1e-6)
    out = _norm_back(t, t["residual"], dres, dn)
    for got, name in zip(out, NAMES):
        assert (got is None) == (name not in ref)
        if got is not None:
            within(got, *ref[name], (name, rows, H, dtype, gate))
    same(out, _norm_back(t, t["residual"], dres, dn), "repeated")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H", [16, 777])
def test_residual_norm_backward_optional_tensors(H, dtype):
    dt = T_OF[dtype]
    rows = 70
    for dres_on, dn_on, post_on, pre_on, post_norm, gate in [
            (True, False, True, False, True, "row"), (False, True, True, True, True, "element"),
            (True, True, False, False, False, "row"), (True, True, True, True, False, "none"),
            (True, False, False, False, True, "none"), (False, True, False, True, False, "row")]:
        t = norm_inputs(rows, H, dt, gate, 31 + H)
        t["post_scale"] = t["post_scale"] if post_on else None
        t["pre_scale"] = t["pre_scale"] if pre_on else None
        dres, dn = (rand((rows, H), dt, 5) if dres_on else None), (rand((rows, H), dt, 6) if dn_on else None)
        ref = R.norm_backward(t["y"], t["residual"], dres, dn, t["gate"], t["post_scale"], t["pre_scale"], post_norm,
                              0.75, 1e-5)
        out = _norm_back(t, t["residual"], dres, dn, post_norm, 0.75, 1e-5)
        for got, name in zip(out, NAMES):
            assert (got is None) == (name not in ref)
            if got is not None:
                within(got, *ref[name], (name, H, dtype, dres_on, dn_on, post_on, pre_on, post_norm, gate))


def test_residual_norm_gradient_by_differences():
    """fp32: <gradient, direction> against central differences of the forward call."""
    rows, H, e = 6, 40, 2.0 ** -7
    for gate in ("row", "element"):
        t = norm_inputs(rows, H, torch.float32, gate, 3)
        t["gate"] = t["gate"].contiguous()
        cr, cn = rand((rows, H), torch.float32, 8), rand((rows, H), torch.float32, 9)

        def f(v):
            a, b = hc.residual_norm(v["y"], v["residual"], gate=v["gate"], post_scale=v["post_scale"],
                                    pre_scale=v["pre_scale"], alpha=0.5, epsilon=1e-3)
            return ((a * cr).double().sum() + (b * cn).double().sum()).item()

        r, _ = hc.residual_norm(t["y"], t["residual"], gate=t["gate"], post_scale=t["post_scale"],
                                pre_scale=t["pre_scale"], alpha=0.5, epsilon=1e-3)
        grads = dict(zip(("y", "residual", "gate", "post_scale", "pre_scale"),
                         _norm_back(t, r, cr, cn, True, 0.5, 1e-3)))
        for name, g in grads.items():
            d = rand(t[name].shape, torch.float32, 12)
            up, down = dict(t), dict(t)
            up[name], down[name] = t[name] + e * d, t[name] - e * d
            num = (f(up) - f(down)) / (2 * e)
            ana = (g.double() * d.double()).sum().item()
            # differences: third derivatives (of order one per element along d) times e^2 / 6 over 240 elements,
            # added up with independent signs, and fp32 noise of f, 2^-24 * sqrt(480) / e
            tol = e * e * 240 ** 0.5 + 2.0 ** -24 * 480 ** 0.5 / e + 1e-3 * abs(ana)
            assert abs(num - ana) <= tol, (gate, name, num, ana, tol)


# ---------------------------------------------------------------- linear and glu

LINEAR_SHAPES = [(1, 1, 1), (1, 8, 8), (3, 33, 17), (2, 2560, 64), (16, 256, 128), (17, 128, 136), (5, 4096, 48),
                 (64, 200, 264), (129, 320, 264), (300, 1003, 777), (257, 64, 512), (1, 10240, 320), (16, 2600, 1000),
                 (40, 5120, 136), (700, 520, 1032), (33, 1, 5), (128, 2057, 8)]


def linear_inputs(m, k, n, dt, seed, bias=True, res=True):
    return (rand((m, k), dt, seed), rand((k, n), dt, seed + 1, k ** -0.5), rand((n,), dt, seed + 2) if bias else None,
            rand((m, n), dt, seed + 3, 2.0) if res else None)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("i,shape", list(enumerate(LINEAR_SHAPES)))
def test_linear(i, shape, dtype):
    m, k, n = shape
    dt = T_OF[dtype]
    act = list(R.ACTS)[i % 6]
    x, w, b, res = linear_inputs(m, k, n, dt, 40 + i, i % 3 != 1, i % 4 != 2)
    y, ey, p, ep = R.linear(x, w, b, res, act)
    print(f"[linear] {shape} {dtype} {act}", flush=True)
    got, pre = hc.linear(x, w, b, res, activation=act, save=True)
    within(got, y, ey, ("y", shape, dtype, act))
    within(pre, p, ep, ("preact", shape, dtype))
    same([got], [hc.linear(x, w, b, res, activation=act)], "without preact")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("i,shape", list(enumerate(LINEAR_SHAPES)))
def test_linear_backward(i, shape, dtype):
    m, k, n = shape
    dt = T_OF[dtype]
    act = list(R.ACTS)[(i + 3) % 6]
    x, w, _, _ = linear_inputs(m, k, n, dt, 60 + i)
    dy, pre = rand((m, n), dt, 3), rand((m, n), dt, 4) if act != "none" else None
    ref = R.linear_backward(x, w, dy, pre, act)
    print(f"[linear_backward] {shape} {dtype} {act}", flush=True)
    out = hc.linear_backward(x, w, dy, pre, activation=act, bias=True)
    for got, name in zip(out, ("dx", "dw0", "db0")):
        within(got, *ref[name], (name, shape, dtype, act))
    again = hc.linear_backward(x, w, dy, pre, activation=act)
    assert again[2] is None
    same(out[:2], again[:2], "without bias")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("i,shape", list(enumerate(LINEAR_SHAPES)))
def test_glu(i, shape, dtype):
    m, k, n = shape
    dt = T_OF[dtype]
    act = list(R.ACTS)[1 + i % 5]
    x, wg, bg, _ = linear_inputs(m, k, n, dt, 80 + i, i % 2 == 0)
    _, wu, bu, _ = linear_inputs(m, k, n, dt, 180 + i, i % 3 == 0)
    ref = R.glu(x, wg, wu, bg, bu, act)
    print(f"[glu] {shape} {dtype} {act}", flush=True)
    out = hc.glu(x, wg, wu, bg, bu, activation=act, save=True)
    for got, name in zip(out, ("h", "g", "u")):
        within(got, *ref[name], (name, shape, dtype, act))
    same(out[:1], [hc.glu(x, wg, wu, bg, bu, activation=act)], "without g and u")


GLU_NAMES = ("dx", "dw0", "dw1", "db0", "db1")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("i,shape", list(enumerate(LINEAR_SHAPES)))
def test_glu_backward(i, shape, dtype):
    m, k, n = shape
    dt = T_OF[dtype]
    act = list(R.ACTS)[1 + (i + 2) % 5]
    x, wg, _, _ = linear_inputs(m, k, n, dt, 90 + i)
    wu = rand((k, n), dt, 191 + i, k ** -0.5)
    g, u, dh = (rand((m, n), dt, s) for s in (3, 4, 5))
    ref = R.glu_backward(x, wg, wu, g, u, dh, act)
    print(f"[glu_backward] {shape} {dtype} {act}", flush=True)
    out = hc.glu_backward(x, wg, wu, g, u, dh, activation=act, bias=True)
    for got, name in zip(out, GLU_NAMES):
        within(got, *ref[name], (name, shape, dtype, act))
    same(out[:3], hc.glu_backward(x, wg, wu, g, u, dh, activation=act)[:3], "without biases")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_products_of_many_tiles(dtype):
    """Enough output tiles for the 256 x 256 kernel in each operand layout,
    with ragged edges, and left-over tiles whose contraction is split."""
    dt = T_OF[dtype]
    for m, k, n in ((4090, 1032, 4088), (4090, 2600, 4600)):
        print(f"[many tiles] linear {m} {k} {n}", flush=True)
        x, w, b, res = linear_inputs(m, k, n, dt, 11)
        within(hc.linear(x, w, b, res, activation="silu"), *R.linear(x, w, b, res, "silu")[:2], ("linear", m, k, n))
    m, k, n = 4090, 264, 2040
    print(f"[many tiles] glu {m} {k} {n}", flush=True)
    x, wg, bg, _ = linear_inputs(m, k, n, dt, 12)
    _, wu, bu, _ = linear_inputs(m, k, n, dt, 13)
    ref = R.glu(x, wg, wu, bg, bu, "gelu")
    for got, name in zip(hc.glu(x, wg, wu, bg, bu, activation="gelu", save=True), ("h", "g", "u")):
        within(got, *ref[name], (name, m, k, n))
    for m, k, n in ((4090, 4088, 520), (520, 4088, 4088)):
        print(f"[many tiles] glu_backward {m} {k} {n}", flush=True)
        x, wg, _, _ = linear_inputs(m, k, n, dt, 14)
        wu = rand((k, n), dt, 15, k ** -0.5)
        g, u, dh = (rand((m, n), dt, s) for s in (3, 4, 5))
        ref = R.glu_backward(x, wg, wu, g, u, dh, "silu")
        for got, name in zip(hc.glu_backward(x, wg, wu, g, u, dh, bias=True), GLU_NAMES):
            within(got, *ref[name], (name, m, k, n))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,k,n", [(3, 520, 96), (150, 264, 200), (150, 263, 201)])
def test_strided_operands_and_unaligned_tensors(m, k, n, dtype):
    """Column ranges of wider tensors (NaN around them must not leak in), and
    tensors one element past a 16-byte boundary, give the contiguous
    operands' values."""
    dt = T_OF[dtype]
    x, w, b, res = linear_inputs(m, k, n, dt, 7)
    wu = rand((k, n), dt, 9, k ** -0.5)

    def inside(t, left, right):
        buf = torch.full((t.shape[0], left + t.shape[1] + right), float("nan"), dtype=dt, device="cuda")
        buf[:, left:left + t.shape[1]] = t
        return buf[:, left:left + t.shape[1]]

    y, ey, _, _ = R.linear(x, w, b, res, "silu")
    ref = R.glu(x, w, wu, None, None, "silu")
    dy = rand((m, n), dt, 5)
    pre = rand((m, n), dt, 6)
    lb, gb = R.linear_backward(x, w, dy, pre, "silu"), R.glu_backward(x, w, wu, pre, res, dy, "gelu")
    for left, right in ((8, 8), (3, 4), (0, 1)):
        merged = torch.full((k, left + 2 * n + 2 * right), float("nan"), dtype=dt, device="cuda")
        merged[:, left:left + n], merged[:, left + n + right:left + 2 * n + right] = w, wu
        xs, ws, us = inside(x, left, right), merged[:, left:left + n], merged[:, left + n + right:left + 2 * n + right]
        rs = inside(res, left, right)
        within(hc.linear(xs, ws, b, rs, activation="silu"), y, ey, ("strided linear", left))
        within(hc.glu(xs, ws, us), *ref["h"], ("strided glu", left))
        for got, name in zip(hc.linear_backward(xs, ws, dy, pre, activation="silu", bias=True), ("dx", "dw0", "db0")):
            within(got, *lb[name], ("strided linear_backward", left, name))
        for got, name in zip(hc.glu_backward(xs, ws, us, pre, res, dy, activation="gelu", bias=True), GLU_NAMES):
            within(got, *gb[name], ("strided glu_backward", left, name))
    s = shifted
    within(hc.linear(s(x), s(w), s(b), s(res), activation="silu", out=s(res)), y, ey, "shifted linear")
    within(hc.glu(s(x), s(w), s(wu)), *ref["h"], "shifted glu")
    for got, name in zip(hc.glu_backward(s(x), s(w), s(wu), s(pre), s(res), s(dy), activation="gelu", bias=True), GLU_NAMES):
        within(got, *gb[name], ("shifted glu_backward", name))


def test_values_that_are_not_finite_stay_in_their_rows():
    """NaN in one row of x, in the padding of the last tile's neighbours: only that row's outputs are NaN."""
    for m, k, n in ((5, 320, 72), (150, 264, 136), (20, 37, 9)):
        for dtype in DTYPES:
            dt = T_OF[dtype]
            x, w, b, res = linear_inputs(m, k, n, dt, 3)
            x[1] = float("nan")
            y = hc.linear(x, w, b, res)
            h = hc.glu(x, w, w.clone())
            for t in (y, h):
                assert torch.isnan(t[1]).all()
                assert torch.isfinite(t[0]).all() and torch.isfinite(t[2:]).all()


def test_zero_rows():
    for dt in T_OF.values():
        x, w = torch.zeros(0, 24, dtype=dt, device="cuda"), torch.ones(24, 40, dtype=dt, device="cuda")
        g = torch.zeros(0, 40, dtype=dt, device="cuda")
        assert hc.linear(x, w).shape == (0, 40) and hc.glu(x, w, w.clone()).shape == (0, 40)
        outs = hc.linear_backward(x, w, g, bias=True) + hc.glu_backward(x, w, w.clone(), g, g, g, bias=True)
        s = torch.ones(24, dtype=dt, device="cuda")
        assert hc.residual_norm(x, x.clone(), pre_scale=s)[1].shape == (0, 24)
        outs += hc.residual_norm_backward(x, x, x, x, post_scale=s, pre_scale=s)
        for t in outs:
            if t is not None:
                assert not t.any()


def test_leading_dimensions_flatten():
    x, w, b, res = linear_inputs(6, 64, 40, torch.bfloat16, 3)
    y = hc.linear(x, w, b, res)
    same([hc.linear(x.view(2, 3, 64), w, b, res.view(2, 3, 40)).view(6, 40)], [y], "linear")
    same([hc.linear(x[0], w, b, res[0])], [hc.linear(x[:1], w, b, res[:1])[0]], "one vector")
    t = norm_inputs(6, 64, torch.bfloat16, "row", 3)
    a = hc.residual_norm(t["y"], t["residual"], gate=t["gate"])
    c = hc.residual_norm(t["y"].view(2, 3, 64), t["residual"].view(2, 3, 64), gate=t["gate"].view(2, 3))
    same([v.view(6, 64) for v in c], a, "norm")


# ---------------------------------------------------------------- workspaces, streams, graphs

def _split_calls(dt, seed):
    """Calls whose contraction is split over workgroups, with their inputs."""
    x, w, b, res = linear_inputs(3, 5120, 264, dt, seed)
    wu = rand((5120, 264), dt, seed + 9, 5120 ** -0.5)
    x2, w2, _, _ = linear_inputs(40, 264, 2560, dt, seed + 20)
    dy = rand((40, 2560), dt, seed + 30)
    x3, w3, _, _ = linear_inputs(900, 96, 200, dt, seed + 40)
    d3 = rand((900, 200), dt, seed + 50)
    return [lambda ws: (hc.linear(x, w, b, res, workspace=ws),), lambda ws: (hc.glu(x, w, wu, workspace=ws),),
            lambda ws: hc.linear_backward(x2, w2, dy, bias=True, workspace=ws)[:3],
            lambda ws: hc.glu_backward(x3, w3, w3, d3, d3, d3, bias=True, workspace=ws),
            lambda ws: hc.residual_norm_backward(d3, d3, d3, d3, post_scale=w3[0], pre_scale=w3[1], workspace=ws)]


WS_BYTES = 64 << 20


@pytest.mark.parametrize("dtype", DTYPES)
def test_one_workspace_serves_every_call(dtype):
    """Split sums meet NaN and each other's leftovers in the scratch, leave the
    counters zero, and repeat bit for bit; hclrmix_run shares the workspace."""
    dt = T_OF[dtype]
    calls = _split_calls(dt, 100)
    fresh = [f(None) for f in calls]
    ws = torch.zeros(WS_BYTES, dtype=torch.uint8, device="cuda")
    ws[4096:] = 0xFF
    w = synth.WORKLOADS["decode_bf16"]
    t = {k: v.cuda() for k, v in synth.block_inputs(w, rows=3).items()}
    names = ("streams", "norm_scale", "down_weight", "up_weight", "inject_weight", "prev_block_output", "prev_post_gate")
    block = lambda ws_: hc.block(*[t[n] for n in names], **w.attrs(), workspace=ws_)  # noqa: E731
    ref_block = block(None)
    for _ in range(3):
        for i, f in enumerate(calls):
            same(f(ws), fresh[i], (dtype, i))
            assert not ws[:4096].any(), i
        same(block(ws), ref_block, "block")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_graphs_replay(dtype):
    """Every call captured once and replayed with new inputs between eager
    work; two graphs with a workspace each replay in turn."""
    dt = T_OF[dtype]
    x, w, b, res = linear_inputs(5, 2560, 200, dt, 1)
    wu = rand((2560, 200), dt, 2, 2560 ** -0.5)
    wd = rand((200, 2560), dt, 3, 200 ** -0.5)
    s = 1 + rand((2560,), dt, 4, 0.1)

    def step(x_, ws):
        r, n = hc.residual_norm(x_, x_ * 0.5, pre_scale=s, post_scale=s)
        h, g, u = hc.glu(n, w, wu, save=True, workspace=ws)
        y = hc.linear(h, wd, None, r, workspace=ws)
        dh, dwd, _ = hc.linear_backward(h, wd, y, workspace=ws)
        dn, dwg, dwu, dbg, dbu = hc.glu_backward(n, w, wu, g, u, dh, bias=True, workspace=ws)
        return (y, dwd, dwg, dwu, dbg, dbu) + hc.residual_norm_backward(x_, r, y, dn, post_scale=s, pre_scale=s, workspace=ws)

    size = 32 << 20
    graphs = []
    for i in range(2):
        xs, ws = x.clone(), torch.zeros(size, dtype=torch.uint8, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(xs, ws)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = step(xs, ws)
        graphs.append((g, xs, outs, ws))  # a graph's buffers live as long as it does
    eager_ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for k in range(4):
        g, xs, outs, _ = graphs[k % 2]
        new = rand((5, 2560), dt, 50 + k)
        xs.copy_(new)
        g.replay()
        torch.cuda.synchronize()
        got = [o.clone() if o is not None else None for o in outs]
        same(got, step(new, eager_ws), ("replay", k))


def test_side_stream():
    """Work goes to the current stream: inputs produced there, outputs ready there."""
    x, w, b, res = linear_inputs(9, 2560, 320, torch.bfloat16, 5)
    ref = hc.linear(x, w, b, res)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        big = torch.randn(4096, 4096, device="cuda")
        for _ in range(4):
            big = big @ big * 1e-4
        x2 = torch.empty_like(x)
        x2.copy_(x)
        got = hc.linear(x2, w, b, res)
    s.synchronize()
    same([got], [ref], "side stream")


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,H,Fw", [(3, 256, 640), (70, 264, 520), (33, 71, 129)])
def test_feed_forward_between_blocks_and_its_gradients(rows, H, Fw, dtype):
    """hclrmix block -> norm -> glu -> linear -> norm with the block's gate ->
    the next block's prologue, each step against fp64 on that step's own
    inputs; then the backward pass down to the block's output."""
    dt = T_OF[dtype]
    C, Rk = 4, 32
    K = C * H
    streams = rand((rows, K), dt, 1)
    ns = 1 + rand((K,), dt, 2, 0.1)
    wd, wu, wi = rand((K, Rk), dt, 3, K ** -0.5), rand((Rk, K), dt, 4, Rk ** -0.5), rand((K, C), dt, 5, K ** -0.5)
    attrs = dict(num_branches=C, epsilon=1e-6, reduction_scale=0.25, silu_alpha=0.25, gate_div=4.0, gate_mul=2.0)
    pre, post, so = hc.block(streams, ns, wd, wu, wi, **attrs)
    gate = post[:, 1]
    s1, s2, s3 = (1 + rand((H,), dt, 6 + i, 0.1) for i in range(3))
    fg, fu, fd = rand((H, Fw), dt, 10, H ** -0.5), rand((H, Fw), dt, 11, H ** -0.5), rand((Fw, H), dt, 12, Fw ** -0.5)
    r0, n0 = hc.residual_norm(pre, None, pre_scale=s1, post_norm=False)
    same([r0], [pre], "no residual, alpha 1")
    within(n0, *R.norm(pre, None, None, None, s1, False, 1.0, 1e-5)["normed"], "n0")
    h, g, u = hc.glu(n0, fg, fu, save=True)
    for got, name in zip((h, g, u), ("h", "g", "u")):
        within(got, *R.glu(n0, fg, fu, None, None, "silu")[name], name)
    y = hc.linear(h, fd)
    within(y, *R.linear(h, fd, None, None, "none")[:2], "y")
    r1, n1 = hc.residual_norm(y, pre, gate=gate, post_scale=s2, pre_scale=s3, alpha=0.5)
    ref = R.norm(y, pre, gate, s2, s3, True, 0.5, 1e-5)
    within(r1, *ref["residual_out"], "r1")
    within(n1, *ref["normed"], "n1")
    _, _, so2 = hc.block(so, ns, wd, wu, wi, n1, post, **attrs)
    prod = (post.float()[:, :, None] * n1.float()[:, None, :]).view(rows, K)
    same([so2], [(so.float() + prod).to(dt)], "prologue of the next block")
    # backward
    dr, dn = rand((rows, H), dt, 20), rand((rows, H), dt, 21)
    dy, dpre, dgate, ds2, ds3 = hc.residual_norm_backward(y, r1, dr, dn, gate=gate, post_scale=s2, pre_scale=s3, alpha=0.5)
    refb = R.norm_backward(y, r1, dr, dn, gate, s2, s3, True, 0.5, 1e-5)
    for got, name in zip((dy, dpre, dgate, ds2, ds3), NAMES):
        within(got, *refb[name], name)
    dh, dfd, _ = hc.linear_backward(h, fd, dy)
    refl = R.linear_backward(h, fd, dy, None, "none")
    within(dh, *refl["dx"], "dh")
    within(dfd, *refl["dw0"], "d_down")
    dn0, dfg, dfu, _, _ = hc.glu_backward(n0, fg, fu, g, u, dh)
    refg = R.glu_backward(n0, fg, fu, g, u, dh, "silu")
    for got, name in zip((dn0, dfg, dfu), GLU_NAMES):
        within(got, *refg[name], name)
    d0, _, _, _, ds1 = hc.residual_norm_backward(pre, r0, dpre, dn0, pre_scale=s1, post_norm=False)
    refn = R.norm_backward(pre, r0, dpre, dn0, None, None, s1, False, 1.0, 1e-5)
    within(d0, *refn["dy"], "d_pre_output")
    within(ds1, *refn["d_pre_scale"], "d_s1")


def test_product_gradients_by_differences():
    """fp32: <gradient, direction> against central differences of the forward calls."""
    m, k, n, e = 6, 24, 20, 2.0 ** -7
    x, w, b, _ = linear_inputs(m, k, n, torch.float32, 1)
    wu, bu = rand((k, n), torch.float32, 7, k ** -0.5), rand((n,), torch.float32, 8)
    c = rand((m, n), torch.float32, 9)
    for act in ("silu", "gelu", "gelu_tanh", "sigmoid"):
        t = {"x": x, "w": w, "b": b, "wu": wu, "bu": bu}
        lin = lambda v: (hc.linear(v["x"], v["w"], v["b"], activation=act) * c).double().sum().item()  # noqa: E731
        glu = lambda v: (hc.glu(v["x"], v["w"], v["wu"], v["b"], v["bu"], activation=act) * c).double().sum().item()  # noqa: E731
        _, p = hc.linear(x, w, b, activation=act, save=True)
        _, g, u = hc.glu(x, w, wu, b, bu, activation=act, save=True)
        gl = dict(zip(("x", "w", "b"), hc.linear_backward(x, w, c, p, activation=act, bias=True)))
        gg = dict(zip(("x", "w", "wu", "b", "bu"), hc.glu_backward(x, w, wu, g, u, c, activation=act, bias=True)))
        for f, grads in ((lin, gl), (glu, gg)):
            for name, gr in grads.items():
                d = rand(t[name].shape, torch.float32, 12, k ** -0.5 if name.startswith("w") else 1.0)
                up, down = dict(t), dict(t)
                up[name], down[name] = t[name] + e * d, t[name] - e * d
                num = (f(up) - f(down)) / (2 * e)
                ana = (gr.double() * d.double()).sum().item()
                # third derivatives of order one (times |u| and |d|^3, a few) per element, e^2 / 6 of them over
                # 120 elements with independent signs; fp32 noise of f over 2 e
                tol = 4 * e * e * 120 ** 0.5 + 2.0 ** -22 * 120 ** 0.5 / e + 1e-3 * abs(ana)
                assert abs(num - ana) <= tol, (act, name, num, ana, tol)


@pytest.mark.parametrize("scale", [2.0 ** -50, 2.0 ** 40])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hidden", [77, 520, 4104])
def test_norm_backward_of_tiny_and_huge_rows(hidden, dtype, scale):
    """No epsilon: 1 / rms^3 of such rows leaves fp32's range, the gradients do not."""
    dt = T_OF[dtype]
    y, r = rand((5, hidden), dt, 1, scale), rand((5, hidden), dt, 2, scale)
    dr, dn = None, rand((5, hidden), dt, 4)
    post, pre = rand((hidden,), dt, 5), rand((hidden,), dt, 6)
    got = hc.residual_norm_backward(y, r, dr, dn, post_scale=post, pre_scale=pre, alpha=0.5, epsilon=0.0)
    ref = R.norm_backward(y, r, dr, dn, None, post, pre, True, 0.5, 0.0)
    for g, name in zip(got, NAMES):
        if g is not None:
            within(g, *ref[name], name)


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_slopes_of_extreme_preactivations(dtype, act):
    """The type's largest and lowest values, and others whose square or cube is infinite in fp32."""
    dt = T_OF[dtype]
    m, k, n = 3, 24, 16
    top = torch.finfo(dt).max
    big = [0.0, -0.0, top, -top, top / 4, -top / 4, 40.0, -40.0, 300.0, -300.0] + ([] if dtype == "f16" else [1e20, -1e20, 1e13, -1e13])
    x, w, dy = rand((m, k), dt, 1), rand((k, n), dt, 2), rand((m, n), dt, 3)
    p = rand((m, n), dt, 4)
    p[1, :len(big)] = torch.tensor(big, dtype=torch.float64).to(dt)
    got = dict(zip(("dx", "dw0", "db0"), hc.linear_backward(x, w, dy, p, activation=act, bias=True)))
    ref = R.linear_backward(x, w, dy, p, act)
    for name, g in got.items():
        within(g, *ref[name], name)


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_nan_preactivation_reaches_its_gradients_only(dtype, act):
    dt = T_OF[dtype]
    m, k, n = 5, 24, 16
    x, w, wu, dy = rand((m, k), dt, 1), rand((k, n), dt, 2), rand((k, n), dt, 5), rand((m, n), dt, 3)
    p, u = rand((m, n), dt, 4), rand((m, n), dt, 6)
    p[2, 7] = math.nan
    rows, cols = torch.arange(m, device="cuda") == 2, torch.arange(n, device="cuda") == 7
    dx, dw, db = hc.linear_backward(x, w, dy, p, activation=act, bias=True)
    gx, gg, gu, bg, bu = hc.glu_backward(x, w, wu, p, u, dy, activation=act, bias=True)
    for d in (dx, gx):
        assert torch.equal(d.isnan(), rows[:, None].expand(m, k))
    for d in (dw, gg, gu):
        assert torch.equal(d.isnan(), cols[None].expand(k, n))
    for d in (db, bg, bu):
        assert torch.equal(d.isnan(), cols)


def test_two_streams_at_once():
    """Calls that overlap, each stream with a workspace of its own: the bits of calls alone."""
    x, w, b, _ = linear_inputs(8, 4096, 320, torch.bfloat16, 3)
    wu = rand((4096, 320), torch.bfloat16, 4, 4096 ** -0.5)
    dy = rand((8, 320), torch.bfloat16, 5)
    size = 32 << 20

    def step(ws):
        h, g, u = hc.glu(x, w, wu, save=True, workspace=ws)
        return (h,) + hc.glu_backward(x, w, wu, g, u, dy, bias=True, workspace=ws)[:3] + (hc.linear(x, w, b, workspace=ws),)

    ref = step(torch.zeros(size, dtype=torch.uint8, device="cuda"))
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        for s, ws in zip(streams, spaces):
            with torch.cuda.stream(s):
                got.append(step(ws))
    torch.cuda.synchronize()
    for g in got:
        same(g, ref, "two streams")


def test_the_same_tensor_as_several_inputs():
    dt = torch.bfloat16
    x, w = rand((33, 72), dt, 1), rand((72, 72), dt, 2, 72 ** -0.5)
    s = rand((72,), dt, 3)
    y = hc.linear(x, w, s, x, activation="silu")
    within(y, *R.linear(x, w, s, x, "silu")[:2], "y")
    h = hc.glu(x, w, w, s, s)
    within(h, *R.glu(x, w, w, s, s, "silu")["h"], "h")
    ref = R.norm(x, x, x, s, s, True, 1.0, 1e-5)
    for got, name in zip(hc.residual_norm(x, x, gate=x, post_scale=s, pre_scale=s), ("residual_out", "normed")):
        within(got, *ref[name], name)


def test_tensors_beyond_4_gib():
    """Rows, outputs and weights whose byte and element offsets pass 32 bits, at their ends."""
    dt = torch.bfloat16
    gen = torch.Generator(device="cuda").manual_seed(11)

    def big(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dt) * std

    # norms: 270,000 rows of 8,200
    rows, h = 270000, 8200
    y, res, gate, s = big(rows, h), big(rows, h), big(rows), 1 + big(h, std=0.1)
    assert y.numel() * 2 > 1 << 32
    pick = torch.tensor([0, 261902, 261903, 261904, rows - 1], device="cuda")
    at = lambda t: t.index_select(0, pick)  # noqa: E731
    r, n = hc.residual_norm(y, res, gate=gate, post_scale=s, pre_scale=s)
    ref = R.norm(at(y), at(res), at(gate), s, s, True, 1.0, 1e-5)
    within(at(r), *ref["residual_out"], "residual_out")
    within(at(n), *ref["normed"], "normed")
    dy, dr, dg, _, _ = hc.residual_norm_backward(y, r, res, n, gate=gate, post_scale=s, pre_scale=s)
    ref = R.norm_backward(at(y), at(r), at(res), at(n), at(gate), s, s, True, 1.0, 1e-5)
    for got, name in zip((dy, dr, dg), NAMES):
        within(at(got), *ref[name], name)
    del y, res, r, n, dy, dr
    # many rows in, out and as the contraction of the weight's gradient
    rows, k, n_ = 1050000, 2056, 24
    x, w, b = big(rows, k), big(k, n_, std=k ** -0.5), big(n_)
    assert x.numel() * 2 > 1 << 32
    pick = torch.tensor([0, 1044481, 1044494, rows - 1], device="cuda")
    y = hc.linear(x, w, b)
    within(at(y), *R.linear(at(x), w, b, None, "none")[:2], "y")
    dx, dw, db = hc.linear_backward(x, w, y, bias=True)
    within(at(dx), *R.linear_backward(at(x), w, at(y), None, "none")["dx"], "dx")
    exact = torch.zeros(k, n_, dtype=torch.float64, device="cuda")
    square = exact.clone()
    for i in range(0, rows, 65536):
        a, c = x[i:i + 65536].double(), y[i:i + 65536].double()
        exact += a.t().contiguous() @ c
        square += (a * a).t().contiguous() @ (c * c)
    # fp32 sums of `rows` products, as in R.product
    within(dw, exact, 8 * R.F * rows ** 0.5 * (square.sqrt() + exact.abs()), "dw")
    yd = y.double()
    within(db, yd.sum(0), (rows / 128 / 4 + 128 + 16) * R.F * yd.abs().sum(0), "db")
    del yd, dx
    wide = rand((n_, k), dt, 12, n_ ** -0.5)
    hh, g, u = hc.glu(y, wide, wide, save=True)
    ref = R.glu(at(y), wide, wide, None, None, "silu")
    for got, name in zip((hh, g, u), ("h", "g", "u")):
        within(at(got), *ref[name], name)
    del x, y, hh, g, u
    # a weight of 2^32 - 2^19 elements
    k, n_ = 65528, 65536
    x, w = big(2, k), big(k, n_, std=k ** -0.5)
    y = hc.linear(x, w)
    cols = torch.tensor([0, 1, 32767, 65535], device="cuda")
    within(y.index_select(1, cols), *R.linear(x, w.index_select(1, cols), None, None, "none")[:2], "y of a wide weight")
    dy = big(2, n_)
    dx, dw, _ = hc.linear_backward(x, w, dy)
    pick = torch.tensor([0, 32767, 32768, k - 1], device="cuda")
    ref = R.linear_backward(x.index_select(1, pick), at(w), dy, None, "none")
    within(dx.index_select(1, pick), *ref["dx"], "dx of a wide weight")
    within(at(dw), *ref["dw0"], "dw of a wide weight")
    del x, w, y, dx, dw
    torch.cuda.empty_cache()


@pytest.mark.parametrize("gate", ["row", "element"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,H", [(6, 6152), (530, 4104), (5, 5001)])
def test_norm_backward_of_two_chunks_a_thread(rows, H, dtype, gate):
    t = norm_inputs(rows, H, T_OF[dtype], gate, 7 + rows + H)
    dres, dn = rand((rows, H), T_OF[dtype], 5), rand((rows, H), T_OF[dtype], 6)
    ref = R.norm_backward(t["y"], t["residual"], dres, dn, t["gate"], t["post_scale"], t["pre_scale"], True, 0.5, 1e-6)
    for got, name in zip(_norm_back(t, t["residual"], dres, dn), NAMES):
        within(got, *ref[name], (name, rows, H, dtype, gate))


# Sizes that between them take every tile shape of every operand layout, whole and split, aligned and not.
TILE_SHAPES_16 = [(1, 776, 8200), (1, 2568, 8200), (1, 8200, 2568), (33, 4104, 200), (130, 520, 8200), (200, 200, 8200),
                  (200, 2568, 8200), (200, 8200, 2568), (200, 2056, 4104), (200, 4104, 2056), (257, 200, 10248),
                  (1025, 200, 8200), (1025, 8200, 200), (1025, 1544, 5128), (130, 10248, 8200), (33, 2569, 201),
                  (257, 201, 10249), (200, 1545, 4105), (200, 1545, 5129), (1025, 321, 4105), (1025, 4105, 201),
                  (16, 10249, 201), (200, 4105, 1545)]
TILE_SHAPES_32 = [(200, 521, 4105), (200, 201, 10249), (1025, 201, 4105), (257, 10249, 201), (200, 4105, 1033),
                  (200, 1033, 4105), (16, 8201, 201), (200, 520, 4104), (200, 200, 10248), (1025, 200, 4104), (200, 1032, 4104),
                  (257, 10248, 200), (200, 4104, 1032), (16, 8200, 200)]


@pytest.mark.parametrize("shape,dtype", [(s, d) for d in ("bf16", "f16") for s in TILE_SHAPES_16] + [(s, "f32") for s in TILE_SHAPES_32])
def test_every_tile_shape(shape, dtype):
    m, k, n = shape
    dt = T_OF[dtype]
    gen = torch.Generator(device="cuda").manual_seed(m + k + n)
    draw = lambda *s, std=1.0: (torch.randn(*s, generator=gen, device="cuda") * std).to(dt)  # noqa: E731
    x, w, wu, b, res = draw(m, k), draw(k, n, std=k ** -0.5), draw(k, n, std=k ** -0.5), draw(n), draw(m, n)
    g, u, dy = draw(m, n), draw(m, n), draw(m, n)
    within(hc.linear(x, w, b, res, activation="silu"), *R.linear(x, w, b, res, "silu")[:2], ("linear", shape, dtype))
    ref = R.glu(x, w, wu, b, None, "gelu")
    for got, name in zip(hc.glu(x, w, wu, b, None, activation="gelu", save=True), ("h", "g", "u")):
        within(got, *ref[name], ("glu", name, shape, dtype))
    ref = R.linear_backward(x, w, dy, g, "sigmoid")
    for got, name in zip(hc.linear_backward(x, w, dy, g, activation="sigmoid", bias=True), ("dx", "dw0", "db0")):
        within(got, *ref[name], ("linear_backward", name, shape, dtype))
    ref = R.glu_backward(x, w, wu, g, u, dy, "silu")
    for got, name in zip(hc.glu_backward(x, w, wu, g, u, dy, bias=True), GLU_NAMES):
        within(got, *ref[name], ("glu_backward", name, shape, dtype))
