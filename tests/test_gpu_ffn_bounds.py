"""GPU tests of where the feed-forward operators write: every output and an
exactly sized workspace lie inside larger buffers of a pattern, which has to be
unchanged around them, and every output element is written (they start as NaN)."""
from __future__ import annotations

import pytest
import torch

import hyper_connection_rank_amd as hc
from _ffn import T_OF, rand

pytestmark = pytest.mark.gpu
DTYPES = ["bf16", "f16", "f32"]
CODE = {"f32": 1, "f16": 10, "bf16": 16}
PAD, PATTERN = 8192, 0xA5


class Inside:
    """A tensor in the middle of a buffer of the pattern, `off` elements past a 16-byte boundary; NaN at first."""

    def __init__(self, shape, dt, off=0):
        es = torch.finfo(dt).bits // 8 if dt.is_floating_point else 1
        n = 1
        for s in shape:
            n *= s
        self.lo, self.hi = PAD + off * es, PAD + (off + n) * es
        self.buf = torch.full((self.hi + PAD + 16,), PATTERN, dtype=torch.uint8, device="cuda")
        self.buf[self.lo:self.hi] = 0xFF
        self.t = self.buf[self.lo:self.hi].view(dt).view(shape)
        assert self.t.data_ptr() % 16 == off * es % 16

    def check(self, label):
        for part, where in ((self.buf[:self.lo], "before"), (self.buf[self.hi:], "behind")):
            bad = (part != PATTERN).nonzero()
            assert not len(bad), f"{label}: {len(bad)} bytes {where} it are written, the first at {bad[0].item()}"


def workspace(need):
    ws = Inside((need,), torch.uint8)
    ws.t[:4096] = 0
    return ws


def checked(call, outs, ws, ref, label):
    """Runs the call and looks at the outputs {name: Inside or None} and the workspace; ref: their values."""
    call()
    torch.cuda.synchronize()
    if ws is not None:
        ws.check((label, "workspace"))
        assert not ws.t[:4096].any(), (label, "counters")
    for (name, o), r in zip(outs.items(), ref):
        if o is None:
            assert r is None, (label, name)
            continue
        o.check((label, name))
        i = torch.int32 if r.dtype == torch.float32 else torch.int16
        assert torch.equal(o.t.contiguous().view(i), r.contiguous().view(i)), (label, name, "values")


# rows, in, out: single elements, ragged edges of every tile, split contractions, whole and split tiles in one launch
PRODUCTS = [(1, 1, 1), (3, 33, 17), (17, 128, 136), (1, 2568, 8200), (5, 8200, 72), (33, 4104, 200), (129, 320, 264),
            (300, 1003, 777), (257, 201, 10249), (718, 72, 64), (1025, 200, 4104), (1229, 8264, 904), (2224, 200, 3601)]


@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,k,n", PRODUCTS)
def test_products_write_their_outputs_alone(m, k, n, dtype, off):
    dt = T_OF[dtype]
    print(f"[bounds] {m} {k} {n} {dtype} off {off}", flush=True)
    x, w, wu = rand((m, k), dt, 1), rand((k, n), dt, 2, k ** -0.5), rand((k, n), dt, 3, k ** -0.5)
    b, res, g, u, dy = rand((n,), dt, 4), rand((m, n), dt, 5), rand((m, n), dt, 6), rand((m, n), dt, 7), rand((m, n), dt, 8)
    p = hc.Product(m, k, n, 0, 0, 0, CODE[dtype], hc.ACTIVATIONS["gelu"])
    mk = lambda **shapes: {name: Inside(s, dt, off) for name, s in shapes.items()}  # noqa: E731

    o, ws = mk(y=(m, n), preact=(m, n)), workspace(hc.hclrmix_linear_workspace_size(p))
    checked(lambda: hc.hclrmix_linear(x, w, b, res, o["y"].t, o["preact"].t, ws.t, p), o, ws,
            hc.linear(x, w, b, res, activation="gelu", save=True), "linear")

    o, ws = mk(h=(m, n), g=(m, n), u=(m, n)), workspace(hc.hclrmix_glu_workspace_size(p))
    checked(lambda: hc.hclrmix_glu(x, w, wu, b, None, o["h"].t, o["g"].t, o["u"].t, ws.t, p), o, ws,
            hc.glu(x, w, wu, b, activation="gelu", save=True), "glu")

    o, ws = mk(dx=(m, k), dw=(k, n), db=(n,)), workspace(hc.hclrmix_linear_backward_workspace_size(p))
    checked(lambda: hc.hclrmix_linear_backward(x, w, g, dy, o["dx"].t, o["dw"].t, o["db"].t, ws.t, p), o, ws,
            hc.linear_backward(x, w, dy, g, activation="gelu", bias=True), "linear_backward")

    o = mk(dx=(m, k), dwg=(k, n), dwu=(k, n), dbg=(n,), dbu=(n,))
    ws = workspace(hc.hclrmix_glu_backward_workspace_size(p))
    checked(lambda: hc.hclrmix_glu_backward(x, w, wu, g, u, dy, *(v.t for v in o.values()), ws.t, p), o, ws,
            hc.glu_backward(x, w, wu, g, u, dy, activation="gelu", bias=True), "glu_backward")


# rows, hidden: one row per wave and per workgroup, one to four chunks a thread, odd ends, several rows per workgroup
NORMS = [(1, 1), (3, 7), (6, 264), (9, 511), (5, 2057), (1030, 2560), (1025, 1001), (2, 8200), (7, 12289), (6, 20001),
         (5, 32768)]


@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("gate", ["row", "element"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,H", NORMS)
def test_norms_write_their_outputs_alone(rows, H, dtype, gate, off):
    dt = T_OF[dtype]
    print(f"[bounds] norm {rows} {H} {dtype} {gate} off {off}", flush=True)
    y, res, dn = rand((rows, H), dt, 1), rand((rows, H), dt, 2), rand((rows, H), dt, 3)
    post, pre = 1 + rand((H,), dt, 4, 0.1), 1 + rand((H,), dt, 5, 0.1)
    row = gate == "row"
    gt = rand((rows,) if row else (rows, H), dt, 6)
    p = hc.NormProblem(rows, H, int(row), CODE[dtype], hc.GATE_ROW if row else hc.GATE_ELEMENT, 1, 0, 0.5, 1e-6)
    mk = lambda **shapes: {name: Inside(s, dt, off) for name, s in shapes.items()}  # noqa: E731
    # rows whose outputs are not 16-byte aligned are summed in the same order: by eight elements a lane
    o = mk(residual_out=(rows, H), normed=(rows, H))
    checked(lambda: hc.hclrmix_residual_norm(y, res, gt, post, pre, o["residual_out"].t, o["normed"].t, p), o, None,
            hc.residual_norm(y, res, gate=gt, post_scale=post, pre_scale=pre, alpha=0.5, epsilon=1e-6), "norm")
    o, ws = mk(dy=(rows, H), dr=(rows, H), dg=tuple(gt.shape), dpost=(H,), dpre=(H,)), workspace(
        hc.hclrmix_residual_norm_workspace_size(p))
    checked(lambda: hc.hclrmix_residual_norm_backward(y, res, gt, post, pre, dn, dn, *(v.t for v in o.values()), ws.t, p), o, ws,
            hc.residual_norm_backward(y, res, dn, dn, gate=gt, post_scale=post, pre_scale=pre, alpha=0.5, epsilon=1e-6), "backward")


@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("dtype", DTYPES)
def test_zero_rows_write_zeros_over_what_was_there(dtype, off):
    dt, k, n = T_OF[dtype], 33, 77
    empty = lambda c: torch.empty(0, c, dtype=dt, device="cuda")  # noqa: E731
    mk = lambda **shapes: {name: Inside(s, dt, off) for name, s in shapes.items()}  # noqa: E731
    w = torch.ones(k, n, dtype=dt, device="cuda")
    p = hc.Product(0, k, n, 0, 0, 0, CODE[dtype], hc.ACTIVATIONS["silu"])
    zeros = lambda o: [torch.zeros_like(v.t) for v in o.values()]  # noqa: E731
    o, ws = mk(dw=(k, n), db=(n,)), workspace(hc.hclrmix_linear_backward_workspace_size(p))
    checked(lambda: hc.hclrmix_linear_backward(empty(k), w, empty(n), empty(n), empty(k), o["dw"].t, o["db"].t, ws.t, p), o, ws,
            zeros(o), "linear_backward")
    o, ws = mk(dwg=(k, n), dwu=(k, n), dbg=(n,), dbu=(n,)), workspace(hc.hclrmix_glu_backward_workspace_size(p))
    checked(lambda: hc.hclrmix_glu_backward(empty(k), w, w, empty(n), empty(n), empty(n), empty(k), *(v.t for v in o.values()),
                                            ws.t, p), o, ws, zeros(o), "glu_backward")
    q = hc.NormProblem(0, k, 0, CODE[dtype], hc.GATE_NONE, 1, 0, 1.0, 1e-6)
    s = torch.ones(k, dtype=dt, device="cuda")
    o, ws = mk(dpost=(k,), dpre=(k,)), workspace(hc.hclrmix_residual_norm_workspace_size(q))
    e = empty(k)
    checked(lambda: hc.hclrmix_residual_norm_backward(e, e, None, s, s, e, e, empty(k), empty(k), None, o["dpost"].t, o["dpre"].t,
                                                      ws.t, q), o, ws, zeros(o), "norm_backward")
