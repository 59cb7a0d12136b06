"""GPU tests of the backward entry points with some of their outputs (and the
inputs that only those need) not given: the others have the bits of a call
with all of them."""
from __future__ import annotations

import itertools

import pytest
import torch

import hyper_connection_rank_amd as hc
from _ffn import T_OF, rand

pytestmark = pytest.mark.gpu
DTYPES = ["bf16", "f16", "f32"]
CODE = {"f32": 1, "f16": 10, "bf16": 16}


def compare(outs, full, label):
    torch.cuda.synchronize()
    for name, o in outs.items():
        t = torch.int32 if o.dtype == torch.float32 else torch.int16
        assert torch.equal(o.view(t), full[name].view(t)), (label, name)


def subsets(names):
    for n in range(1, len(names)):
        yield from itertools.combinations(names, n)


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,k,n", [(5, 72, 40), (70, 264, 1032), (70, 33, 77)])
def test_linear_backward_in_parts(m, k, n, dtype, act):
    dt = T_OF[dtype]
    x, w, dy = rand((m, k), dt, 1), rand((k, n), dt, 2), rand((m, n), dt, 3)
    pre = None if act == "none" else rand((m, n), dt, 4)
    p = hc.Product(m, k, n, 0, 0, 0, CODE[dtype], hc.ACTIVATIONS[act])
    ws = torch.zeros(hc.hclrmix_linear_backward_workspace_size(p), dtype=torch.uint8, device="cuda")
    full = dict(zip(("dx", "dw", "db"), hc.linear_backward(x, w, dy, pre, activation=act, bias=True)))
    for names in subsets(("dx", "dw", "db")):
        o = {c: torch.full_like(full[c], float("nan")) for c in names}
        hc.hclrmix_linear_backward(x if "dw" in o else None, w if "dx" in o else None, pre, dy, o.get("dx"), o.get("dw"),
                                   o.get("db"), ws, p)
        compare(o, full, (m, k, n, dtype, act, names))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,k,n", [(5, 72, 40), (70, 264, 1032), (70, 33, 77)])
def test_glu_backward_in_parts(m, k, n, dtype):
    dt = T_OF[dtype]
    x, wg, wu = rand((m, k), dt, 1), rand((k, n), dt, 2), rand((k, n), dt, 3)
    g, u, dh = rand((m, n), dt, 4), rand((m, n), dt, 5), rand((m, n), dt, 6)
    p = hc.Product(m, k, n, 0, 0, 0, CODE[dtype], hc.ACTIVATIONS["gelu"])
    ws = torch.zeros(hc.hclrmix_glu_backward_workspace_size(p), dtype=torch.uint8, device="cuda")
    order = ("dx", "dwg", "dwu", "dbg", "dbu")
    full = dict(zip(order, hc.glu_backward(x, wg, wu, g, u, dh, activation="gelu", bias=True)))
    for parts in subsets((("dx",), ("dwg", "dwu"), ("dbg", "dbu"))):
        names = sum(parts, ())
        o = {c: torch.full_like(full[c], float("nan")) for c in names}
        dx, dw = "dx" in o, "dwg" in o
        hc.hclrmix_glu_backward(x if dw else None, wg if dx else None, wu if dx else None, g, u, dh, *(o.get(c) for c in order),
                                ws, p)
        compare(o, full, (m, k, n, dtype, names))


@pytest.mark.parametrize("gate", ["row", "element"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,H", [(3, 264), (70, 77), (9, 2056), (6, 9001)])
def test_norm_backward_in_parts(rows, H, dtype, gate):
    dt, row = T_OF[dtype], gate == "row"
    y, r, dr, dn = (rand((rows, H), dt, i) for i in range(4))
    post, pre = rand((H,), dt, 5), rand((H,), dt, 6)
    gt = rand((rows,) if row else (rows, H), dt, 7)
    p = hc.NormProblem(rows, H, int(row), CODE[dtype], hc.GATE_ROW if row else hc.GATE_ELEMENT, 1, 0, 0.5, 1e-6)
    ws = torch.zeros(hc.hclrmix_residual_norm_workspace_size(p), dtype=torch.uint8, device="cuda")
    order = ("dy", "d_residual", "d_gate", "d_post", "d_pre")
    full = dict(zip(order, hc.residual_norm_backward(y, r, dr, dn, gate=gt, post_scale=post, pre_scale=pre, alpha=0.5,
                                                     epsilon=1e-6)))
    for names in subsets(order):
        o = {c: torch.full_like(full[c], float("nan")) for c in names}
        sums = "d_post" in o or "d_pre" in o
        hc.hclrmix_residual_norm_backward(y, r, gt, post, pre, dr, dn, *(o.get(c) for c in order), ws if sums else None, p)
        compare(o, full, (rows, H, dtype, gate, names))
