"""GPU tests of linear, glu and their gradients at sizes that take the plans
(tile shape, alignment, tiles whole, split or both in one launch) that the
other tests' sizes do not; tests/test_ffn_plan.py shows that together they take
every plan of the operators' range."""
from __future__ import annotations

import pytest
import torch

import _ffn as R
import hyper_connection_rank_amd as hc
from _ffn import T_OF, within

pytestmark = pytest.mark.gpu

PLANS_16 = [(1, 72, 217), (7183, 385, 72), (924, 4144, 72), (66, 7368, 320), (266, 80, 11928), (304, 335, 11032),
            (4651, 1736, 65), (1728, 80, 4176), (1298, 71, 8240), (1198, 6759, 195), (2224, 200, 3601),
            (1233, 160, 8248), (693, 504, 10888), (1463, 11032, 760), (4857, 3413, 240), (347, 11061, 2304),
            (6633, 560, 1368), (2081, 11512, 296), (451, 2152, 8352), (495, 2648, 6240), (6603, 529, 2472),
            (6268, 560, 2592), (1714, 10008, 1784), (160, 2080, 10928), (4094, 136, 11800), (1970, 1312, 8912),
            (718, 72, 64), (3695, 144, 5744)]
PLANS_32 = [(1, 283, 11349), (162, 64, 81), (1, 104, 8304), (1, 8720, 64), (1, 11168, 65), (199, 167, 8537),
            (195, 184, 8640), (267, 64, 10272), (602, 64, 5165), (303, 10881, 75), (269, 10936, 216), (267, 264, 11464),
            (441, 392, 8197), (753, 11248, 67), (4844, 1688, 72), (168, 6896, 1176), (265, 11808, 711), (2586, 3208, 165),
            (5499, 1493, 168), (5155, 165, 1663), (3880, 184, 2144)]
# A backward pass whose weights' gradients are whole and split 256 x 256 tiles in one launch, the split ones in the
# second weight's.
PLANS_16 += [(1229, 8264, 904)]


@pytest.mark.parametrize("shape,dtype", [(s, d) for d in ("bf16", "f16") for s in PLANS_16] + [(s, "f32") for s in PLANS_32])
def test_every_plan(shape, dtype):
    m, k, n = shape
    dt = T_OF[dtype]
    gen = torch.Generator(device="cuda").manual_seed(3 * m + k + n)
    draw = lambda *s, std=1.0: (torch.randn(*s, generator=gen, device="cuda") * std).to(dt)  # noqa: E731
    x, w, wu, b, res = draw(m, k), draw(k, n, std=k ** -0.5), draw(k, n, std=k ** -0.5), draw(n), draw(m, n)
    g, u, dy = draw(m, n), draw(m, n), draw(m, n)
    print(f"[plans] {shape} {dtype}", flush=True)
    within(hc.linear(x, w, b, res, activation="gelu_tanh"), *R.linear(x, w, b, res, "gelu_tanh")[:2], ("linear", shape, dtype))
    ref = R.glu(x, w, wu, None, b, "silu")
    for got, name in zip(hc.glu(x, w, wu, None, b, activation="silu", save=True), ("h", "g", "u")):
        within(got, *ref[name], ("glu", name, shape, dtype))
    ref = R.linear_backward(x, w, dy, g, "relu")
    for got, name in zip(hc.linear_backward(x, w, dy, g, activation="relu", bias=True), ("dx", "dw0", "db0")):
        within(got, *ref[name], ("linear_backward", name, shape, dtype))
    ref = R.glu_backward(x, w, wu, g, u, dy, "gelu")
    for got, name in zip(hc.glu_backward(x, w, wu, g, u, dy, activation="gelu", bias=True), ("dx", "dw0", "dw1", "db0", "db1")):
        within(got, *ref[name], ("glu_backward", name, shape, dtype))
