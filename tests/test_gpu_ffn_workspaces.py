"""GPU tests of the feed-forward operators' workspaces: one that is sized for
the most rows and full of leftovers, and graphs captured without one."""
from __future__ import annotations

import pytest
import torch

import hyper_connection_rank_amd as hc
from _ffn import T_OF, rand

pytestmark = pytest.mark.gpu


def same(got, ref, label):
    for i, (a, b) in enumerate(zip(got, ref)):
        assert (a is None) == (b is None), (label, i)
        if a is not None:
            t = torch.int32 if a.dtype == torch.float32 else torch.int16
            assert torch.equal(a.contiguous().view(t), b.contiguous().view(t)), (label, i)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("k,n", [(2560, 1032), (1032, 2560), (777, 513)])
def test_a_workspace_for_the_most_rows_serves_fewer(k, n, dtype):
    """As a prompt is followed by single tokens. The counters stay zero from call to call."""
    dt, most = T_OF[dtype], 1100
    x, dy = rand((most, k), dt, 1), rand((most, n), dt, 2)
    w, wu = rand((k, n), dt, 3, k ** -0.5), rand((k, n), dt, 4, k ** -0.5)
    s = 1 + rand((k,), dt, 5, 0.1)

    def dirty(need):
        ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
        ws[:4096] = 0
        return ws

    calls = [(dirty(hc.linear_workspace_size(most, k, n, dt)), lambda r, ws: (hc.linear(x[:r], w, workspace=ws),)),
             (dirty(hc.glu_workspace_size(most, k, n, dt)), lambda r, ws: (hc.glu(x[:r], w, wu, workspace=ws),)),
             (dirty(hc.linear_workspace_size(most, k, n, dt, backward=True)),
              lambda r, ws: hc.linear_backward(x[:r], w, dy[:r], dy[:r], activation="silu", bias=True, workspace=ws)),
             (dirty(hc.glu_workspace_size(most, k, n, dt, backward=True)),
              lambda r, ws: hc.glu_backward(x[:r], w, wu, dy[:r], dy[:r], dy[:r], bias=True, workspace=ws)),
             (dirty(hc.residual_norm_workspace_size(most, k, dt)),
              lambda r, ws: hc.residual_norm_backward(x[:r], x[:r], x[:r], x[:r], post_scale=s, pre_scale=s, workspace=ws))]
    for r in (most, 1025, 513, 300, 65, 17, 16, 5, 3, 1):
        for i, (ws, f) in enumerate(calls):
            same(f(r, ws), f(r, None), (k, n, dtype, r, i))
            assert not ws[:4096].any(), (r, i)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_graph_of_calls_without_workspaces_replays(dtype):
    """Each call's own workspace is cleared by the graph; eager work between the replays."""
    dt = T_OF[dtype]
    m, k, n = 5, 2560, 264
    w, wu, wd = rand((k, n), dt, 1, k ** -0.5), rand((k, n), dt, 2, k ** -0.5), rand((n, k), dt, 3, n ** -0.5)
    s = 1 + rand((k,), dt, 4, 0.1)
    x = rand((m, k), dt, 5)

    def step(x_):
        r, v = hc.residual_norm(x_, x_ * 0.5, pre_scale=s, post_scale=s)
        h, g, u = hc.glu(v, w, wu, save=True)
        y = hc.linear(h, wd, None, r)
        dh, dwd, _ = hc.linear_backward(h, wd, y)
        dv, dwg, dwu, dbg, dbu = hc.glu_backward(v, w, wu, g, u, dh, bias=True)
        return (y, dwd, dwg, dwu, dbg, dbu) + hc.residual_norm_backward(x_, r, y, dv, post_scale=s, pre_scale=s)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(x)
    for i in range(4):
        new = rand((m, k), dt, 20 + i)
        x.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        got = [None if o is None else o.clone() for o in outs]
        same(got, step(new), ("replay", i))
        torch.cuda.synchronize()
