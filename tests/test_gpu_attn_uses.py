"""GPU tests of how the attention operators are used: where they write, captured graphs, streams, offsets beyond 32 bits,
extreme values, gradients by differences, and a layer of them in a row."""
from __future__ import annotations

import math
import random

import pytest
import torch

import _attn as ref
import hyper_connection_rank_amd as hc
from _ffn import T_OF, U, rand, within
from test_gpu_attn import TYPES, cache, check, make
from test_gpu_ffn_bounds import Inside, workspace

pytestmark = pytest.mark.gpu


def starts_of(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- where they write

@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("dim,off", [(64, 0), (96, 0), (128, 0), (200, 0), (57, 0), (64, 1), (128, 3)])
def test_only_the_outputs_are_written(dt, dim, off):
    """Packed sequences with rows before, and behind them that belong to none: those keep what they held."""
    t, es = T_OF[dt], 4 if dt == "f32" else 2
    lens, heads, kv, lead, tail = [70, 0, 33, 129], 4, 2, 3, 5
    n = lead + sum(lens) + tail
    st = starts_of(lens) + lead
    q, k, v, do = (rand((n, h, dim), t, i) for i, h in enumerate((heads, kv, kv, heads)))
    kw = dict(q_starts=st, window=50, sinks=2)
    want, lse = hc.attention(q, k, v, save=True, **kw)
    ws = workspace(hc.attention_workspace_size(4, n, n, heads, kv, dim, t, packed=True))
    out = Inside((n, heads, dim), t, off)
    hc.attention(q, k, v, out=out.t, workspace=ws.t, **kw)
    out.check("out")
    ws.check("workspace")
    live = slice(lead, n - tail)
    assert torch.equal(out.t[live], want[live])
    raw = out.buf[out.lo:out.hi].view(n, heads * dim * es)
    assert (raw[:lead] == 0xFF).all() and (raw[n - tail:] == 0xFF).all()
    assert not want[:lead].any() and not want[n - tail:].any() and not lse[n - tail:].any()
    grads = hc.attention_backward(q, k, v, want, lse, do, **kw)
    ws = workspace(hc.attention_workspace_size(4, n, n, heads, kv, dim, t, packed=True, backward=True))
    got = [Inside(x.shape, t, off) for x in grads]
    hc.attention_backward(q, k, v, want, lse, do, grads=[x.t for x in got], workspace=ws.t, **kw)
    ws.check("workspace")
    for x, y in zip(got, grads):
        x.check("grads")
        assert torch.equal(x.t[live], y[live])
        raw = x.buf[x.lo:x.hi].view(n, -1)
        assert (raw[:lead] == 0xFF).all() and (raw[n - tail:] == 0xFF).all()
        assert not y[:lead].any() and not y[n - tail:].any()


@pytest.mark.parametrize("dt", TYPES)
def test_split_rows_write_their_outputs_alone(dt):
    """Enough rows for the backward pass to split them over workgroups, whose parts are joined."""
    t, heads, dim = T_OF[dt], 8, 64
    q, k, v = make(dt, 1, 1500, 700, heads, 1, dim)
    do = rand(tuple(q.shape), t, 9)
    out, lse = hc.attention(q, k, v, save=True, causal=False)
    want = ref.attention_backward(q, k, v, out, lse, do, causal=False)
    ws = workspace(hc.attention_workspace_size(1, 1500, 700, heads, 1, dim, t, backward=True))
    for some in ((True, True, True), (False, True, False), (False, False, True), (True, False, False)):
        got = [Inside(x.shape, t) if w else None for x, w in zip((q, k, v), some)]
        hc.attention_backward(q, k, v, out, lse, do, causal=False, grads=[x and x.t for x in got], workspace=ws.t)
        ws.check("workspace")
        for x, n in zip(got, ("dq", "dk", "dv")):
            if x is not None:
                x.check(n)
                within(x.t, *want[n], f"{dt} {some} {n}")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("dim,off", [(64, 0), (128, 0), (256, 0), (57, 0), (64, 1)])
def test_paged_writes_its_output_alone(dt, dim, off):
    t, lens = T_OF[dt], [3000, 0, 1, 517]
    kc, vc, table, n = cache(dt, lens, 2, dim, 16)
    q = rand((4, 6, dim), t, 3)
    want = hc.paged_attention(q, kc, vc, table, n)
    out = Inside(q.shape, t, off)
    ws = workspace(hc.paged_attention_workspace_size(4, table.shape[1], 16, 6, 2, dim, t))
    hc.paged_attention(q, kc, vc, table, n, out=out.t, workspace=ws.t)
    out.check("out")
    ws.check("workspace")
    assert torch.equal(out.t, want)


@pytest.mark.parametrize("dt", TYPES)
def test_wrong_starts_stay_inside_the_tensors(dt):
    """Starts that descend or lie outside: what comes out is unspecified, but nothing else is written."""
    t, n, heads, dim = T_OF[dt], 150, 4, 64
    q, k, v, do = (rand((n, heads, dim), t, i) for i in range(4))
    for st in ([0, 100, 20, 150], [-7, 40, 10 ** 9], [150, 0], [2 ** 31 - 1, -2 ** 31, 5], [60, 60, 60]):
        s = torch.tensor(st, dtype=torch.int32, device="cuda")
        out = Inside(q.shape, t)
        hc.attention(q, k, v, out=out.t, q_starts=s)
        out.check(f"{st}")
        lse = torch.zeros(n, heads, device="cuda")
        grads = [Inside(q.shape, t) for _ in range(3)]
        ws = workspace(hc.attention_workspace_size(len(st) - 1, n, n, heads, heads, dim, t, packed=True, backward=True))
        hc.attention_backward(q, k, v, q, lse, do, q_starts=s, grads=[g.t for g in grads], workspace=ws.t)
        ws.check(f"{st}")
        for g in grads:
            g.check(f"{st}")


# ---------------------------------------------------------------- graphs, streams, workspaces

@pytest.mark.parametrize("dt", TYPES)
def test_a_decode_step_in_a_graph(dt):
    """map, store, attend captured once and replayed step after step, its counters moved on by the graph itself; beside it an
    eager run of the same steps."""
    t, heads, kv, dim, page, batch = T_OF[dt], 8, 2, 64, 16, 3
    free = torch.randperm(60, generator=torch.Generator().manual_seed(2)).to(torch.int32).cuda()
    kvs = [(rand((batch, kv, dim), t, 10 + i), rand((batch, kv, dim), t, 50 + i), rand((batch, heads, dim), t, 90 + i)) for i in range(6)]

    class Side:
        def __init__(self):
            self.kc, self.vc = (torch.zeros(60, page, kv, dim, dtype=t, device="cuda") for _ in range(2))
            self.table = torch.zeros(batch, 9, dtype=torch.int32, device="cuda")
            self.cached = torch.tensor([0, 15, 130], dtype=torch.int32, device="cuda")
            self.table[1, 0], self.table[2] = 59, torch.arange(50, 59)
            self.first = torch.zeros(1, dtype=torch.int32, device="cuda")
            self.fresh = torch.ones(batch, dtype=torch.int32, device="cuda")
            self.k, self.v, self.q = (x.clone() for x in kvs[0])
            self.ws = torch.zeros(hc.paged_attention_workspace_size(batch, 9, page, heads, kv, dim, t), dtype=torch.uint8, device="cuda")

        def step(self):
            starts, lengths, positions, slots, taken = hc.page_map(self.cached, self.fresh, self.table, free, page_size=page,
                                                                   tokens=batch, free_start=self.first)
            hc.cache_store(self.k, self.v, self.kc, self.vc, slots)
            self.out = hc.paged_attention(self.q, self.kc, self.vc, self.table, lengths, workspace=self.ws)
            self.cached.copy_(lengths)
            self.first.add_(taken[-1:])

    graph_side, eager = Side(), Side()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    warm = Side()
    with torch.cuda.stream(side):
        warm.step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graph_side.step()
    for k, v, q in kvs:
        for s in (graph_side, eager):
            s.k.copy_(k), s.v.copy_(v), s.q.copy_(q)
        eager.step()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(graph_side.out, eager.out)
        assert torch.equal(graph_side.table, eager.table) and torch.equal(graph_side.kc, eager.kc)
    within(eager.out, *ref.paged(eager.q, eager.kc, eager.vc, eager.table, eager.cached), "last step")


@pytest.mark.parametrize("dt", TYPES)
def test_training_in_graphs(dt):
    """Forward and backward captured with a workspace each, two graphs replayed in turn with new inputs between eager calls."""
    t, heads, kv, dim = T_OF[dt], 4, 1, 64
    lens = [300, 0, 401, 77]
    st, n = starts_of(lens), sum(lens) + 2

    def step(q, k, v, do, ws):
        out, lse = hc.attention(q, k, v, save=True, q_starts=st, window=100, sinks=3, workspace=ws)
        return (out, lse) + hc.attention_backward(q, k, v, out, lse, do, q_starts=st, window=100, sinks=3, workspace=ws)

    def inputs(seed):
        return [rand((n, h, dim), t, seed + i) for i, h in enumerate((heads, kv, kv, heads))]
    graphs = []
    for i in range(2):
        x = inputs(i)
        ws = torch.zeros(max(hc.attention_workspace_size(4, n, n, heads, kv, dim, t, packed=True, backward=b) for b in (False, True)),
                         dtype=torch.uint8, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(*x, ws)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(*x, ws)
        graphs.append((g, x, out, ws))
    for seed in range(40, 46):
        for i, (g, x, out, _) in enumerate(graphs):
            new = inputs(seed + 100 * i)
            want = step(*new, None)
            for a, b in zip(x, new):
                a.copy_(b)
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), (seed, i)


@pytest.mark.parametrize("dt", TYPES)
def test_two_streams_at_once(dt):
    q, k, v = make(dt, 1, 700, 700, 8, 2, 64)
    do = rand(tuple(q.shape), q.dtype, 5)
    kc, vc, table, n = cache(dt, [3000, 777], 2, 64, 16)
    qp = rand((2, 8, 64), q.dtype, 6)

    def work():
        out, lse = hc.attention(q, k, v, save=True)
        return (out, hc.paged_attention(qp, kc, vc, table, n)) + hc.attention_backward(q, k, v, out, lse, do)
    want = work()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(work())
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))


def test_one_workspace_after_another_operator():
    """The operators share a workspace with the others and leave its counters zero."""
    dt = torch.bfloat16
    x, w = rand((3, 5120), dt, 1), rand((5120, 264), dt, 2)
    q, k, v = make("bf16", 1, 900, 900, 4, 1, 64)
    kc, vc, table, n = cache("bf16", [5000], 1, 64, 16)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    want = hc.linear(x, w)
    for _ in range(2):
        ws[4096:].fill_(0xFF)
        out, lse = hc.attention(q, k, v, save=True, workspace=ws)
        got = hc.attention_backward(q, k, v, out, lse, out, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, hc.attention_backward(q, k, v, out, lse, out)))
        p = hc.paged_attention(q[0, :1], kc, vc, table, n, workspace=ws)
        assert torch.equal(p, hc.paged_attention(q[0, :1], kc, vc, table, n))
        assert not ws[:4096].any()
        assert torch.equal(hc.linear(x, w, workspace=ws), want)


# ---------------------------------------------------------------- far offsets

def test_a_cache_beyond_32_bits():
    """Pages whose bytes lie beyond 2^32, and slots there."""
    t, page, kv, dim = torch.bfloat16, 16, 8, 128
    pages = (1 << 32) // (page * kv * dim * 2) + 300
    kc, vc = (torch.empty(pages, page, kv, dim, dtype=t, device="cuda") for _ in range(2))
    table = torch.stack([torch.arange(pages - 1, pages - 41, -1), torch.arange(0, 40)]).to(torch.int32).cuda()
    n = torch.tensor([600, 635], dtype=torch.int32, device="cuda")
    for b in range(2):
        k, v = rand((640, kv, dim), t, 1 + b), rand((640, kv, dim), t, 3 + b)
        j = torch.arange(640, device="cuda")
        slots = (table[b].long()[j // page] * page + j % page).to(torch.int32)
        hc.cache_store(k, v, kc, vc, slots)
        assert torch.equal(kc[table[b].long()].view(640, kv, dim), k)
    q = rand((2, 16, dim), t, 7)
    within(hc.paged_attention(q, kc, vc, table, n), *ref.paged(q, kc, vc, table, n), "far pages")


def test_rows_beyond_32_bits():
    """Tokens a megabyte and more apart: offsets from the first beyond 2^32 bytes."""
    t, n, dim = torch.float16, 2500, 64
    wide = torch.empty(n, 1 << 20, dtype=t, device="cuda")
    parts = [rand((n, 2, dim), t, i) for i in range(4)]
    views = []
    for i, p in enumerate(parts):
        views.append(wide[:, 4096 * i:4096 * i + 2 * dim].view(n, 2, dim))
        views[-1].copy_(p)
    out, lse = hc.attention(*parts[:3], save=True, window=200)
    o2, l2 = hc.attention(*views[:3], save=True, window=200)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    grads = [wide[:, 65536 + 4096 * i:65536 + 4096 * i + 2 * dim].view(n, 2, dim) for i in range(3)]
    want = hc.attention_backward(*parts[:3], out, lse, parts[3], window=200)
    got = hc.attention_backward(*views[:3], out, lse, views[3], window=200, grads=grads)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    eo, bo, _, _ = ref.attention(*parts[:3], window=200)
    within(out, eo, bo, "far rows")


# ---------------------------------------------------------------- values

@pytest.mark.parametrize("dt", TYPES)
def test_scores_that_grow_and_fall(dt):
    """Maxima that grow at every tile of keys by more and by less than the sums wait for, and that come first."""
    for step in (0.02, 0.2, 3.0, -0.02, -0.2, -3.0):
        q, k, v = make(dt, 1, 70, 1000, 2, 2, 64)
        q.zero_()
        q[..., 0] = 1
        k[..., 0] = (torch.arange(1000, device="cuda") * step).clamp(-500, 500).to(k.dtype)[None, :, None]
        check(q, k, v, f"{dt} {step}", causal=False, scale=1.0)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("size", [1e-6, 1e-3, 30.0])
def test_gradients_of_any_size(dt, size):
    """d_out small and large: fp16's dS keeps its accuracy by a power of two of its own (the bound counts 2^-36 of the
    largest value before)."""
    q, k, v = make(dt, 1, 600, 600, 4, 2, 64)
    out, lse = hc.attention(q, k, v, save=True)
    do = (rand(tuple(q.shape), torch.float32, 8) * size).to(q.dtype)
    do[:, ::3] *= 0.01
    got = hc.attention_backward(q, k, v, out, lse, do)
    want = ref.attention_backward(q, k, v, out, lse, do)
    for n, g in zip(("dq", "dk", "dv"), got):
        within(g, *want[n], f"{dt} {size} {n}")


@pytest.mark.parametrize("dt", TYPES)
def test_rows_of_no_sequence_may_hold_anything(dt):
    t, dim = T_OF[dt], 64
    lens = [40, 90]
    n = 5 + sum(lens) + 70
    st = starts_of(lens) + 5
    x = [rand((n, h, dim), t, i) for i, h in enumerate((4, 2, 2, 4))]
    kw = dict(q_starts=st)
    out, lse = hc.attention(*x[:3], save=True, **kw)
    want = hc.attention_backward(*x[:3], out, lse, x[3], **kw)
    for bad in (math.nan, math.inf, torch.finfo(t).min):
        y = [a.clone() for a in x]
        for a in y:
            a[:5], a[135:] = bad, bad
        o2, l2 = hc.attention(*y[:3], save=True, **kw)
        assert torch.equal(out, o2) and torch.equal(lse, l2)
        l2[:5], l2[135:], o2[:5], o2[135:] = bad if abs(bad) == math.inf or bad != bad else -1e38, math.nan, math.nan, math.nan
        assert all(torch.equal(a, b) for a, b in zip(want, hc.attention_backward(*y[:3], o2, l2, y[3], **kw)))


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (37, 0), (37, 5)])
def test_unseen_keys_of_a_cache_may_hold_anything(dt, window, sinks):
    t, lens, page = T_OF[dt], [200, 3, 71], 16
    kc, vc, table, n = cache(dt, lens, 2, 64, page)
    q = rand((3, 4, 64), t, 3)
    want = hc.paged_attention(q, kc, vc, table, n, window=window, sinks=sinks)
    seen = torch.zeros(kc.shape[:2], dtype=torch.bool)
    for b, m in enumerate(lens):
        for j in range(m):
            if not window or j >= m - window or j < sinks:
                seen[table[b, j // page], j % page] = True
    for bad in (math.nan, math.inf, -math.inf, torch.finfo(t).max):
        k2, v2 = kc.clone(), vc.clone()
        k2[~seen], v2[~seen] = bad, bad
        assert torch.equal(want, hc.paged_attention(q, k2, v2, table, n, window=window, sinks=sinks))


@pytest.mark.parametrize("dt", TYPES)
def test_infinities_and_nan_reach_what_sees_them(dt):
    q, k, v = make(dt, 1, 64, 64, 2, 2, 64)
    k[0, 10, 0, 3] = math.nan
    v[0, 20, 1, 5] = math.inf
    out = hc.attention(q, k, v)
    assert out[0, 10:, 0].isnan().all() and out[0, :10, 0].isfinite().all()
    assert (out[0, 20:, 1, 5] == math.inf).all() and out[0, :, 1, :5].isfinite().all() and out[0, :, 1, 6:].isfinite().all()
    kc, vc, table, n = cache(dt, [50], 2, 64, 16)
    kc[table[0, 0].long(), 3, 0, 1] = math.nan
    p = hc.paged_attention(q[0, :1], kc, vc, table, n)
    assert p[0, 0].isnan().all() and p[0, 1].isfinite().all()


def test_gradients_by_differences():
    """fp32: central differences of sum <out, d_out> in random directions. The step's error is of third order: with inputs of
    size 1 and a step of 2^-6, (2^-6)^2 / 6 times third derivatives of the order of the first; fp32 rounding of the two
    sums adds about 2^-24 sqrt(elements) / 2^-6. One percent of the 2-norms' product covers both."""
    for kw in (dict(), dict(causal=False), dict(window=9, sinks=2)):
        q, k, v = (x * 0.5 for x in make("f32", 1, 40, 50, 4, 2, 16))
        do = rand(tuple(q.shape), torch.float32, 9)
        out, lse = hc.attention(q, k, v, save=True, **kw)
        grads = hc.attention_backward(q, k, v, out, lse, do, **kw)
        for i, x in enumerate((q, k, v)):
            for seed in range(3):
                d = rand(tuple(x.shape), torch.float32, 20 + seed)
                h = 2.0 ** -6 / d.norm() * math.sqrt(16)

                def f(s):
                    y = [q, k, v]
                    y[i] = x + s * h * d
                    return (hc.attention(*y, **kw).double() * do.double()).sum()
                slope = (f(1) - f(-1)) / (2 * h.double())
                exact = (grads[i].double() * d.double()).sum()
                assert abs(slope - exact) <= 0.01 * grads[i].double().norm() * d.double().norm(), (kw, i, seed, slope, exact)


# ---------------------------------------------------------------- in a row

@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_a_layer_forward_and_backward(dt):
    """qkv product, attention, output product added to the residual, and all gradients, the attention's into columns of one
    tensor that the qkv product's backward pass takes; compared with fp64 autograd within a few roundings."""
    t, n, hidden, heads, kv, dim = T_OF[dt], 203, 192, 6, 2, 32
    width = (heads + 2 * kv) * dim
    x, w, wo, dy = rand((n, hidden), t, 1), rand((hidden, width), t, 2, hidden ** -0.5), rand((heads * dim, hidden), t, 3, hidden ** -0.5), rand((n, hidden), t, 4)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")

    def columns(m):
        return [m[:, a * dim:b * dim].view(n, b - a, dim) for a, b in ((0, heads), (heads, heads + kv), (heads + kv, heads + 2 * kv))]
    qkv = hc.linear(x, w, workspace=ws)
    out, lse = hc.attention(*columns(qkv), save=True, window=64, sinks=2, workspace=ws)
    y = hc.linear(out.view(n, -1), wo, residual=x, workspace=ws)
    do, dwo, _ = hc.linear_backward(out.view(n, -1), wo, dy, workspace=ws)
    d_qkv = torch.empty_like(qkv)
    hc.attention_backward(*columns(qkv), out, lse, do.view(n, heads, dim), window=64, sinks=2, grads=columns(d_qkv), workspace=ws)
    dx, dw, _ = hc.linear_backward(x, w, d_qkv, workspace=ws)

    X, W, WO = (a.double().requires_grad_() for a in (x, w, wo))
    q, k, v = columns(X @ W)
    see = ref.visible(n, n, True, 64, 2)
    s = torch.einsum("ihd,jhd->hij", q, k.repeat_interleave(heads // kv, 1)) * dim ** -0.5
    p = torch.softmax(s.masked_fill(~see, -math.inf), -1)
    Y = X + torch.einsum("hij,jhd->ihd", p, v.repeat_interleave(heads // kv, 1)).reshape(n, -1) @ WO
    gx, gw, gwo = torch.autograd.grad(Y, [X, W, WO], dy.double())
    # Each chain has at most seven roundings to T (qkv, weights, out, do, dS, d_qkv, the result), each of at most U
    # relative to its tensor and independent; the residual path's dy is not in dx here.
    tol = 8 * U(t) + 2.0 ** -18
    for name, got, want in (("y", y, Y.detach()), ("dwo", dwo, gwo), ("dw", dw, gw), ("dx", dx, gx - dy.double())):
        err = (got.double() - want).norm() / want.norm()
        assert err <= tol, (name, err.item(), tol)
