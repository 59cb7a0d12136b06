"""The attention operators' boundary on the CPU: every refusal happens on the host before any launch (fake,
never-dereferenced device pointers), and the binding refuses tensors whose layout the entry points cannot take."""
from __future__ import annotations

import ctypes

import pytest
import torch

import hyper_connection_rank_amd as hc

E, U, W, OK = (hc.HCLRMIX_ERR_INVALID_ARGUMENT, hc.HCLRMIX_ERR_UNSUPPORTED, hc.HCLRMIX_ERR_WORKSPACE_TOO_SMALL,
               hc.HCLRMIX_OK)
BASE = 1 << 40
BF16 = hc.HCLRMIX_BF16

ORDER = {
    "hclrmix_attention": ("q", "k", "v", "q_starts", "k_starts", "out", "lse", "workspace"),
    "hclrmix_attention_backward": ("q", "k", "v", "out", "lse", "d_out", "q_starts", "k_starts", "dq", "dk", "dv", "workspace"),
    "hclrmix_paged_attention": ("q", "k_cache", "v_cache", "table", "lengths", "out", "workspace"),
    "hclrmix_cache_store": ("k", "v", "slots", "k_cache", "v_cache"),
    "hclrmix_page_map": ("cached", "fresh", "free_pages", "free_start", "table", "starts", "lengths", "positions", "slots", "taken"),
}
SIZES = {"hclrmix_attention": "hclrmix_attention_workspace_size",
         "hclrmix_attention_backward": "hclrmix_attention_backward_workspace_size",
         "hclrmix_paged_attention": "hclrmix_paged_attention_workspace_size"}


def problem(name):
    if name.startswith("hclrmix_attention"):
        return hc.AttentionProblem(2, 64, 64, 8, 2, 64, BF16, 1, 0, 0, 0, 0.125)
    if name == "hclrmix_paged_attention":
        return hc.PagedProblem(2, 100, 16, 30, 0, 8, 2, 64, BF16, 0, 0, 0.125)
    if name == "hclrmix_cache_store":
        return hc.StoreProblem(33, 100, 16, 2, 64, BF16)
    return hc.MapProblem(4, 50, 16, 30, 0, 200)


class Call:
    def __init__(self, name, **given):
        self.name, self.problem = name, problem(name)
        self.p = {n: BASE + ((i + 1) << 36) for i, n in enumerate(ORDER[name])}
        for n in ("q_starts", "k_starts"):
            if n in self.p:
                self.p[n] = None
        self.p.update(given)
        self.ws_bytes = 1 << 35

    def run(self):
        args = []
        for n in ORDER[self.name]:
            args.append(self.p[n])
            if n == "workspace":
                args.append(self.ws_bytes)
        return getattr(hc.library(), self.name)(*args, ctypes.byref(self.problem), None)


def expect(call, status, part=""):
    assert call.run() == status, hc.hclrmix_last_error()
    assert part in hc.hclrmix_last_error(), hc.hclrmix_last_error()


def test_null_problem():
    for name, order in ORDER.items():
        args = [None] * len(order) + ([0] if "workspace" in order else [])
        assert getattr(hc.library(), name)(*args, None, None) == E
    for name in SIZES.values():
        n = ctypes.c_size_t()
        assert getattr(hc.library(), name)(None, ctypes.byref(n)) == E


WHOLE = ("hclrmix_attention", "hclrmix_attention_backward")
COMMON = [("dtype", 11, U), ("heads", 0, E), ("kv_heads", 0, E), ("kv_heads", 3, E), ("heads", 2048, U), ("dim", 0, E), ("dim", 257, U),
          ("window", -1, E), ("sinks", -1, E), ("scale", 0.0, E), ("scale", -1.0, E), ("scale", float("nan"), E), ("scale", float("inf"), E),
          ("batch", -1, E), ("batch", 65537, U)]


@pytest.mark.parametrize("name", WHOLE)
@pytest.mark.parametrize("field,value,status", COMMON + [
    ("causal", 2, E), ("causal", -1, E), ("packed", 2, E), ("q_tokens", -1, E), ("k_tokens", -1, E), ("q_tokens", (1 << 21) + 1, U),
    ("k_tokens", (1 << 21) + 1, U), ("heads", 514, E), ("q_token", (1 << 21) + 1, U), ("k_sequence", (1 << 40) + 1, U), ("q_head", -1, E),
    ("v_token", -1, E), ("lse_token", 7, E), ("lse_head", -1, E), ("out_sequence", -1, E), ("q_token", 511, E), ("k_head", 63, E), ("out_head", 63, E)])
def test_attention_problems(name, field, value, status):
    c = Call(name)
    if field == "heads" and value == 514:
        c.problem.kv_heads = 4
    setattr(c.problem, field, value)
    expect(c, status)


def test_attention_limits():
    for name in WHOLE:
        c = Call(name)
        c.problem.batch, c.problem.q_tokens = 1 << 10, 1 << 17
        expect(c, U, "2^29")
        c = Call(name)
        c.problem.batch, c.problem.q_tokens, c.problem.heads = 65536, 1, 32
        expect(c, U, "2^20")
        n = ctypes.c_size_t()
        assert getattr(hc.library(), SIZES[name])(ctypes.byref(c.problem), ctypes.byref(n)) == U
        assert getattr(hc.library(), SIZES[name])(ctypes.byref(problem(name)), None) == E


@pytest.mark.parametrize("name", WHOLE)
def test_attention_reserved(name):
    c = Call(name)
    c.problem.reserved = 1
    expect(c, E, "reserved")
    for x in (-1, 2):
        c = Call(name)
        c.problem.zero_rest = x
        expect(c, E, "zero_rest")


@pytest.mark.parametrize("name,missing", [(n, m) for n in WHOLE for m in ("q", "k", "v", "out")] +
                         [(WHOLE[1], "lse"), (WHOLE[1], "d_out")] +
                         [("hclrmix_paged_attention", m) for m in ("q", "k_cache", "v_cache", "table", "lengths", "out")] +
                         [("hclrmix_cache_store", m) for m in ORDER["hclrmix_cache_store"]] +
                         [("hclrmix_page_map", m) for m in ORDER["hclrmix_page_map"] if m != "free_start"])
def test_required_pointers(name, missing):
    expect(Call(name, **{missing: None}), E)


def test_backward_wants_a_gradient():
    expect(Call(WHOLE[1], dq=None, dk=None, dv=None), E, "no gradient")


@pytest.mark.parametrize("name", WHOLE)
def test_starts_must_match(name):
    expect(Call(name, q_starts=BASE), E, "packed")
    expect(Call(name, k_starts=BASE), E, "packed")
    c = Call(name)
    c.problem.packed = 1
    expect(c, E, "packed")
    c = Call(name, q_starts=BASE)
    c.problem.packed, c.problem.k_tokens = 1, 65
    expect(c, E, "k_starts")
    c = Call(name, q_starts=BASE + 2)
    c.problem.packed = 1
    expect(c, U, "aligned")


@pytest.mark.parametrize("name", list(SIZES))
def test_workspaces(name):
    n = ctypes.c_size_t()
    assert getattr(hc.library(), SIZES[name])(ctypes.byref(problem(name)), ctypes.byref(n)) == OK
    assert n.value >= 4096
    c = Call(name)
    c.ws_bytes = n.value - 1
    expect(c, W, "workspace")
    expect(Call(name, workspace=None), W, "workspace")
    expect(Call(name, workspace=BASE + 8), U, "workspace")


@pytest.mark.parametrize("name,tensor", [(n, t) for n in ORDER for t in ORDER[n] if t not in ("workspace", "q_starts", "k_starts")])
def test_alignment(name, tensor):
    c = Call(name)
    c.p[tensor] += 1
    expect(c, U, "align")


@pytest.mark.parametrize("name,out", [("hclrmix_attention", "out"), ("hclrmix_attention", "lse"), ("hclrmix_attention", "workspace")] +
                         [(WHOLE[1], x) for x in ("dq", "dk", "dv", "workspace")] +
                         [("hclrmix_paged_attention", "out"), ("hclrmix_paged_attention", "workspace")] +
                         [("hclrmix_cache_store", x) for x in ("k_cache", "v_cache")] +
                         [("hclrmix_page_map", x) for x in ("table", "starts", "lengths", "positions", "slots", "taken")])
def test_outputs_lie_apart(name, out):
    for other in ORDER[name]:
        c = Call(name)
        if other == out or c.p[other] is None:
            continue
        c.p[out] = c.p[other]
        expect(c, E, "overlap")


def test_columns_of_one_matrix_are_apart():
    """q, k, v and their gradients as columns of merged rows: what does not share a byte is taken (a workspace that is
    too small is then the refusal), what does is refused."""
    h, hk, d = 8, 2, 64
    row = (h + 2 * hk) * d

    def call(shift=0, sequence=64 * row):
        c = Call(WHOLE[1])
        c.ws_bytes = 0
        for n, at in (("q", 0), ("k", h * d), ("v", (h + hk) * d)):
            c.p["d" + n] = (1 << 50) + 2 * at + (2 * shift if n == "k" else 0)
            for f in (n, "d" + n):
                setattr(c.problem, f + "_token", row)
                setattr(c.problem, f + "_sequence", sequence)
            c.p[n] = (1 << 51) + 2 * at
        return c
    expect(call(), W)
    expect(call(-8), E, "overlap")
    expect(call(8), E, "overlap")
    expect(call(sequence=64 * row + 8), E, "overlap")
    c = call()
    c.p["dv"] = c.p["v"]
    expect(c, E, "overlap")


@pytest.mark.parametrize("field,value,status", COMMON + [
    ("pages", -1, E), ("page_size", 0, E), ("page_size", 65537, U), ("most_pages", -1, E), ("most_pages", (1 << 25) + 1, U),
    ("table_stride", 29, E), ("table_stride", -1, E), ("reserved", 1, E), ("cache_token", -1, E), ("cache_token", (1 << 21) + 1, U),
    ("cache_sequence", 64, E), ("cache_sequence", (1 << 40) + 1, U), ("q_sequence", 64, E), ("out_sequence", 64, E)])
def test_paged_problems(field, value, status):
    c = Call("hclrmix_paged_attention")
    setattr(c.problem, field, value)
    expect(c, status)


@pytest.mark.parametrize("field,value,status", [
    ("tokens", -1, E), ("tokens", (1 << 21) + 1, U), ("pages", -1, E), ("pages", 1 << 31, U), ("page_size", 0, E), ("page_size", 65537, U),
    ("kv_heads", 0, E), ("kv_heads", 1025, U), ("dim", 257, U), ("dtype", 2, U), ("reserved", 1, E), ("k_token", 64, E), ("v_head", 32, E),
    ("cache_head", 1, E)])
def test_store_problems(field, value, status):
    c = Call("hclrmix_cache_store")
    setattr(c.problem, field, value)
    expect(c, status)


@pytest.mark.parametrize("field,value,status", [
    ("batch", -1, E), ("batch", 65537, U), ("tokens", -1, E), ("tokens", (1 << 21) + 1, U), ("page_size", 0, E), ("page_size", 65537, U),
    ("most_pages", -1, E), ("most_pages", 1 << 31, U), ("table_stride", 29, E), ("free_count", -1, E), ("free_count", 1 << 31, U),
    ("reserved", 1, E)])
def test_map_problems(field, value, status):
    c = Call("hclrmix_page_map")
    setattr(c.problem, field, value)
    expect(c, status)


def test_nothing_to_do():
    for name, field in (("hclrmix_attention", "batch"), ("hclrmix_attention", "q_tokens"), (WHOLE[1], "batch"),
                        ("hclrmix_paged_attention", "batch"), ("hclrmix_cache_store", "tokens"), ("hclrmix_cache_store", "pages")):
        c = Call(name)
        setattr(c.problem, field, 0)
        expect(c, OK)


# ---------------------------------------------------------------- the binding

def t(*s, dtype=torch.bfloat16):
    return torch.zeros(*s, dtype=dtype)


def ints(*s):
    return torch.zeros(*s, dtype=torch.int32)


def calls():
    """Each function's tensors that take part in gradients, and a call with them."""
    q, k, lse = lambda: t(2, 5, 4, 8), lambda: t(2, 5, 2, 8), t(2, 5, 4, dtype=torch.float32)  # noqa: E731
    kc = lambda: t(3, 16, 2, 8)  # noqa: E731
    return {"attention": ([q(), k(), k()], hc.attention),
            "attention_backward": ([q(), k(), k(), q(), q()], lambda a, b, c, o, g: hc.attention_backward(a, b, c, o, lse, g)),
            "paged_attention": ([t(2, 4, 8), kc(), kc()], lambda a, b, c: hc.paged_attention(a, b, c, ints(2, 3), ints(2))),
            "cache_store": ([t(5, 2, 8), t(5, 2, 8), kc(), kc()], lambda a, b, c, d: hc.cache_store(a, b, c, d, ints(5)))}


@pytest.mark.parametrize("name", list(calls()))
def test_autograd_records_none(name):
    tensors, call = calls()[name]
    for i, x in enumerate(tensors):
        given = list(tensors)
        given[i] = x.clone().requires_grad_()
        with pytest.raises(hc.HclrmixError, match="autograd"):
            call(*given)
        with torch.no_grad(), pytest.raises(hc.HclrmixError, match="GPU"):
            call(*given)


def refused(f, *args, part="", **kw):
    with pytest.raises(hc.HclrmixError) as e:
        f(*args, **kw)
    assert part in str(e.value), str(e.value)


def test_attention_tensors():
    q, k = t(2, 5, 4, 8), t(2, 7, 2, 8)
    a = hc.attention
    refused(a, q.double(), k, k, part="dtype")
    refused(a, q[0, 0], k, k, part="q must be")
    refused(a, q, k[0], k, part="dimensions")
    refused(a, q, k, k[:, :6], part="v must be")
    refused(a, q, t(2, 7, 2, 9), k, part="k must be")
    refused(a, q, k.float(), k, part="dtype")
    refused(a, q, t(2, 7, 8, 2).transpose(2, 3), k, part="contiguous")
    refused(a, q, t(2, 7, 1, 8).expand(2, 7, 2, 8), k, part="expand")
    refused(a, t(2, 1, 4, 8).expand(2, 5, 4, 8), k, k, part="expand")
    refused(a, q, k, k, window=-1, part="window")
    refused(a, q, k, k, sinks=1 << 31, part="sinks")
    refused(a, q, k, k, scale=0.0, part="scale")
    refused(a, q, t(2, 7, 3, 8), t(2, 7, 3, 8), part="multiple")
    refused(a, q, k, k, q_starts=ints(3), part="packed")
    refused(a, q[0], k[0], k[0], k_starts=ints(3), part="q_starts")
    refused(a, q[0], k[0], k[0], q_starts=ints(3), part="k_starts")
    refused(a, q[0], k[0], k[0], q_starts=ints(3), k_starts=ints(2), part="k_starts")
    refused(a, q[0], k[0], k[0], q_starts=ints(3).long(), part="int32")
    refused(a, q, k, k, out=t(2, 5, 4, 9), part="out must be")
    refused(a, q, k, k, workspace=torch.zeros(2, 8192, dtype=torch.uint8)[:, ::2], part="workspace")


def test_backward_tensors():
    q, k, lse = t(2, 5, 4, 8), t(2, 7, 2, 8), t(2, 5, 4, dtype=torch.float32)
    b = hc.attention_backward
    refused(b, q, k, k, q, lse.bfloat16(), q, part="lse")
    refused(b, q, k, k, q, lse[..., :1].expand(2, 5, 4), q, part="lse")
    refused(b, q, k, k, q, lse[:, :4], q, part="lse")
    refused(b, q, k, k, q[:, :4], lse, q, part="out")
    refused(b, q, k, k, q, lse, t(2, 5, 1, 8).expand(2, 5, 4, 8), part="d_out")
    refused(b, q, k, k, q, lse, q, grads=(None, None, None), part="GPU")
    refused(b, q, k, k, q, lse, q, grads=(None, q, None), part="dk")


def test_paged_tensors():
    q, kc, table, n = t(2, 4, 8), t(3, 16, 2, 8), ints(2, 5), ints(2)
    p = hc.paged_attention
    refused(p, q[0], kc, kc, table, n, part="q must be")
    refused(p, q, kc[0], kc, table, n, part="k_cache")
    refused(p, q, kc, t(4, 16, 2, 8), table, n, part="v_cache")
    refused(p, q, kc, t(3, 2, 16, 8).transpose(1, 2), table, n, part="strides")
    refused(p, q, t(3, 16, 2, 9), t(3, 16, 2, 9), table, n, part="k_cache")
    refused(p, q, kc, kc, table.long(), n, part="int32")
    refused(p, q, kc, kc, ints(3, 5), n, part="block_table")
    refused(p, q, kc, kc, ints(1, 5).expand(2, 5), n, part="block_table")
    refused(p, q, kc, kc, table, ints(3), part="lengths")
    refused(p, q, kc, kc, table, n.long(), part="lengths")


def test_store_and_map_tensors():
    k, kc = t(5, 2, 8), t(3, 16, 2, 8)
    refused(hc.cache_store, k[0], k, kc, kc, ints(5), part="k must be")
    refused(hc.cache_store, k, k[:4], kc, kc.clone(), ints(5), part="v must be")
    refused(hc.cache_store, k, k, kc, kc.clone(), ints(4), part="slots")
    refused(hc.cache_store, k, k, kc, kc.clone(), ints(5).long(), part="slots")
    m = hc.page_map
    kw = dict(page_size=16, tokens=9)
    refused(m, ints(3).long(), ints(3), ints(3, 4), ints(9), **kw, part="cached")
    refused(m, ints(3), ints(2), ints(3, 4), ints(9), **kw, part="fresh")
    refused(m, ints(3), ints(3), ints(2, 4), ints(9), **kw, part="block_table")
    refused(m, ints(3), ints(3), ints(3, 4), ints(9, 2), **kw, part="free_pages")
    refused(m, ints(3), ints(3), ints(3, 4), ints(9), free_start=ints(2), **kw, part="free_start")
    refused(m, ints(3), ints(3), ints(3, 4), ints(9), page_size=16, tokens=-1, part="tokens")
    refused(m, ints(3), ints(3), ints(3, 4), ints(9), out=(ints(4), ints(3), ints(9), ints(8), ints(4)), **kw, part="slots")


@pytest.mark.parametrize("dtype", [torch.float64, torch.int8, None])
def test_workspace_sizes_of_other_types(dtype):
    refused(hc.attention_workspace_size, 1, 8, 8, 4, 2, 64, dtype, part="dtype")
    refused(hc.paged_attention_workspace_size, 1, 8, 16, 4, 2, 64, dtype, part="dtype")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("heads,kv,dim", [(1, 1, 8), (8, 2, 64), (20, 4, 128), (64, 1, 128), (34, 2, 200), (16, 16, 256)])
def test_a_workspace_for_the_most_serves_fewer(dtype, heads, kv, dim):
    steps = sorted({1, 2, 3, 5, 7, 8, 15, 16, 17, 31, 33, 64, 100, 129, 255, 400, 513, 1000, 1024, 3000})
    for backward in (False, True):
        for packed in (False, True):
            for a in ([hc.attention_workspace_size(b, 300, 300, heads, kv, dim, dtype, packed=packed, backward=backward) for b in steps],
                      [hc.attention_workspace_size(2, n, 300, heads, kv, dim, dtype, packed=packed, backward=backward) for n in steps],
                      [hc.attention_workspace_size(2, 300, n, heads, kv, dim, dtype, packed=packed, backward=backward) for n in steps]):
                assert a == sorted(a), (backward, packed)
    for page in (1, 16, 256):
        for b in (1, 3, 40, 700):
            a = [hc.paged_attention_workspace_size(b, n, page, heads, kv, dim, dtype) for n in steps]
            assert a == sorted(a)
        for n in (1, 30, 800):
            a = [hc.paged_attention_workspace_size(b, n, page, heads, kv, dim, dtype) for b in steps]
            assert a == sorted(a)
