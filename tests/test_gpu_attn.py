"""The attention operators on the GPU against fp64 formulas, within bounds derived from their roundings
(``tests/_attn.py``)."""
from __future__ import annotations

import math
import random

import pytest
import torch

import _attn as ref
import hyper_connection_rank_amd as hc
from _ffn import T_OF, rand, within

pytestmark = pytest.mark.gpu

TYPES = ["bf16", "f16", "f32"]


def make(dt, batch, ql, kl, heads, kv, dim, seed=0):
    t = T_OF[dt]
    return (rand((batch, ql, heads, dim), t, seed + 1), rand((batch, kl, kv, dim), t, seed + 2),
            rand((batch, kl, kv, dim), t, seed + 3))


def check(q, k, v, label, ql=None, kl=None, back=True, **mask):
    """Forward with statistics and backward against the formulas; returns what the calls gave."""
    kw = dict(mask)
    if ql is not None:
        def sums(x):
            return torch.tensor([sum(x[:i]) for i in range(len(x) + 1)], dtype=torch.int32, device="cuda")
        kw["q_starts"] = sums(ql)
        if kl is not None:
            kw["k_starts"] = sums(kl)
    out, lse = hc.attention(q, k, v, save=True, **kw)
    eo, bo, el, bl = ref.attention(q, k, v, ql=ql, kl=kl, **mask)
    within(out, eo, bo, f"{label} out")
    none = el == -math.inf
    assert torch.equal(lse == -math.inf, none), label
    within(lse.masked_fill(none, 0.0), el.masked_fill(none, 0.0), bl.masked_fill(none, 0.0), f"{label} lse")
    assert torch.equal(hc.attention(q, k, v, **kw), out), label
    if back:
        do = rand(tuple(q.shape), q.dtype, 77)
        got = hc.attention_backward(q, k, v, out, lse, do, **kw)
        want = ref.attention_backward(q, k, v, out, lse, do, ql=ql, kl=kl, **mask)
        for n, g in zip(("dq", "dk", "dv"), got):
            within(g, *want[n], f"{label} {n}")
        again = hc.attention_backward(q, k, v, out, lse, do, **kw)
        assert all(torch.equal(x, y) for x, y in zip(got, again)), label
    return out, lse


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("ql,kl", [(1, 1), (1, 65), (31, 33), (64, 64), (65, 129), (128, 128), (200, 77), (130, 300)])
def test_lengths(dt, ql, kl):
    for causal in (True, False):
        check(*make(dt, 2, ql, kl, 4, 2, 64), f"{dt} {ql} {kl} {causal}", causal=causal)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("dim", [1, 7, 8, 24, 57, 63, 64, 65, 72, 80, 96, 97, 100, 120, 128, 129, 136, 160, 192, 200, 255, 256])
def test_head_sizes(dt, dim):
    check(*make(dt, 1, 97, 131, 3, 3, dim), f"{dt} {dim}")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 1), (5, 5), (8, 2), (10, 2), (16, 1), (40, 2), (7, 7)])
def test_heads(dt, heads, kv):
    check(*make(dt, 2, 70, 90, heads, kv, 32), f"{dt} {heads} {kv}")


MASKS = [(True, 1, 0), (True, 1, 1), (True, 16, 0), (True, 17, 4), (True, 64, 70), (True, 100, 17), (True, 500, 3), (False, 1, 0),
         (False, 20, 0), (False, 20, 5), (False, 70, 130), (True, 2 ** 31 - 1, 0), (True, 33, 2 ** 31 - 1)]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("causal,window,sinks", MASKS)
def test_windows_and_first_tokens(dt, causal, window, sinks):
    for ql, kl in ((300, 300), (37, 401), (301, 150)):
        check(*make(dt, 1, ql, kl, 4, 2, 64), f"{dt} {causal} {window} {sinks} {ql} {kl}", causal=causal, window=window, sinks=sinks)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("dim", [97, 127, 129, 193, 255, 256])
def test_wide_heads_over_many_tiles(dt, dim):
    """Sizes whose kernels hold more than the registers do, with groups, masks and packed rows over several tiles."""
    for mask in (dict(), dict(causal=False), dict(window=150, sinks=5)):
        check(*make(dt, 2, 333, 421, 6, 2, dim), f"{dt} {dim} {mask}", **mask)
    lens, t = [301, 0, 1, 130], T_OF[dt]
    n = sum(lens) + 2
    q, k, v = rand((n, 6, dim), t, 1), rand((n, 2, dim), t, 2), rand((n, 2, dim), t, 3)
    for mask in (dict(), dict(window=70, sinks=3)):
        check(q, k, v, f"{dt} {dim} packed {mask}", ql=lens, **mask)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("lens", [[5], [0], [0, 0, 3], [1, 1, 1, 1], [128, 1, 129, 0, 64], [300, 2, 31, 33, 0, 0, 257, 1], [1] * 70, [3, 0] * 100])
def test_packed_sequences(dt, lens):
    n = sum(lens) + 3
    t = T_OF[dt]
    q, k, v = rand((n, 6, 64), t, 1), rand((n, 2, 64), t, 2), rand((n, 2, 64), t, 3)
    for mask in (dict(causal=True), dict(causal=False), dict(causal=True, window=40, sinks=3)):
        check(q, k, v, f"{dt} {lens} {mask}", ql=lens, **mask)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("ql,kl,heads,kv,dim", [(1, 5000, 4, 1, 64), (7, 3100, 3, 3, 128), (40, 2100, 5, 1, 57), (1, 9000, 1, 1, 256), (200, 1030, 2, 1, 96)])
def test_few_queries_over_many_keys(dt, ql, kl, heads, kv, dim):
    """The keys split over workgroups, whose parts are joined; some of them see nothing."""
    for mask in (dict(), dict(causal=False), dict(window=600, sinks=5), dict(window=2000)):
        check(*make(dt, 2, ql, kl, heads, kv, dim), f"{dt} {ql} {kl} {dim} {mask}", **mask)
    t = T_OF[dt]
    lens_q, lens_k = [ql, 0, 1, 3], [kl, 700, 1, 0]
    q, k, v = rand((sum(lens_q) + 2, heads, dim), t, 1), rand((sum(lens_k), kv, dim), t, 2), rand((sum(lens_k), kv, dim), t, 3)
    check(q, k, v, f"{dt} {ql} {kl} {dim} packed", ql=lens_q, kl=lens_k)


@pytest.mark.parametrize("dt", TYPES)
def test_no_sequences(dt):
    t = T_OF[dt]
    x = [rand((9, h, 64), t, h) for h in (4, 2, 2)]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = hc.attention(*x, save=True, q_starts=st)
    assert not out.any() and not lse.any()
    assert not any(g.any() for g in hc.attention_backward(*x, out, lse, x[0], q_starts=st))
    empty = [y[:0] for y in x]
    out, lse = hc.attention(*empty, save=True)
    assert out.shape == (0, 4, 64)
    assert [g.shape for g in hc.attention_backward(*empty, out, lse, empty[0])] == [y.shape for y in empty]
    out, lse = hc.attention(x[0], x[1][:0], x[2][:0], save=True)
    assert not out.any() and (lse == -math.inf).all()
    assert not hc.attention_backward(x[0], x[1][:0], x[2][:0], out, lse, x[0])[0].any()
    out, lse = hc.attention(x[0][:0], *x[1:], save=True)
    dq, dk, dv = hc.attention_backward(x[0][:0], *x[1:], out, lse, x[0][:0])
    assert not dk.any() and not dv.any()


@pytest.mark.parametrize("dt", TYPES)
def test_packed_sequences_with_other_key_lengths(dt):
    ql, kl = [3, 0, 70, 1, 200], [40, 9, 70, 0, 90]
    t = T_OF[dt]
    q, k, v = rand((sum(ql) + 1, 4, 80), t, 1), rand((sum(kl) + 5, 4, 80), t, 2), rand((sum(kl) + 5, 4, 80), t, 3)
    for causal in (True, False):
        check(q, k, v, f"{dt} {causal}", ql=ql, kl=kl, causal=causal)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("dim", [64, 72, 31])
def test_layouts(dt, dim):
    """Columns of a merged projection (odd paddings make them unaligned), heads before tokens, tokens before sequences; the
    gradients into columns of one merged tensor; statistics of another layout."""
    b, n, heads, kv = 2, 150, 4, 2
    t = T_OF[dt]
    for pad in (0, 8, 1):
        width = (heads + 2 * kv) * dim + pad
        qkv = rand((b, n, width), t, 3)
        grad = rand((b, n, width), t, 4)

        def columns(x):
            c = [x[..., i * dim:j * dim].view(b, n, j - i, dim) for i, j in ((0, heads), (heads, heads + kv), (heads + kv, heads + 2 * kv))]
            return c
        q, k, v = columns(qkv)
        out, lse = check(q, k, v, f"{dt} {dim} merged {pad}", window=70, sinks=3)
        do = rand((b, n, heads, dim), t, 5)
        want = hc.attention_backward(q, k, v, out, lse, do)
        rest = grad[..., (heads + 2 * kv) * dim:].clone()
        odd = torch.empty(heads, n, b, device="cuda").permute(2, 1, 0)
        odd.copy_(lse)
        got = hc.attention_backward(q, k, v, out, odd, do, grads=columns(grad))
        assert all(torch.equal(x, y) for x, y in zip(want, got))
        assert torch.equal(torch.cat([x.flatten(2) for x in want], 2), grad[..., :(heads + 2 * kv) * dim])
        assert torch.equal(rest, grad[..., (heads + 2 * kv) * dim:])
    q, k, v = (rand((b, h, n, dim), t, 6 + h).transpose(1, 2) for h in (heads, kv, kv))
    check(q, k, v, f"{dt} {dim} heads first", causal=False)
    q, k, v = (rand((n, h, b, dim), t, 6 + h).permute(2, 0, 1, 3) for h in (heads, kv, kv))
    check(q, k, v, f"{dt} {dim} sequences last")


# ---------------------------------------------------------------- the cache in pages

def cache(dt, lens, kv, dim, page, seed=5, spare=3):
    """Caches, a table with entries of no page behind each sequence's last, and the lengths."""
    t = T_OF[dt]
    held = [-(-n // page) for n in lens]
    pages = sum(held) + spare
    order = list(range(pages))
    random.Random(seed).shuffle(order)
    table = torch.full((len(lens), max(held + [1])), -1, dtype=torch.int32)
    for b, n in enumerate(held):
        for i in range(n):
            table[b, i] = order.pop()
    kc, vc = rand((pages, page, kv, dim), t, seed + 1), rand((pages, page, kv, dim), t, seed + 2)
    return kc, vc, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")


def check_paged(dt, lens, heads, kv, dim, page, label="", **mask):
    kc, vc, table, n = cache(dt, lens, kv, dim, page)
    q = rand((len(lens), heads, dim), T_OF[dt], 9)
    out = hc.paged_attention(q, kc, vc, table, n, **mask)
    within(out, *ref.paged(q, kc, vc, table, n, **mask), f"paged {label} {dt} {lens[:6]} {heads} {kv} {dim} {page} {mask}")
    assert torch.equal(out, hc.paged_attention(q, kc, vc, table, n, **mask))
    return out


LENS = [[1], [0], [2, 0, 1], [15, 16, 17, 63, 64, 65], [1000, 1, 0, 333], [5000]]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("page", [1, 16, 17, 64, 256])
def test_paged_lengths(dt, lens, page):
    check_paged(dt, lens, 8, 2, 64, page)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("dim", [1, 7, 16, 57, 64, 80, 96, 100, 128, 129, 192, 255, 256])
def test_paged_head_sizes(dt, dim):
    check_paged(dt, [300, 70, 1], 6, 3, dim, 16)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("heads,kv", [(1, 1), (5, 1), (16, 1), (17, 1), (40, 2), (7, 7), (64, 2)])
def test_paged_heads(dt, heads, kv):
    check_paged(dt, [130, 700], heads, kv, 128, 16)


@pytest.mark.parametrize("dt", TYPES)
def test_paged_layouts(dt):
    """Both caches in one tensor, heads before rows, queries as columns of a merged projection; a table wider than needed;
    pages that the cache does not have."""
    lens, heads, kv, dim, page = [100, 33, 1], 8, 4, 64, 16
    kc, vc, table, n = cache(dt, lens, kv, dim, page)
    t = T_OF[dt]
    for shift in (0, 1):
        merged = rand((len(lens), heads * dim + 24 + shift), t, 9)
        q = merged[:, shift:shift + heads * dim].view(len(lens), heads, dim)
        want = ref.paged(q, kc, vc, table, n)
        within(hc.paged_attention(q, kc, vc, table, n), *want, f"merged {dt} {shift}")
        both = torch.empty(2, kc.shape[0], kv, page, dim, dtype=t, device="cuda").transpose(2, 3)
        both[0], both[1] = kc, vc
        wide = torch.full((len(lens), 40), 1 << 30, dtype=torch.int32, device="cuda")
        wide[:, 3:3 + table.shape[1]] = table
        out = torch.zeros(len(lens), heads, dim + 8, dtype=t, device="cuda")
        hc.paged_attention(q, both[0], both[1], wide[:, 3:30], n, out=out[:, :, :dim])
        within(out[:, :, :dim], *want, f"heads first {dt} {shift}")
        assert not out[:, :, dim:].any()
    for bad in (-1, -2 ** 31, kc.shape[0], 2 ** 31 - 1):
        wrong = table.clone()
        wrong[0, 2], wrong[1, 0], wrong[2, 0] = bad, bad, bad
        within(hc.paged_attention(q, kc, vc, wrong, n), *ref.paged(q, kc, vc, wrong, n), f"bad page {bad}")
    for length in (-5, 2 ** 31 - 1):
        m = torch.tensor([100, length, 7], dtype=torch.int32, device="cuda")
        within(hc.paged_attention(q, kc, vc, table, m), *ref.paged(q, kc, vc, table, m), f"length {length}")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (100, 4), (100, 130), (64, 64), (700, 3), (2 ** 31 - 1, 0), (5, 2 ** 31 - 1)])
def test_paged_windows(dt, window, sinks):
    check_paged(dt, [1, 64, 129, 700, 3000, 0], 4, 2, 64, 16, window=window, sinks=sinks)


def test_store_and_map_in_a_row():
    """Requests grow step by step: map, store, attend; the cache then holds what a contiguous one would."""
    rng = random.Random(4)
    page, most, heads, kv, dim = 16, 12, 8, 2, 64
    batch, t = 5, torch.bfloat16
    kc, vc = torch.full((40, page, kv, dim), math.nan, dtype=t, device="cuda"), torch.full((40, page, kv, dim), math.nan, dtype=t, device="cuda")
    free = torch.randperm(40, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    first = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = torch.full((batch, most), -7, dtype=torch.int32, device="cuda")
    cached = torch.zeros(batch, dtype=torch.int32, device="cuda")
    held = [[] for _ in range(batch)]
    for step in range(12):
        new = [rng.choice([0, 1, 1, 1, 17]) if step else rng.randint(0, 40) for _ in range(batch)]
        tokens = sum(new) + 3
        fresh = torch.tensor(new, dtype=torch.int32, device="cuda")
        want = ref.page_map(cached.tolist(), new, table.tolist(), free.tolist(), page, tokens, int(first))
        starts, lengths, positions, slots, taken = hc.page_map(cached, fresh, table, free, page_size=page, tokens=tokens, free_start=first)
        for x, y in zip((starts, lengths, positions, slots, taken, table), want):
            assert x.tolist() == y
        k, v = rand((tokens, kv, dim), t, 100 + step), rand((tokens, kv, dim), t, 200 + step)
        hc.cache_store(k, v, kc, vc, slots)
        for b in range(batch):
            held[b] += [(k[i], v[i]) for i in range(sum(new[:b]), sum(new[:b + 1]))]
        q = rand((batch, heads, dim), t, 300 + step)
        out = hc.paged_attention(q, kc, vc, table, lengths)
        within(out, *ref.paged(q, kc, vc, table, lengths), f"step {step}")
        for b in range(batch):
            if held[b]:
                kb, vb = torch.stack([x[0] for x in held[b]]), torch.stack([x[1] for x in held[b]])
                eo, bo, _, _ = ref.attention(q[b:b + 1], kb, vb)
                within(out[b:b + 1], eo, bo, f"step {step} sequence {b}")
        cached, first = lengths.clone(), first + taken[-1:]
    assert int(first) <= 40


@pytest.mark.parametrize("batch", [0, 1, 63, 1023, 1024, 1025, 3000])
@pytest.mark.parametrize("page", [1, 16, 17])
def test_maps(batch, page):
    rng = random.Random(batch * 31 + page)
    most = 40
    cached = [rng.choice([0, 1, page, page * 3, rng.randint(0, 39 * page), -5]) for _ in range(batch)]
    fresh = [rng.choice([0, 1, 1, 2, rng.randint(0, 3 * page), -2]) for _ in range(batch)]
    table = [[rng.randint(0, 99) for _ in range(most)] for _ in range(batch)]
    free = [rng.randint(0, 1 << 20) for _ in range(sum(max(x, 0) for x in fresh) // page + batch // 2)]
    tokens = max(0, sum(max(x, 0) for x in fresh) + rng.choice([-4, 0, 9]))

    def ints(x, shape):
        return torch.tensor(x, dtype=torch.int32).reshape(shape).cuda()
    tb = ints(table, (batch, most))
    got = hc.page_map(ints(cached, (batch,)), ints(fresh, (batch,)), tb, ints(free, (len(free),)), page_size=page, tokens=tokens)
    want = ref.page_map(cached, fresh, table, free, page, tokens)
    for x, y in zip(got + (tb,), want):
        assert x.tolist() == y


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("tokens,kv,dim,page", [(1, 1, 1, 1), (5, 3, 57, 7), (64, 8, 128, 16), (300, 2, 64, 256), (33, 1, 256, 17)])
def test_store(dt, tokens, kv, dim, page):
    t = T_OF[dt]
    pages = tokens // page + 3
    kc, vc = rand((pages, page, kv, dim), t, 1), rand((pages, page, kv, dim), t, 2)
    merged = rand((tokens, 2 * kv * dim), t, 3)
    k, v = merged[:, :kv * dim].view(tokens, kv, dim), merged[:, kv * dim:].view(tokens, kv, dim)
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(6))[:tokens].to(torch.int32)
    slots[::7] = -1
    if tokens > 4:
        slots[3], slots[4] = pages * page, 2 ** 31 - 1
    want = [kc.clone(), vc.clone()]
    for i, s in enumerate(slots.tolist()):
        if 0 <= s < pages * page:
            want[0][s // page, s % page], want[1][s // page, s % page] = k[i], v[i]
    hc.cache_store(k, v, kc, vc, slots.cuda())
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])
