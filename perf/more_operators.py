"""The attention operators as measured cases: attention over packed or batched
sequences with a window and first tokens that stay visible (attention), its
gradients (attention_backward), one new token of each sequence over a paged
cache (paged_attention), the write into that cache (cache_store) and the
tables that say where tokens live (page_map).

Where ``own`` is false ``run`` computes the plain form: elementary torch
operations in fp32, rounded once at the end. Where it is true, ``run`` calls
hyper_connection_rank_amd.

Sizes: 20 heads of 128 are hidden 2560, 32 heads of 128 hidden 4096, as in the
decode, prefill and wide blocks; the rest is generic.
"""
import itertools
import math
import random

import torch

own = False

_T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # A prompt of 8192 tokens at the wide block's width.
        {"name": "att_prompt", "op": "att", "batch": 1, "q_len": 8192, "k_len": 8192, "ragged": False, "heads": 32, "kv_heads": 8,
         "dim": 128, "dtype": "bf16", "causal": True, "window": 0, "sinks": 0, "save": False},
        # Training on packed documents of odd lengths, window and first tokens, statistics kept for the backward pass.
        {"name": "att_packed", "op": "att", "batch": 7, "q_len": 3001, "k_len": 3001, "ragged": True, "heads": 20, "kv_heads": 4,
         "dim": 64, "dtype": "f16", "causal": True, "window": 512, "sinks": 4, "save": True},
        # A short encoder batch in fp32: every key visible, odd lengths and an odd head size.
        {"name": "att_odd", "op": "att", "batch": 3, "q_len": 197, "k_len": 211, "ragged": False, "heads": 6, "kv_heads": 6,
         "dim": 57, "dtype": "f32", "causal": False, "window": 0, "sinks": 0, "save": True},
        # The backward pass of two sequences of 4096 tokens at the decode block's width.
        {"name": "back_train", "op": "att_back", "batch": 2, "q_len": 4096, "k_len": 4096, "ragged": False, "heads": 20, "kv_heads": 4,
         "dim": 128, "dtype": "bf16", "causal": True, "window": 0, "sinks": 0, "save": True},
        # The backward pass of packed documents with a window and first tokens.
        {"name": "back_packed", "op": "att_back", "batch": 9, "q_len": 1501, "k_len": 1501, "ragged": True, "heads": 12, "kv_heads": 12,
         "dim": 80, "dtype": "f16", "causal": True, "window": 300, "sinks": 2, "save": True},
        # One long conversation: a single sequence fills the card only if its length is split.
        {"name": "paged_one", "op": "paged", "batch": 1, "length": 32768, "ragged": False, "heads": 32, "kv_heads": 8, "dim": 128,
         "dtype": "bf16", "page": 16, "window": 0, "sinks": 0},
        # A serving batch of 64 sequences, their lengths spread over 1 to 16384.
        {"name": "paged_batch", "op": "paged", "batch": 64, "length": 16384, "ragged": True, "heads": 20, "kv_heads": 4, "dim": 128,
         "dtype": "bf16", "page": 64, "window": 0, "sinks": 0},
        # Long sequences of which a window and the first tokens are read.
        {"name": "paged_window", "op": "paged", "batch": 33, "length": 20011, "ragged": True, "heads": 16, "kv_heads": 16, "dim": 96,
         "dtype": "f16", "page": 32, "window": 2048, "sinks": 4},
        # A decode step's tokens into the cache. Latency only.
        {"name": "store_step", "op": "store", "tokens": 64, "kv_heads": 4, "dim": 128, "dtype": "bf16", "page": 64, "padding": 0},
        # A prompt's tokens into the cache, from a batch padded at its end.
        {"name": "store_prompt", "op": "store", "tokens": 16384, "kv_heads": 8, "dim": 128, "dtype": "bf16", "page": 16, "padding": 300},
        # The tables of a decode step: one new token for each of 64 sequences. Latency only.
        {"name": "map_step", "op": "map", "batch": 64, "new": 1, "cached": 16384, "page": 64, "padding": 0},
        # The tables of a mixed batch of 1000 requests, from single tokens to new prompts.
        {"name": "map_mixed", "op": "map", "batch": 1000, "new": 160, "cached": 4096, "page": 16, "padding": 777},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """Lengths over their logarithms, 1 to 8192 tokens (a cache: to 65536); head sizes up to 256, a quarter of them odd."""
    op = rng.choice(["att", "att", "att_back", "att_back", "paged", "paged", "store", "map"])
    dtype = rng.choice(["bf16", "f16", "bf16", "f16", "f32"])
    kv = rng.choice([1, 2, 3, 4, 8, 16])
    dim = _log_int(rng, 16, 256)
    dim = dim | 1 if rng.random() < 0.25 else max(16, dim & ~7)
    if rng.random() < 0.4:
        dim = rng.choice([64, 128])
    window = _log_int(rng, 1, 4096) if rng.random() < 0.4 else 0
    sinks = rng.choice([0, 1, 4, 17]) if window else 0
    if op == "store":
        tokens = _log_int(rng, 1, 16384)
        return {"op": op, "tokens": tokens, "kv_heads": kv, "dim": dim, "dtype": dtype, "page": rng.choice([1, 16, 17, 64, 256]),
                "padding": rng.choice([0, 0, tokens // 7])}
    if op == "map":
        batch, new = _log_int(rng, 1, 4096), _log_int(rng, 1, 4096)
        page = rng.choice([1, 16, 17, 64, 256])
        cached = min(_log_int(rng, 1, 32768), max(1, 2000000 * page // batch))  # at most about 2 million entries in the table
        return {"op": op, "batch": batch, "new": min(new, max(1, 400000 // batch)), "cached": cached, "page": page,
                "padding": rng.choice([0, 5, 1000])}
    group = rng.choice([1, 1, 2, 4, 5, 8, 16])
    while kv * group > 64:
        group //= 2
    if op == "paged":
        batch, length = _log_int(rng, 1, 128), _log_int(rng, 1, 65536)
        # At most about 1 GB of cache for the longest sequences.
        length = max(1, min(length, int(1e9 / (2 * _SIZE[dtype] * batch * kv * dim))))
        return {"op": op, "batch": batch, "length": length, "ragged": rng.random() < 0.7, "heads": kv * group, "kv_heads": kv, "dim": dim,
                "dtype": dtype, "page": rng.choice([1, 16, 16, 17, 64, 64, 256]), "window": window, "sinks": sinks}
    batch, q_len = _log_int(rng, 1, 16), _log_int(rng, 1, 8192)
    # No more than the largest listed case's pairs of positions (backward: half; fp32: an eighth).
    most = 2 ** 31 // (2 if op == "att_back" else 1) // (8 if dtype == "f32" else 1) // (batch * kv * group)
    q_len = max(1, min(q_len, int(math.sqrt(most))))
    ragged = rng.random() < 0.5
    k_len = q_len
    if not ragged and rng.random() < 0.4:  # a chunk of a longer sequence, or a short query over a long context
        k_len = max(1, min(_log_int(rng, 1, 16384), most // q_len))
    return {"op": op, "batch": batch, "q_len": q_len, "k_len": k_len, "ragged": ragged, "heads": kv * group, "kv_heads": kv, "dim": dim,
            "dtype": dtype, "causal": rng.random() < 0.8, "window": window, "sinks": sinks, "save": op == "att_back" or rng.random() < 0.5}


def _lengths(n, longest, ragged, least=1):
    """The sequences' lengths of a case: all the longest, or spread over least to longest with the longest among them."""
    if not ragged:
        return [longest] * n
    rng = random.Random(1000003 * n + longest)
    out = [rng.randint(min(least, longest), longest) for _ in range(n)]
    out[rng.randrange(n)] = longest
    return out


def _new_lengths(case):
    """Mixed request sizes: two thirds single tokens where a batch holds prompts."""
    rng = random.Random(7919 * case["batch"] + case["new"])
    return [1 if rng.random() < 2 / 3 else rng.randint(0, 3 * case["new"]) for _ in range(case["batch"])] if case["new"] > 1 else [1] * case["batch"]


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _sums(values):
    return list(itertools.accumulate(values, initial=0))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(_T[case["dtype"]])

    def perm(n):
        return torch.randperm(n, generator=gen, device="cuda").to(torch.int32)

    if case["op"] in ("att", "att_back"):
        hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
        if case["ragged"]:  # packed rows of one merged projection, two rows of padding at the end
            lens = _lengths(case["batch"], case["q_len"], True)
            rows = sum(lens) + 2
            qkv = normal(rows, (hq + 2 * hk) * d)
            s["q"] = qkv[:, :hq * d].view(rows, hq, d)
            s["k"] = qkv[:, hq * d:(hq + hk) * d].view(rows, hk, d)
            s["v"] = qkv[:, (hq + hk) * d:].view(rows, hk, d)
            s["starts"] = _int(_sums(lens))
        else:
            b, ql, kl = case["batch"], case["q_len"], case["k_len"]
            s["q"], s["k"], s["v"] = normal(b, ql, hq, d), normal(b, kl, hk, d), normal(b, kl, hk, d)
            s["starts"] = None
        if case["op"] == "att_back":
            s["d_out"] = normal(*s["q"].shape)
            s["out"], s["lse"] = _plain_att({**s, "case": {**case, "save": True}}).values()
        return s
    if case["op"] == "paged":
        b, hk, d, ps = case["batch"], case["kv_heads"], case["dim"], case["page"]
        lens = _lengths(b, case["length"], case["ragged"])
        most = (max(lens) + ps - 1) // ps
        pages = sum((n + ps - 1) // ps for n in lens) + 3
        s["k_cache"], s["v_cache"] = normal(pages, ps, hk, d), normal(pages, ps, hk, d)
        s["q"] = normal(b, case["heads"], d)
        s["lengths"] = _int(lens)
        # Every sequence's pages anywhere in the cache; the table's entries behind its last page name none.
        order, held = perm(pages), (s["lengths"] + ps - 1) // ps
        first = torch.cumsum(held, 0) - held
        at = torch.arange(most, device="cuda")[None]
        s["table"] = torch.where(at < held[:, None], order[(first[:, None] + at).clamp(max=pages - 1)], -1).to(torch.int32)
        return s
    if case["op"] == "store":
        n, hk, d, ps = case["tokens"], case["kv_heads"], case["dim"], case["page"]
        kv = normal(n, 2 * hk * d)
        s["k"], s["v"] = kv[:, :hk * d].view(n, hk, d), kv[:, hk * d:].view(n, hk, d)
        pages = (n + ps - 1) // ps + 5
        s["k_cache"], s["v_cache"] = normal(pages, ps, hk, d), normal(pages, ps, hk, d)
        s["slots"] = perm(pages * ps)[:n].contiguous()
        if case["padding"]:
            s["slots"][n - case["padding"]:] = -1
        return s
    b, ps = case["batch"], case["page"]
    new = _new_lengths(case)
    cached = torch.randint(0, case["cached"] + 1, (b,), generator=gen, device="cuda").to(torch.int32)
    s["cached"], s["new"] = cached, _int(new)
    held = (cached + ps - 1) // ps
    most = (case["cached"] + max(new) + ps - 1) // ps
    free = sum((n + ps - 1) // ps + 1 for n in new)
    pages = b * most + free
    order = perm(pages)
    at = torch.arange(most, device="cuda")[None]
    s["table"] = torch.where(at < held[:, None], order[:b * most].view(b, most), -1).to(torch.int32)
    s["free"] = order[b * most:].contiguous()
    s["rows"] = sum(new) + case["padding"]
    return s


# ---------------------------------------------------------------- plain form

def _padded(s):
    """Packed rows as a batch [sequences, longest]: each element's row, and each row's element (behind the last sequence: none)."""
    c, starts = s["case"], s["starts"].long()
    at = torch.arange(c["q_len"], device="cuda")[None]
    rows = (starts[:-1, None] + at).clamp(max=s["q"].shape[0] - 1)
    flat = torch.arange(s["q"].shape[0], device="cuda")
    seq = (torch.searchsorted(starts, flat, right=True) - 1).clamp(max=c["batch"] - 1)
    lens = starts[1:] - starts[:-1]
    real = flat < starts[-1]
    return rows, torch.where(real, seq * c["q_len"] + flat - starts[seq], 0), real, lens


def _heads_first(x, kv_heads):
    """[batch, length, heads, dim] as fp32 [batch * kv_heads, group * length, dim]."""
    b, n, h, d = x.shape
    return x.float().view(b, n, kv_heads, h // kv_heads, d).permute(0, 2, 3, 1, 4).reshape(b * kv_heads, h // kv_heads * n, d)


def _heads_last(x, batch, length):
    kv = x.shape[0] // batch
    g = x.shape[1] // length
    return x.view(batch, kv, g, length, x.shape[2]).permute(0, 3, 1, 2, 4).reshape(batch, length, kv * g, x.shape[2])


def _plain_inputs(s, names):
    c = s["case"]
    if s["starts"] is None:
        return [s[n] for n in names], None
    pad = _padded(s)
    return [s[n][pad[0]] for n in names], pad


def _plain_rows(x, s, pad, dtype):
    """Back to packed rows; zeros behind the last sequence."""
    if pad is not None:
        x = torch.where(pad[2].view(-1, *[1] * (x.dim() - 2)), x.flatten(0, 1)[pad[1]], torch.zeros((), device="cuda"))
    return x.to(dtype)


def _plain_visible(c, pad):
    """[batch or 1, 1, 1, q_len, k_len]: which keys a query sees."""
    ql, kl = c["q_len"], c["k_len"]
    i, j = torch.arange(ql, device="cuda")[:, None], torch.arange(kl, device="cuda")[None]
    p = i + (kl - ql)
    see = torch.ones(ql, kl, dtype=torch.bool, device="cuda")
    if c["causal"]:
        see = see & (j <= p)
    if c["window"]:
        see = see & (((p - j).abs() < c["window"]) | (j < c["sinks"]))
    see = see[None]
    if pad is not None:
        n = pad[3][:, None, None]
        see = see & (i < n) & (j < n)
    return see[:, None, None]


def _plain_scores(q, k, c, pad):
    """Scores [batch * kv_heads, group * q_len, k_len], -inf where a key is not seen."""
    s = torch.bmm(q, k.transpose(1, 2)) * c["dim"] ** -0.5
    v = s.view(c["batch"], c["kv_heads"], -1, c["q_len"], c["k_len"])
    v.masked_fill_(~_plain_visible(c, pad), -math.inf)
    return s


def _plain_att(s):
    c = s["case"]
    hk = c["kv_heads"]
    (q, k, v), pad = _plain_inputs(s, ("q", "k", "v"))
    p = _plain_scores(_heads_first(q, hk), _heads_first(k, hk), c, pad)
    m = p.amax(2, keepdim=True)
    safe = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = p.sub_(safe).exp_()
    n = p.sum(2, keepdim=True)
    out = torch.bmm(p, _heads_first(v, hk)) / torch.where(n == 0, torch.ones_like(n), n)
    got = {"out": _plain_rows(_heads_last(out, c["batch"], c["q_len"]), s, pad, s["q"].dtype)}
    if c["save"]:
        lse = _heads_last(torch.where(n == 0, torch.full_like(n, -math.inf), safe + torch.log(n)), c["batch"], c["q_len"])
        got["lse"] = _plain_rows(lse, s, pad, torch.float32)[..., 0]
    return got


def _plain_att_back(s):
    c = s["case"]
    hk, dt = c["kv_heads"], s["q"].dtype
    (q, k, v, out, do, lse), pad = _plain_inputs({**s, "lse4": s["lse"][..., None]}, ("q", "k", "v", "out", "d_out", "lse4"))
    q, k, v, out, do, lse = (_heads_first(x, hk) for x in (q, k, v, out, do, lse))
    scale = c["dim"] ** -0.5
    lse = torch.where(lse == -math.inf, torch.zeros_like(lse), lse)
    p = _plain_scores(q, k, c, pad).sub_(lse).exp_()
    dv = torch.bmm(p.transpose(1, 2), do)
    ds = torch.bmm(do, v.transpose(1, 2)).sub_((out * do).sum(2, keepdim=True)).mul_(p)
    dq = torch.bmm(ds, k) * scale
    dk = torch.bmm(ds.transpose(1, 2), q) * scale
    got = {"dq": _heads_last(dq, c["batch"], c["q_len"]), "dk": _heads_last(dk, c["batch"], c["k_len"]),
           "dv": _heads_last(dv, c["batch"], c["k_len"])}
    return {n: _plain_rows(x, s, pad, dt) for n, x in got.items()}


def _plain_paged(s):
    c = s["case"]
    b, hq, hk, d, ps = c["batch"], c["heads"], c["kv_heads"], c["dim"], c["page"]
    n = s["table"].shape[1] * ps
    at = torch.arange(n, device="cuda")
    rows = (s["table"].long().clamp(min=0)[:, :, None] * ps + torch.arange(ps, device="cuda")).view(b, n)
    k = s["k_cache"].view(-1, hk, d)[rows].float().transpose(1, 2)  # [batch, kv_heads, keys, dim]
    v = s["v_cache"].view(-1, hk, d)[rows].float().transpose(1, 2)
    p = s["lengths"].long()[:, None] - 1
    see = at[None] <= p
    if c["window"]:
        see = see & ((p - at < c["window"]) | (at < c["sinks"]))
    q = s["q"].float().view(b, hk, hq // hk, d)
    x = torch.matmul(q, k.transpose(2, 3)) * d ** -0.5
    x = x.masked_fill(~see[:, None, None], -math.inf)
    m = x.amax(3, keepdim=True)
    x = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    t = x.sum(3, keepdim=True)
    out = torch.matmul(x, v) / torch.where(t == 0, torch.ones_like(t), t)
    return {"out": out.view(b, hq, d).to(s["q"].dtype)}


def _plain_store(s):
    """Rows whose slot is negative go nowhere: they are sent behind the cache's end, in a copy one row longer."""
    out = {}
    for name in ("k", "v"):
        cache = s[name + "_cache"]
        n = cache.shape[0] * cache.shape[1]
        longer = torch.cat([cache.view(n, -1), cache.new_zeros(1, cache[0, 0].numel())])
        slots = s["slots"].long()
        longer[torch.where(slots < 0, torch.full_like(slots, n), slots)] = s[name].reshape(slots.numel(), -1)
        out[name + "_cache"] = longer[:n].view(cache.shape)
    return out


def _plain_map(s):
    c = s["case"]
    ps, b, n = c["page"], c["batch"], s["rows"]
    cached, new, table = s["cached"].long(), s["new"].long(), s["table"].long()
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    starts = torch.cat([zero, torch.cumsum(new, 0)])
    held = (cached + ps - 1) // ps
    need = (cached + new + ps - 1) // ps
    taken = torch.cat([zero, torch.cumsum(need - held, 0)])
    at = torch.arange(table.shape[1], device="cuda")[None]
    fresh = s["free"].long()[(taken[:-1, None] + at - held[:, None]).clamp(0, s["free"].numel() - 1)]
    table = torch.where((at >= held[:, None]) & (at < need[:, None]), fresh, table)
    t = torch.arange(n, device="cuda")
    seq = (torch.searchsorted(starts, t, right=True) - 1).clamp(max=b - 1)
    real = t < starts[-1]
    pos = torch.where(real, cached[seq] + t - starts[seq], zero)
    slots = torch.where(real, table[seq, pos // ps] * ps + pos % ps, zero - 1)
    got = {"table": table, "starts": starts, "lengths": cached + new, "positions": pos, "slots": slots, "taken": taken}
    return {k: v.to(torch.int32) for k, v in got.items()}


_PLAIN = {"att": _plain_att, "att_back": _plain_att_back, "paged": _plain_paged, "store": _plain_store, "map": _plain_map}


# ---------------------------------------------------------------- the library's calls

_kept = {}  # workspaces by device and stream, the largest last; none is freed, since a captured graph may use it


def _workspace(nbytes):
    """The zero-filled workspace that a program keeps for the calls on its stream, grown to the largest (outside a
    capture, as its first calls are)."""
    device = torch.cuda.current_device()
    kept = _kept.setdefault((device, torch._C._cuda_getCurrentRawStream(device)), [])
    if not kept or kept[-1].numel() < nbytes:
        kept.append(torch.zeros(nbytes, dtype=torch.uint8, device="cuda"))
    return kept[-1]


def _own(s):
    import hyper_connection_rank_amd as hc
    c = s["case"]
    op = c["op"]
    if op in ("att", "att_back"):
        back = op == "att_back"
        q_tokens, k_tokens = (s["q"].shape[0], s["k"].shape[0]) if c["ragged"] else (c["q_len"], c["k_len"])
        ws = _workspace(hc.attention_workspace_size(c["batch"], q_tokens, k_tokens, c["heads"], c["kv_heads"], c["dim"], s["q"].dtype,
                                                    packed=c["ragged"], backward=back))
        kw = dict(causal=c["causal"], window=c["window"], sinks=c["sinks"], q_starts=s["starts"], workspace=ws)
        if back:
            return dict(zip(("dq", "dk", "dv"), hc.attention_backward(s["q"], s["k"], s["v"], s["out"], s["lse"], s["d_out"], **kw)))
        got = hc.attention(s["q"], s["k"], s["v"], save=c["save"], **kw)
        return dict(zip(("out", "lse"), got)) if c["save"] else {"out": got}
    if op == "paged":
        ws = _workspace(hc.paged_attention_workspace_size(c["batch"], s["table"].shape[1], c["page"], c["heads"], c["kv_heads"], c["dim"],
                                                          s["q"].dtype))
        return {"out": hc.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], window=c["window"],
                                          sinks=c["sinks"], workspace=ws)}
    if op == "store":
        hc.cache_store(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"])
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    starts, lengths, positions, slots, taken = hc.page_map(s["cached"], s["new"], s["table"], s["free"], page_size=c["page"],
                                                           tokens=s["rows"])
    return {"table": s["table"], "starts": starts, "lengths": lengths, "positions": positions, "slots": slots, "taken": taken}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- work and the exact results

def _pairs(ql, kl, causal, window, sinks):
    """How many (query, key) pairs of one sequence are seen."""
    def seen(p):
        hi = max(0, min(kl, p + 1) if causal else (min(kl, p + window) if window else kl))
        lo = min(hi, max(0, p - window + 1)) if window else 0
        first = min(sinks, max(0, min(kl, p + 1) if causal else kl)) if window else 0
        return hi - lo + first - max(0, min(hi, first) - lo)

    return sum(seen(p) for p in range(kl - ql, kl))


def work(case):
    if case["op"] == "store":
        e = _SIZE[case["dtype"]]
        real = case["tokens"] - case["padding"]
        return {"bytes": 4 * e * real * case["kv_heads"] * case["dim"] + 4 * case["tokens"], "flops": 0}
    if case["op"] == "map":
        rows, new = sum(_new_lengths(case)) + case["padding"], sum(_new_lengths(case))
        # The lengths, the sums, an entry of the table read and one written per page, two numbers written per row.
        return {"bytes": 4 * (5 * case["batch"] + 2 * (new // case["page"] + case["batch"]) + 2 * rows), "flops": 0}
    e, hq, hk, d = _SIZE[case["dtype"]], case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "paged":
        seen = sum(_pairs(1, n, True, case["window"], case["sinks"]) for n in _lengths(case["batch"], case["length"], case["ragged"]))
        return {"bytes": 2 * e * seen * hk * d + 2 * e * case["batch"] * hq * d + 4 * (seen // case["page"] + case["batch"]),
                "flops": 4 * seen * hq * d}
    lens = _lengths(case["batch"], case["q_len"], case["ragged"])
    pairs = sum(lens.count(n) * _pairs(n, n if case["ragged"] else case["k_len"], case["causal"], case["window"], case["sinks"])
                for n in set(lens))
    q_rows = sum(lens)
    k_rows = q_rows if case["ragged"] else case["batch"] * case["k_len"]
    back = case["op"] == "att_back"
    values = (4 if back else 2) * q_rows * hq * d + (4 if back else 2) * k_rows * hk * d
    return {"bytes": e * values + (4 * q_rows * hq if case["save"] else 0), "flops": (10 if back else 4) * pairs * hq * d}


def _exact_mask(ql, kl, c):
    p = torch.arange(kl - ql, kl, device="cuda").unsqueeze(1)
    j = torch.arange(kl, device="cuda").unsqueeze(0)
    hidden = torch.zeros(ql, kl, dtype=torch.bool, device="cuda")
    if c["causal"]:
        hidden |= j > p
    if c["window"]:
        hidden |= ((j <= p - c["window"]) | (j >= p + c["window"])) & (j >= c["sinks"])
    return hidden


def _exact_one(q, k, v, hidden, scale):
    """One head of one sequence in fp64: (out, lse); a query that sees nothing gives zeros and -inf."""
    x = torch.mm(q, k.T).mul(scale).masked_fill(hidden, -math.inf)
    lse = torch.logsumexp(x, dim=1)
    none = torch.isinf(lse)
    w = torch.exp(x - lse.masked_fill(none, 0.0).unsqueeze(1))
    return torch.mm(w, v), lse


def exact(case, seed):
    """The definitions in fp64, one head of one sequence after the other; gradients by differentiating."""
    if case["op"] == "map":
        return None
    s = prepare(case, seed)
    if case["op"] == "store":
        return None  # copies: compared with the plain form
    scale = 1 / math.sqrt(case["dim"])
    hq, hk = case["heads"], case["kv_heads"]
    if case["op"] == "paged":
        ps, out = case["page"], torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        for b, n in enumerate(_lengths(case["batch"], case["length"], case["ragged"])):
            pages = s["table"][b, :(n + ps - 1) // ps].long()
            hidden = _exact_mask(1, n, {**case, "causal": True})[0]
            keep = (~hidden).nonzero().flatten()
            k = s["k_cache"][pages[keep // ps], keep % ps].double()
            v = s["v_cache"][pages[keep // ps], keep % ps].double()
            q = s["q"][b].double()
            for h in range(hk):
                g = slice(h * hq // hk, (h + 1) * hq // hk)
                out[b, g] = torch.mm(torch.softmax(torch.mm(q[g], k[:, h].T.contiguous()) * scale, dim=1), v[:, h].contiguous())
        return {"out": out}
    packed = case["ragged"]
    lens = _lengths(case["batch"], case["q_len"], packed)
    back = case["op"] == "att_back"
    grads = {n: torch.zeros(s[n].shape, dtype=torch.float64, device="cuda") for n in ("q", "k", "v")}
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:-1], dtype=torch.float64, device="cuda")
    first = _sums(lens)
    for b, n in enumerate(lens):
        at = (slice(first[b], first[b + 1]),) if packed else (b,)
        hidden = _exact_mask(n, n if packed else case["k_len"], case)
        for h in range(hq):
            kh = h * hk // hq
            q, k, v = s["q"][at][:, h].double(), s["k"][at][:, kh].double(), s["v"][at][:, kh].double()
            if back:
                q, k, v = q.requires_grad_(), k.requires_grad_(), v.requires_grad_()
                o, _ = _exact_one(q, k, v, hidden, scale)
                got = torch.autograd.grad(o, [q, k, v], grad_outputs=s["d_out"][at][:, h].double())
                for name, head, g in zip("qkv", (h, kh, kh), got):
                    grads[name][at][:, head] += g
            else:
                out[at][:, h], lse[at][:, h] = _exact_one(q, k, v, hidden, scale)
    if back:
        return {"d" + n: g for n, g in grads.items()}
    return {"out": out, "lse": lse} if case["save"] else {"out": out}
