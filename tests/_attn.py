"""The attention operators in fp64 and the error bounds of their tests.

U, F and ``within`` as in ``_ffn``. The bounds add up, for one query:
 - a score: an fp32 sum over dim products, 8 F sqrt(dim) (2-norm of the
   products + |s|) times the scale (see ``_ffn.product``); then the factor
   log2 e, the subtraction of the maximum (or of lse, itself multiplied) and
   the exponential, whose errors are relative to the exponents: 8 F (|s| +
   |m| + 1). So a weight's relative error is below e_j. The backward pass of
   16-bit types starts the sums of s and dP from -lse over the scale and
   -delta: their dim additions round relative to those too, 8 F sqrt(dim)
   (|lse| and |delta|) more.
 - weights rounded to T as 16-bit operands: every term of the sum over keys
   moves by an independent error with standard deviation below
   U |term| / sqrt(3); 4 U norm2(terms) is 6.9 of them. fp16 weights are kept
   2^7 times (backward 2^15 times) as large: where they fall below the normal
   numbers half a step is 2^-25, 2^-32 (2^-40) of the largest weight.
 - dS rounded to T likewise; in fp16 scaled so that a column's largest value
   so far is at least 2^11: half a step is 2^-36 of it.
 - the hardware's exponential has no subnormal results, nor have the matrix
   units subnormal operands: a weight or dS below 2^-126 may count as 0, an
   absolute error of at most 2^-126 each, LEAST = 2^-125 for both.
 - fp32 sums over n keys (or rows): 8 F sqrt(n) (norm2(terms) + |sum|), and a
   few rescalings of the sums, 64 F sum|terms|.
"""
from __future__ import annotations

import math

import torch

from _ffn import F, U

LEAST = 2.0 ** -125


def visible(ql, kl, causal, window, sinks, device="cuda"):
    p = torch.arange(ql, device=device)[:, None] + (kl - ql)
    j = torch.arange(kl, device=device)[None]
    see = torch.ones(ql, kl, dtype=torch.bool, device=device)
    if causal:
        see &= j <= p
    if window:
        see &= ((p - j).abs() < window) | (j < sinks)
    return see


def n2(a, b):
    return torch.sqrt((a * a) @ (b * b))


def head(q, k, v, see, scale, dt):
    """(out, bound, lse, bound) of one head of one sequence: q [ql, d], k and v [kl, d]."""
    q, k, v = q.double(), k.double(), v.double()
    d = q.shape[1]
    s = scale * (q @ k.t())
    es = 8 * F * math.sqrt(d) * (scale * n2(q, k.t()) + s.abs())
    s = s.masked_fill(~see, -math.inf)
    m = s.amax(1, keepdim=True) if s.shape[1] else s.new_full((s.shape[0], 1), -math.inf)
    none = m == -math.inf
    m = m.masked_fill(none, 0.0)
    x = torch.exp(s - m)
    n = x.sum(1, keepdim=True)
    p = x / n.masked_fill(none, 1.0)
    lse = (m + torch.log(n)).masked_fill(none, -math.inf)
    e = es + 8 * F * (s.masked_fill(~see, 0.0).abs() + m.abs() + 1)
    e = e.masked_fill(~see, 0.0)
    o = p @ v
    cnt = max(s.shape[1], 1)
    pv = torch.sqrt((p * p) @ (v * v))
    bound = (p * e) @ v.abs() + (p * e).sum(1, keepdim=True) * o.abs()
    bound = bound + 8 * F * math.sqrt(cnt) * (pv + 2 * o.abs()) + 64 * F * (p @ v.abs()) + LEAST * (see.double() @ v.abs())
    if dt != torch.float32:
        bound = bound + 4 * U(dt) * pv
    if dt == torch.float16:
        bound = bound + 2.0 ** -32 * (see.double() @ v.abs())
    el = (p * e).sum(1, keepdim=True) + 8 * F * math.sqrt(cnt) + 4 * F * lse.masked_fill(none, 0.0).abs() + 16 * F * (m.abs() + 1)
    return o, bound, lse[:, 0], el[:, 0]


def head_backward(q, k, v, out, lse, do, see, scale, dt):
    """{name: (exact, bound)} of one query head's dq and its parts of dk and dv, from the given out and lse."""
    q, k, v, out, lse, do = (t.double() for t in (q, k, v, out, lse, do))
    d, r = q.shape[1], math.sqrt(q.shape[1])
    s = scale * (q @ k.t())
    es = 8 * F * r * (scale * n2(q, k.t()) + s.abs())
    l0 = lse.masked_fill(lse == -math.inf, 0.0)[:, None]
    p = torch.exp(s - l0).masked_fill(~see, 0.0)
    low = dt != torch.float32
    e = es + 8 * F * (s.abs() + l0.abs() + 1) + (8 * F * r * l0.abs() if low else 0)
    dp = do @ v.t()
    edp = 8 * F * r * (n2(do, v.t()) + dp.abs())
    delta = (out * do).sum(1, keepdim=True)
    edl = 8 * F * r * (torch.sqrt((out * out * do * do).sum(1, keepdim=True)) + (2 if low else 1) * delta.abs())
    t = dp - delta
    ds = p * t
    seen = see.double()
    eds = p * (e * t.abs() + edp + edl + 4 * F * (dp.abs() + delta.abs())) + LEAST * seen * (1 + t.abs())

    def total(a, ea, b, small):
        """a^T b summed over a's rows, its bound; small: the absolute rounding of an operand that leaves the normal numbers."""
        x = a.t() @ b
        nx = torch.sqrt((a * a).t() @ (b * b))
        bound = ea.t() @ b.abs() + 8 * F * math.sqrt(max(a.shape[0], 1)) * (nx + x.abs()) + 64 * F * (a.abs().t() @ b.abs())
        if low:
            bound = bound + 4 * U(dt) * nx
        if dt == torch.float16:
            bound = bound + small * b.abs().sum(0)[None]
        return x, bound

    def top(a):
        return 2.0 ** -36 * (a.abs().amax(0)[:, None] if a.shape[0] else 0.0)

    dq, bq = total(ds.t(), eds.t(), k, top(ds.t()))
    dk, bk = total(ds, eds, q, top(ds))
    dv, bv = total(p, p * e + LEAST * seen, do, 2.0 ** -40)
    return {"dq": (scale * dq, scale * bq), "dk": (scale * dk, scale * bk), "dv": (dv, bv)}


def each(q, k, ql, kl):
    """(index of q's rows, index of k's rows) of every sequence of batched (ql None) or packed tensors."""
    if ql is None:
        if q.dim() == 3:
            return [((slice(None),), (slice(None),))]
        return [((b,), (b,)) for b in range(q.shape[0])]
    out, i, j = [], 0, 0
    for a, b in zip(ql, kl):
        out.append(((slice(i, i + a),), (slice(j, j + b),)))
        i, j = i + a, j + b
    return out


def attention(q, k, v, *, causal=True, window=0, sinks=0, scale=None, ql=None, kl=None):
    """(out, bound, lse, bound); ql, kl: the lengths of packed sequences. Rows of no sequence: zeros."""
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    bound, lse = out.clone(), out[..., 0].clone()
    el = lse.clone()
    g = q.shape[-2] // k.shape[-2]
    for a, b in each(q, k, ql, kl or ql):
        for h in range(q.shape[-2]):
            qq, kk, vv = q[a][:, h], k[b][:, h // g], v[b][:, h // g]
            see = visible(qq.shape[0], kk.shape[0], causal, window, sinks, q.device)
            out[a][:, h], bound[a][:, h], lse[a][:, h], el[a][:, h] = head(qq, kk, vv, see, scale, q.dtype)
    return out, bound, lse, el


def attention_backward(q, k, v, out, lse, do, *, causal=True, window=0, sinks=0, scale=None, ql=None, kl=None):
    """{name: (exact, bound)}."""
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    names = ("dq", "dk", "dv")
    got = {n: [torch.zeros(t.shape, dtype=torch.float64, device=q.device) for _ in range(2)] for n, t in zip(names, (q, k, v))}
    g = q.shape[-2] // k.shape[-2]
    for a, b in each(q, k, ql, kl or ql):
        for h in range(q.shape[-2]):
            qq, kk, vv = q[a][:, h], k[b][:, h // g], v[b][:, h // g]
            see = visible(qq.shape[0], kk.shape[0], causal, window, sinks, q.device)
            one = head_backward(qq, kk, vv, out[a][:, h], lse[a][:, h], do[a][:, h], see, scale, q.dtype)
            for n, at, hh in (("dq", a, h), ("dk", b, h // g), ("dv", b, h // g)):
                for i in range(2):
                    got[n][i][at][:, hh] += one[n][i]
    return {n: tuple(x) for n, x in got.items()}


def paged(q, kc, vc, table, lengths, *, window=0, sinks=0, scale=None):
    """(out, bound) of one token per sequence; keys on pages that the cache does not have are not seen."""
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    bound = out.clone()
    g = q.shape[1] // kc.shape[2]
    pages, ps = kc.shape[:2]
    for b, n in enumerate(lengths.tolist()):
        n = min(max(n, 0), table.shape[1] * ps)
        if n == 0:
            continue
        j = torch.arange(n, device=q.device)
        page = table[b].long()[j // ps]
        see = visible(1, n, True, window, sinks, q.device)[0] & (page >= 0) & (page < pages)
        at = j[see]
        k, v = kc[page[see], at % ps], vc[page[see], at % ps]
        for h in range(q.shape[1]):
            one = torch.ones(1, len(at), dtype=torch.bool, device=q.device)
            o, e, _, _ = head(q[b, h][None], k[:, h // g], v[:, h // g], one, scale, q.dtype)
            out[b, h], bound[b, h] = o[0], e[0]
    return out, bound


def page_map(cached, fresh, table, free, page, tokens, first=0):
    """The five arrays and the table, by counting (python numbers)."""
    table = [list(r) for r in table]
    starts, taken, lengths, positions, slots = [0], [0], [], [], []
    for b, (c, n) in enumerate(zip(cached, fresh)):
        c, n = max(c, 0), max(n, 0)
        held, need = -(-c // page), -(-(c + n) // page)
        for i in range(held, need):
            u = first + taken[-1] + i - held
            if i < len(table[b]):
                table[b][i] = free[u] if u < len(free) else -1
        for p in range(c, c + n):
            pg = table[b][p // page] if p // page < len(table[b]) else -1
            positions.append(p)
            slots.append(pg * page + p % page if pg >= 0 else -1)
        starts.append(starts[-1] + n)
        taken.append(taken[-1] + need - held)
        lengths.append(c + n)
    real = min(len(slots), tokens)
    positions = positions[:real] + [0] * (tokens - real)
    slots = slots[:real] + [-1] * (tokens - real)
    return starts, lengths, positions, slots, taken, table
