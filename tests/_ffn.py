"""The feed-forward operators in fp64 and the error bounds of their tests.

U[T] is half a step of T relative to the value (one rounding). F = 2^-24 is
the same for fp32. The bounds below add up:
 - one rounding of an output to T: U |value|;
 - fp32 sums. A sum over one row of a norm runs over at most 64 values per
   lane, six butterfly steps and up to 16 waves, so its error is at most
   86 F sum|terms|; 128 F sum|terms| also covers the products inside it and
   the steps after it. Sums over rows go through at most rows / 64 + 64 + 16
   additions (stated as ``n`` where used).
 - products' sums over K terms with independent signs: each addition rounds by
   at most F |partial sum|, the signs of the roundings are independent, and
   the partial sums stay within about 3 times the terms' 2-norm (or grow
   evenly to the result), so one standard deviation is below
   F sqrt(K) 3 norm2 / sqrt(3); 8 F sqrt(K) (norm2 + |result|) is over 4.6 of them.
 - a factor rounded to T before a product (dz of the backward passes): every
   term moves by an independent error with standard deviation below
   U |term| / sqrt(3); 4 U norm2(terms) is 6.9 of them.
"""
from __future__ import annotations

import math

import torch

T_OF = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
F = 2.0 ** -24


def U(dt):
    return torch.finfo(dt).eps / 2


def tiny(dt):
    """Half the spacing of T's subnormal numbers: the rounding error of values near zero."""
    return torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2


def rand(shape, dt, seed, std=1.0, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dt).to(device)


def within(got, exact, bound, label):
    """|got - exact| <= bound + one rounding of exact to got's type."""
    assert got.shape == exact.shape, (label, got.shape, exact.shape)
    dt = got.dtype
    err = (got.double() - exact).abs()
    tol = bound + U(dt) * (exact.abs() + bound) + tiny(dt)
    bad = ~(err <= tol)
    if bad.any():
        i = int((err / tol).nan_to_num(nan=math.inf).argmax())
        raise AssertionError(f"{label}: {int(bad.sum())} of {bad.numel()} off; worst at {i}: got "
                             f"{got.flatten()[i].item()}, exact {exact.flatten()[i].item()}, "
                             f"error {err.flatten()[i].item():.3e}, allowed {tol.flatten()[i].item():.3e}")


ACTS = {"none": lambda v: v, "relu": torch.relu, "sigmoid": torch.sigmoid, "silu": torch.nn.functional.silu,
        "gelu": torch.nn.functional.gelu, "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}


def act_and_slope(name, v):
    v = v.detach().clone().requires_grad_()
    a = ACTS[name](v)
    d, = torch.autograd.grad(a.sum(), v)
    return a.detach(), d


def product(x, w):
    """x @ w in fp64 and the bound of its fp32 sums."""
    x, w = x.double(), w.double()
    r = x @ w
    n2 = torch.sqrt((x * x) @ (w * w))
    return r, 8 * F * math.sqrt(x.shape[1]) * (n2 + r.abs())


def linear(x, w, b, res, act):
    """(y, bound, preact, preact's bound)."""
    p, e = product(x, w)
    if b is not None:
        p = p + b.double()
        e = e + 2 * F * (p.abs() + b.double().abs())
    a, d = act_and_slope(act, p)
    # the slope is at most 1.13 (gelu); the activation itself rounds a few times relative to |p|
    y, ey = a, 1.13 * e + (0 if act == "none" else 16) * F * (p.abs() + 1)
    if res is not None:
        y = y + res.double()
        ey = ey + 2 * F * (y.abs() + res.double().abs())
    return y, ey, p, e


def linear_backward(x, w, dy, preact, act):
    """{name: (exact, bound)} of dx, d_weight, d_bias."""
    dt = x.dtype
    dz = dy.double()
    if act != "none":
        dz = dz * act_and_slope(act, preact.double())[1]
    return _product_grads(x, [(w, dz, dy, act != "none")], dt)


def _slope_error(dz, dy):
    """fp32 error of dy times a slope: a few roundings relative to |dy| (slopes are at most 1.13)."""
    return 32 * F * dy.double().abs()


def _product_grads(x, branches, dt):
    """branches: (weight, exact dz, magnitude of the factor dz came from, whether dz is rounded to T)."""
    xd = x.double()
    dx = ex = 0
    out = {}
    for i, (w, dz, mag, rounded) in enumerate(branches):
        e = _slope_error(dz, mag) if rounded else torch.zeros_like(dz)
        wd = w.double()
        r, b = product(dz, wd.t())
        dx = dx + r
        ex = ex + b + e @ wd.abs().t()
        rw, bw = product(xd.t(), dz)
        bw = bw + xd.abs().t() @ e
        if rounded and dt != torch.float32:
            # dz rounded to T is off by at most U |dz|, or half a step of T's subnormal numbers where that is
            # more (fp16, |dz| < 2^-14: 2^-25); the latter's sum is at most 2^-25 times the factors' absolute sum
            ex = ex + 4 * U(dt) * torch.sqrt((dz * dz) @ (wd * wd).t()) + tiny(dt) * wd.abs().sum(1)
            bw = bw + 4 * U(dt) * torch.sqrt((xd * xd).t() @ (dz * dz)) + tiny(dt) * xd.abs().sum(0)[:, None]
        n = dz.shape[0] / 64 + 64 + 16
        out[f"dw{i}"] = (rw, bw)
        out[f"db{i}"] = (dz.sum(0), n * F * dz.abs().sum(0) + e.sum(0))
    out["dx"] = (dx, ex)
    return out


def glu(x, wg, wu, bg, bu, act):
    """{name: (exact, bound)} of h, g, u."""
    g, eg = product(x, wg)
    u, eu = product(x, wu)
    if bg is not None:
        g = g + bg.double()
        eg = eg + 2 * F * (g.abs() + bg.double().abs())
    if bu is not None:
        u = u + bu.double()
        eu = eu + 2 * F * (u.abs() + bu.double().abs())
    a = ACTS[act](g)
    ea = 1.13 * eg + 16 * F * (g.abs() + 1)
    return {"h": (a * u, (a.abs() + ea) * eu + ea * u.abs() + 2 * F * (a * u).abs()), "g": (g, eg), "u": (u, eu)}


def glu_backward(x, wg, wu, g, u, dh, act):
    a, d = act_and_slope(act, g.double())
    gd, ud, hd = g.double(), u.double(), dh.double()
    dg, du = hd * ud * d, hd * a
    return _product_grads(x, [(wg, dg, hd * ud, True), (wu, du, hd * (1 + gd.abs()), True)], x.dtype)


def norm(y, res, gate, post, pre, post_norm, alpha, eps):
    """{name: (exact, bound)} of residual_out and normed."""
    yd = y.double()
    z = yd
    if post_norm:
        z = yd * torch.rsqrt((yd * yd).mean(-1, keepdim=True) + eps)
    if post is not None:
        z = z * post.double()
    if gate is not None:
        z = z * (gate.double()[:, None] if gate.dim() == 1 else gate.double())
    z = alpha * z
    r = z if res is None else res.double() + z
    er = 128 * F * z.abs() + 2 * F * r.abs()
    rr = torch.rsqrt((r * r).mean(-1, keepdim=True) + eps)
    p = torch.ones_like(r[0]) if pre is None else pre.double()
    n = r * rr * p
    # r's error directly, and through rms: relative to it at most the rms of r's error over the rms of r
    en = er * rr * p.abs() + n.abs() * (torch.sqrt((er * er).mean(-1, keepdim=True)) * rr + 128 * F)
    return {"residual_out": (r, er), "normed": (n, en)}


def norm_backward(y, r, dres, dn, gate, post, pre, post_norm, alpha, eps):
    """{name: (exact, bound)}; every intermediate's bound is its magnitude (a sum of absolute values) times 128 F
    per row sum that it passed (three at most), and sums over rows add n F."""
    yd, rd = y.double(), r.double()
    one = torch.ones_like(rd[0])
    pw, qw = one if pre is None else pre.double(), one if post is None else post.double()
    rr = torch.rsqrt((rd * rd).mean(-1, keepdim=True) + eps)
    nh = rd * rr
    t = torch.zeros_like(rd) if dn is None else dn.double() * pw
    d0 = torch.zeros_like(rd) if dres is None else dres.double()
    d = d0 + rr * (t - nh * (t * nh).mean(-1, keepdim=True))
    dm = d0.abs() + rr * (t.abs() + nh.abs() * (t * nh).abs().mean(-1, keepdim=True))
    gd = torch.ones_like(rd[:, :1]) if gate is None else (gate.double()[:, None] if gate.dim() == 1 else gate.double())
    ry = torch.rsqrt((yd * yd).mean(-1, keepdim=True) + eps) if post_norm else torch.ones_like(rr)
    yh = yd * ry
    dz, dzm = alpha * gd * d, abs(alpha) * gd.abs() * dm
    q, qm = dz * qw, dzm * qw.abs()
    dy, dym = q, qm
    if post_norm:
        dy = ry * (q - yh * (q * yh).mean(-1, keepdim=True))
        dym = ry * (qm + yh.abs() * (qm * yh.abs()).mean(-1, keepdim=True))
    zd, zdm = alpha * yh * qw * d, abs(alpha) * (yh * qw).abs() * dm
    n = r.shape[0] / 64 + 64 + 16 + 768 / 16
    c = 128 * F
    out = {"dy": (dy, 3 * c * dym), "d_residual": (d, c * dm)}
    if gate is not None:
        out["d_gate"] = (zd.sum(-1), 3 * c * zdm.sum(-1)) if gate.dim() == 1 else (zd, 2 * c * zdm)
    if post is not None:
        out["d_post_scale"] = ((dz * yh).sum(0), (2 * c + n * F) * (dzm * yh.abs()).sum(0))
    if pre is not None:
        out["d_pre_scale"] = ((dn.double() * nh).sum(0), (c + n * F) * (dn.double() * nh).abs().sum(0))
    return out
