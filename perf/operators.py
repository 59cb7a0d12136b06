"""The feed-forward operators as measured cases: the norms around a block
(residual_norm), the gated feed-forward product (glu) and the matrix product
with its epilogue (linear), each forward and backward.

Where ``own`` is false ``run`` computes the plain form: elementary torch
operations in fp32, rounded once at the end. Where it is true, ``run`` calls
hyper_connection_rank_amd.

Sizes: hidden 2560 and 4 x 2560 = 10240 are the decode and prefill blocks' own
(C = 4, H = 2560), 4096 the wide block's; the rest is generic.
"""
import math

import torch

own = False

_T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}
_EPS = 1e-6


def listed():
    return [
        # One token of a decode step: both norms, the hyper-connection's gate of the row. Latency only.
        {"name": "norm_token", "op": "norm", "rows": 1, "hidden": 2560, "dtype": "bf16", "gate": "row", "post": True},
        # A prompt of 8192 tokens at the prefill block's width.
        {"name": "norm_prompt", "op": "norm", "rows": 8192, "hidden": 2560, "dtype": "bf16", "gate": "row", "post": True},
        # Training step at the wide block's width, all gradients.
        {"name": "norm_train", "op": "norm_back", "rows": 8192, "hidden": 4096, "dtype": "f16", "gate": "row", "post": True},
        # Odd rows and odd width in fp32 with a gate per element, all gradients.
        {"name": "norm_odd", "op": "norm_back", "rows": 1021, "hidden": 2057, "dtype": "f32", "gate": "element", "post": True},
        # One token through the gate and up projections: the weights' bytes.
        {"name": "glu_token", "op": "glu", "rows": 1, "in": 2560, "out": 10240, "dtype": "bf16", "act": "silu", "bias": False, "save": False},
        # A serving batch of 48 sequences at the wide block's width.
        {"name": "glu_batch", "op": "glu", "rows": 48, "in": 4096, "out": 12288, "dtype": "f16", "act": "gelu_tanh", "bias": False, "save": False},
        # Training forward of 8192 tokens, g and u kept for the backward pass.
        {"name": "glu_train", "op": "glu", "rows": 8192, "in": 2560, "out": 10240, "dtype": "bf16", "act": "silu", "bias": False, "save": True},
        # The backward pass of 4096 tokens: gradients of x, both weights and both biases.
        {"name": "glu_back", "op": "glu_back", "rows": 4096, "in": 2560, "out": 10240, "dtype": "bf16", "act": "silu", "bias": True, "save": True},
        # The down projection of eight sequences' tokens, added to the residual.
        {"name": "linear_tokens", "op": "linear", "rows": 8, "in": 10240, "out": 2560, "dtype": "bf16", "act": "none", "bias": True, "residual": True},
        # The down projection of a prompt, added to the residual.
        {"name": "linear_prompt", "op": "linear", "rows": 8192, "in": 10240, "out": 2560, "dtype": "bf16", "act": "none", "bias": True, "residual": True},
        # A projection with activation, backward, at a ragged token count.
        {"name": "linear_back", "op": "linear_back", "rows": 2011, "in": 2560, "out": 4096, "dtype": "f16", "act": "gelu", "bias": True, "residual": False},
        # Odd sizes in every dimension, fp32.
        {"name": "linear_odd", "op": "linear", "rows": 301, "in": 1003, "out": 777, "dtype": "f32", "act": "silu", "bias": True, "residual": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """Rows 1 to 8192 and widths 64 to 16384, over their logarithms; a third
    of the widths are odd numbers, the rest multiples of 8."""
    def width(lo, hi):
        n = _log_int(rng, lo, hi)
        return n | 1 if rng.random() < 1 / 3 else max(8, n & ~7)

    op = rng.choice(["norm", "norm_back", "glu", "glu_back", "linear", "linear_back"])
    dtype = rng.choice(["bf16", "f16", "bf16", "f16", "f32"])
    rows = _log_int(rng, 1, 8192)
    if op.startswith("norm"):
        hidden = width(64, 16384)
        rows = min(rows, 8192 * 4096 // hidden)
        return {"op": op, "rows": rows, "hidden": hidden, "dtype": dtype, "gate": rng.choice(["none", "row", "element"]),
                "post": rng.random() < 0.75}
    k, n = width(64, 12288), width(64, 12288)
    # No more work than the largest listed case (fp32: an eighth of it).
    most = 8192 * 2560 * 10240 // (8 if dtype == "f32" else 1) // (2 if op.endswith("back") else 1)
    rows = max(1, min(rows, most // (k * n)))
    case = {"op": op, "rows": rows, "in": k, "out": n, "dtype": dtype, "bias": rng.random() < 0.5}
    if op.startswith("glu"):
        case["act"] = rng.choice(["silu", "gelu", "gelu_tanh", "relu", "sigmoid"])
        case["save"] = op == "glu_back" or rng.random() < 0.5
    else:
        case["act"] = rng.choice(["none", "silu", "gelu", "gelu_tanh", "relu", "sigmoid"])
        case["residual"] = op == "linear" and rng.random() < 0.5
    return case


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = _T[case["dtype"]]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dt)

    s = {"case": case}
    m = case["rows"]
    if case["op"].startswith("norm"):
        h = case["hidden"]
        s["y"] = normal(m, h)
        s["residual"] = normal(m, h, std=2.0)  # backward: the saved residual_out
        s["pre_scale"] = 1 + normal(h, std=0.1)
        s["post_scale"] = 1 + normal(h, std=0.1) if case["post"] else None
        s["gate"] = None
        if case["gate"] == "row":  # one column of a block's post_gate [rows, 4], sigmoid * 2
            s["gate"] = (2 * torch.sigmoid(torch.randn(m, 4, generator=gen, device="cuda"))).to(dt)[:, 1]
        elif case["gate"] == "element":
            s["gate"] = torch.sigmoid(torch.randn(m, h, generator=gen, device="cuda")).to(dt)
        if case["op"] == "norm_back":
            s["d_residual_out"] = normal(m, h)
            s["d_normed"] = normal(m, h)
        return s
    k, n = case["in"], case["out"]
    s["x"] = normal(m, k)
    glu = case["op"].startswith("glu")
    for name in ("wg", "wu") if glu else ("w",):
        s[name] = normal(k, n, std=k ** -0.5)
    for name in ("bg", "bu") if glu else ("b",):
        s[name] = normal(n, std=0.1) if case["bias"] else None
    if case["op"] == "linear":
        s["residual"] = normal(m, n, std=2.0) if case["residual"] else None
    elif case["op"] == "glu_back":
        s["g"], s["u"], s["dh"] = normal(m, n), normal(m, n), normal(m, n)
    elif case["op"] == "linear_back":
        s["preact"] = normal(m, n) if case["act"] != "none" else None
        s["dy"] = normal(m, n)
    return s


# ---------------------------------------------------------------- plain form

_GELU_C = math.sqrt(2 / math.pi)


def _sig(x):
    return 1 / (1 + torch.exp(-x))


def _act(name, x):
    if name == "none":
        return x
    if name == "relu":
        return torch.where(x > 0, x, torch.zeros_like(x))
    if name == "sigmoid":
        return _sig(x)
    if name == "silu":
        return x * _sig(x)
    if name == "gelu":
        return 0.5 * x * (1 + torch.erf(x * math.sqrt(0.5)))
    return 0.5 * x * (1 + torch.tanh(_GELU_C * (x + 0.044715 * x * x * x)))


def _dact(name, x):
    if name == "none":
        return torch.ones_like(x)
    if name == "relu":
        return torch.where(x > 0, torch.ones_like(x), torch.zeros_like(x))
    if name == "sigmoid":
        s = _sig(x)
        return s * (1 - s)
    if name == "silu":
        s = _sig(x)
        return s * (1 + x * (1 - s))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(x * math.sqrt(0.5))) + x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
    t = torch.tanh(_GELU_C * (x + 0.044715 * x * x * x))
    return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * _GELU_C * (1 + 3 * 0.044715 * x * x)


def _f(t):
    return None if t is None else t.float()


def _plain_norm(s):
    y, r = _f(s["y"]), _f(s["residual"])
    z = y
    if s["post_scale"] is not None:
        z = y / torch.sqrt((y * y).mean(1, keepdim=True) + _EPS) * _f(s["post_scale"])
    if s["gate"] is not None:
        g = _f(s["gate"])
        z = z * (g[:, None] if g.dim() == 1 else g)
    r = r + _ALPHA * z
    n = r / torch.sqrt((r * r).mean(1, keepdim=True) + _EPS) * _f(s["pre_scale"])
    dt = s["y"].dtype
    return {"residual_out": r.to(dt), "normed": n.to(dt)}


def _plain_norm_back(s):
    y, r, dr, dn, w = (_f(s[k]) for k in ("y", "residual", "d_residual_out", "d_normed", "pre_scale"))
    post, gate = _f(s["post_scale"]), _f(s["gate"])
    rr = 1 / torch.sqrt((r * r).mean(1, keepdim=True) + _EPS)
    nh = r * rr
    t = dn * w
    d = dr + rr * (t - nh * (t * nh).mean(1, keepdim=True))
    out = {"d_residual": d, "d_pre_scale": (dn * nh).sum(0)}
    yh = z = y
    if post is not None:
        ry = 1 / torch.sqrt((y * y).mean(1, keepdim=True) + _EPS)
        yh = y * ry
        z = yh * post
    dz = _ALPHA * d
    if gate is not None:
        zd = _ALPHA * z * d
        out["d_gate"] = zd.sum(1) if gate.dim() == 1 else zd
        dz = dz * (gate[:, None] if gate.dim() == 1 else gate)
    dy = dz
    if post is not None:
        out["d_post_scale"] = (dz * yh).sum(0)
        q = dz * post
        dy = ry * (q - yh * (q * yh).mean(1, keepdim=True))
    out["dy"] = dy
    dt = s["y"].dtype
    return {k: v.to(dt) for k, v in out.items()}


def _plain_glu(s):
    c, x = s["case"], _f(s["x"])
    g, u = x @ _f(s["wg"]), x @ _f(s["wu"])
    if c["bias"]:
        g, u = g + _f(s["bg"]), u + _f(s["bu"])
    out = {"h": _act(c["act"], g) * u}
    if c["save"]:
        out["g"], out["u"] = g, u
    return {k: v.to(s["x"].dtype) for k, v in out.items()}


def _plain_glu_back(s):
    c, x, g, u, dh = s["case"], _f(s["x"]), _f(s["g"]), _f(s["u"]), _f(s["dh"])
    dg = dh * u * _dact(c["act"], g)
    du = dh * _act(c["act"], g)
    out = {"dx": dg @ _f(s["wg"]).t() + du @ _f(s["wu"]).t(), "d_gate_weight": x.t() @ dg, "d_up_weight": x.t() @ du}
    if c["bias"]:
        out["d_gate_bias"], out["d_up_bias"] = dg.sum(0), du.sum(0)
    return {k: v.to(s["x"].dtype) for k, v in out.items()}


def _plain_linear(s):
    c = s["case"]
    p = _f(s["x"]) @ _f(s["w"])
    if c["bias"]:
        p = p + _f(s["b"])
    y = _act(c["act"], p)
    if c["residual"]:
        y = y + _f(s["residual"])
    return {"y": y.to(s["x"].dtype)}


def _plain_linear_back(s):
    c = s["case"]
    dz = _f(s["dy"])
    if c["act"] != "none":
        dz = dz * _dact(c["act"], _f(s["preact"]))
    out = {"dx": dz @ _f(s["w"]).t(), "d_weight": _f(s["x"]).t() @ dz}
    if c["bias"]:
        out["d_bias"] = dz.sum(0)
    return {k: v.to(s["x"].dtype) for k, v in out.items()}


_ALPHA = 0.5  # the residual scale of the norm cases
_PLAIN = {"norm": _plain_norm, "norm_back": _plain_norm_back, "glu": _plain_glu, "glu_back": _plain_glu_back,
          "linear": _plain_linear, "linear_back": _plain_linear_back}


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
    if op == "norm":
        r, n = hc.residual_norm(s["y"], s["residual"], gate=s["gate"], post_scale=s["post_scale"], pre_scale=s["pre_scale"],
                                post_norm=c["post"], alpha=_ALPHA, epsilon=_EPS)
        return {"residual_out": r, "normed": n}
    if op == "norm_back":
        ws = _workspace(hc.residual_norm_workspace_size(c["rows"], c["hidden"], s["y"].dtype))
        dy, dr, dg, dpost, dpre = hc.residual_norm_backward(
            s["y"], s["residual"], s["d_residual_out"], s["d_normed"], gate=s["gate"], post_scale=s["post_scale"],
            pre_scale=s["pre_scale"], post_norm=c["post"], alpha=_ALPHA, epsilon=_EPS, workspace=ws)
        out = {"d_residual": dr, "d_pre_scale": dpre}
        if dg is not None:
            out["d_gate"] = dg
        if dpost is not None:
            out["d_post_scale"] = dpost
        out["dy"] = dy
        return out
    back = op.endswith("back")
    size = hc.glu_workspace_size if op.startswith("glu") else hc.linear_workspace_size
    ws = _workspace(size(c["rows"], c["in"], c["out"], s["x"].dtype, backward=back))
    if op == "glu":
        got = hc.glu(s["x"], s["wg"], s["wu"], s["bg"], s["bu"], activation=c["act"], save=c["save"], workspace=ws)
        return dict(zip(("h", "g", "u"), got)) if c["save"] else {"h": got}
    if op == "glu_back":
        got = hc.glu_backward(s["x"], s["wg"], s["wu"], s["g"], s["u"], s["dh"], activation=c["act"], bias=c["bias"], workspace=ws)
        return {k: v for k, v in zip(("dx", "d_gate_weight", "d_up_weight", "d_gate_bias", "d_up_bias"), got) if v is not None}
    if op == "linear":
        return {"y": hc.linear(s["x"], s["w"], s["b"], s["residual"], activation=c["act"], workspace=ws)}
    got = hc.linear_backward(s["x"], s["w"], s["dy"], s["preact"], activation=c["act"], bias=c["bias"], workspace=ws)
    return {k: v for k, v in zip(("dx", "d_weight", "d_bias"), got) if v is not None}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- work and the exact results

def work(case):
    e = _SIZE[case["dtype"]]
    m = case["rows"]
    if case["op"].startswith("norm"):
        h = case["hidden"]
        back = case["op"] == "norm_back"
        gate = {"none": 0, "row": m, "element": m * h}[case["gate"]] * (2 if back else 1)
        scales = h * (2 if case["post"] else 1) * (2 if back else 1)
        return {"bytes": e * ((6 if back else 4) * m * h + gate + scales), "flops": m * h * (22 if back else 9)}
    k, n = case["in"], case["out"]
    two = 2 if case["op"].startswith("glu") else 1
    weights = two * k * n
    bias = two * n if case["bias"] else 0
    if case["op"].endswith("back"):
        acts = m * k * 2 + m * n * (3 if two == 2 else (2 if case["act"] != "none" else 1))
        return {"bytes": e * (acts + 2 * weights + bias), "flops": 4 * m * weights}
    acts = m * k + m * n * (1 + (2 if case.get("save") else 0) + (1 if case.get("residual") else 0))
    return {"bytes": e * (acts + weights + bias), "flops": 2 * m * weights}


def _act64(name, x):
    nn = torch.nn.functional
    return {"none": lambda v: v, "relu": nn.relu, "sigmoid": torch.sigmoid, "silu": nn.silu, "gelu": nn.gelu,
            "gelu_tanh": lambda v: nn.gelu(v, approximate="tanh")}[name](x)


def exact(case, seed):
    """The definitions in fp64; gradients by differentiating the forward definition."""
    s = {k: v.double() if torch.is_tensor(v) else v for k, v in prepare(case, seed).items()}

    def rms_norm(v, scale):
        return v * torch.rsqrt(v.pow(2).mean(-1, keepdim=True) + _EPS) * scale

    def branch(y, gate, post):
        z = y if post is None else rms_norm(y, post)
        if gate is None:
            return _ALPHA * z
        return _ALPHA * (gate.unsqueeze(1) if gate.dim() == 1 else gate) * z

    def grads(pairs, cotangents, leaves):
        """{name: gradient} of sum <output, cotangent> with respect to the named leaves."""
        total = sum((o * c).sum() for o, c in zip(pairs, cotangents))
        return dict(zip(leaves, torch.autograd.grad(total, list(leaves.values()))))

    op = case["op"]
    if op == "norm":
        r = s["residual"] + branch(s["y"], s["gate"], s["post_scale"])
        return {"residual_out": r, "normed": rms_norm(r, s["pre_scale"])}
    if op == "norm_back":
        r, pre = s["residual"].requires_grad_(), s["pre_scale"].requires_grad_()
        top = grads([rms_norm(r, pre)], [s["d_normed"]], {"r": r, "pre": pre})
        d = s["d_residual_out"] + top["r"]
        leaves = {"dy": s["y"].requires_grad_()}
        if s["gate"] is not None:
            leaves["d_gate"] = s["gate"].requires_grad_()
        if s["post_scale"] is not None:
            leaves["d_post_scale"] = s["post_scale"].requires_grad_()
        low = grads([branch(s["y"], s["gate"], s["post_scale"])], [d], leaves)
        return {"d_residual": d, "d_pre_scale": top["pre"],
                **{k: low[k] for k in ("d_gate", "d_post_scale", "dy") if k in low}}
    x = s["x"]
    if op == "glu":
        g = torch.mm(x, s["wg"]) if s["bg"] is None else torch.addmm(s["bg"], x, s["wg"])
        u = torch.mm(x, s["wu"]) if s["bu"] is None else torch.addmm(s["bu"], x, s["wu"])
        out = {"h": _act64(case["act"], g).mul(u)}
        return {**out, "g": g, "u": u} if case["save"] else out
    if op == "glu_back":
        g, u = s["g"].requires_grad_(), s["u"].requires_grad_()
        d = grads([_act64(case["act"], g) * u], [s["dh"]], {"g": g, "u": u})
        out = {"dx": torch.mm(d["g"], s["wg"].T).addmm(d["u"], s["wu"].T),
               "d_gate_weight": torch.mm(x.T, d["g"]), "d_up_weight": torch.mm(x.T, d["u"])}
        if case["bias"]:
            out["d_gate_bias"], out["d_up_bias"] = d["g"].sum(dim=0), d["u"].sum(dim=0)
        return out
    if op == "linear":
        p = torch.mm(x, s["w"]) if s["b"] is None else torch.addmm(s["b"], x, s["w"])
        y = _act64(case["act"], p)
        return {"y": y if s["residual"] is None else s["residual"].add(y)}
    dz = s["dy"]
    if s["preact"] is not None:
        p = s["preact"].requires_grad_()
        dz = grads([_act64(case["act"], p)], [dz], {"p": p})["p"]
    out = {"dx": torch.mm(dz, s["w"].T), "d_weight": torch.mm(x.T, dz)}
    if case["bias"]:
        out["d_bias"] = dz.sum(dim=0)
    return out
