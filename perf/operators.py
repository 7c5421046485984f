"""The measured cases of the transformer-block operators.

Three operators that stand around the rotated attention of a block:

- norm: RMS norms before and after a block, with the per-sample scale and shift of a
  modulated norm, the gate on the block's output and the scaled residual, and their backward;
- ffn: the gated feed-forward block act(x Wg^T) * (x Wu^T), and its backward;
- q8: a linear layer in 8-bit integers, one scale a token and one a channel.

`run` computes a case in its plain form (elementary torch operations) or, where `own` is
true, with the calls a user makes of rope_ltx3drope_amd.
"""
from __future__ import annotations

import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_EPS = 1e-6


# ---- cases -------------------------------------------------------------------------------------

def _norm(name, kind, dtype, batch, rows, dim, params, post, gate, nxt, offset, res_scale):
    return {"name": name, "op": "norm", "kind": kind, "dtype": dtype, "batch": batch, "rows": rows, "dim": dim,
            "params": params, "post": post, "gate": gate, "next": nxt, "offset": offset, "res_scale": res_scale}


def _ffn(name, kind, dtype, tokens, dim, hidden, act):
    return {"name": name, "op": "ffn", "kind": kind, "dtype": dtype, "tokens": tokens, "dim": dim, "hidden": hidden,
            "act": act}


def _q8(name, dtype, tokens, dim, out, bias):
    return {"name": name, "op": "q8", "dtype": dtype, "tokens": tokens, "dim": dim, "out": out, "bias": bias}


def listed():
    return [
        # one new token of four sequences in a text model: norm after the block, residual, next norm
        _norm("norm_token", "after", "bf16", 4, 1, 4096, "bf16", True, False, True, 1.0, 1.0),
        # a modulated norm before a block, three ragged samples of a width that no vector divides
        _norm("norm_ragged_f32", "before", "f32", 3, 1021, 2053, "f32", False, False, True, 0.0, 1.0),
        # a block of a diffusion transformer over a 17x34x60 grid: gate, residual, next modulated norm
        _norm("norm_grid", "after", "bf16", 2, 34680, 2048, "f32", True, True, True, 0.0, 1.0),
        # the same in training, a 9x34x60 grid: every gradient of the gated residual and both norms
        _norm("norm_grid_backward", "after_backward", "bf16", 2, 18360, 2048, "f32", True, True, True, 0.0, 1.0),
        # one token through the feed-forward block: its weights are read once
        _ffn("ffn_token", "forward", "bf16", 1, 4096, 10240, "gelu_tanh"),
        # a prompt of 509 tokens through a block of odd width
        _ffn("ffn_ragged", "forward", "bf16", 509, 1544, 4331, "gelu_tanh"),
        # a long prompt, or a batch of them
        _ffn("ffn_prompt", "forward", "bf16", 8192, 4096, 10240, "silu"),
        # a training step's share of the block: forward, then the gradients of input and weights
        _ffn("ffn_train", "train", "bf16", 4096, 2048, 8192, "silu"),
        # the same in 32 bits at odd sizes
        _ffn("ffn_train_f32", "train", "f32", 301, 1100, 2777, "gelu"),
        # one token through a down projection held in 8 bits
        _q8("q8_token", "bf16", 1, 10240, 4096, False),
        # a short prompt at odd sizes, 32-bit activations, with a bias
        _q8("q8_ragged", "f32", 77, 4100, 2053, True),
        # a long prompt through the down projection
        _q8("q8_prompt", "bf16", 8192, 10240, 4096, False),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """Widths: most are multiples of 64 or 8, some are any number."""
    step = rng.choice([64, 64, 8, 1])
    return max(step, _spread(rng, lo, hi) // step * step)


def _draw_once(rng):
    op = rng.choice(["norm", "ffn", "q8"])
    if op == "norm":
        kind = rng.choice(["before", "after", "before_backward", "after_backward"])
        return _norm("", kind, rng.choice(["bf16", "f32"]), rng.randint(1, 5), _spread(rng, 1, 35000),
                     _width(rng, 64, 8192), rng.choice(["bf16", "f32"]), rng.random() < 0.6, rng.random() < 0.6,
                     rng.random() < 0.7, rng.choice([0.0, 1.0]), rng.choice([1.0, 0.5]))
    if op == "ffn":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        return _ffn("", rng.choice(["forward", "train"]), dtype, _spread(rng, 1, 8192), _width(rng, 128, 4096),
                    _width(rng, 256, 10240), rng.choice(["silu", "gelu", "gelu_tanh"]))
    return _q8("", rng.choice(["bf16", "f32"]), _spread(rng, 1, 8192), _width(rng, 128, 10240),
               _width(rng, 128, 8192), rng.random() < 0.5)


def draw(rng):
    while True:
        c = _draw_once(rng)
        if c["op"] == "norm":
            if c["kind"].startswith("before"):
                c.update(post=False, gate=False, next=True, res_scale=1.0)
            if c["dtype"] == "f32":
                c["params"] = "f32"
        w = work(c)
        limit = 3e11 if c["dtype"] == "f32" and c["op"] == "ffn" else 1.2e12
        if w["bytes"] <= 1.1e9 and w["flops"] <= limit:
            del c["name"]
            return c


# ---- inputs ------------------------------------------------------------------------------------

def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["dtype"]]

    def normal(*shape, dtype=dt, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std + mean).to(dtype)

    if case["op"] == "norm":
        B, S, D = case["batch"], case["rows"], case["dim"]
        pt = _DT[case["params"]]
        t = {}
        mean_w = 1.0 - case["offset"]
        if case["kind"].startswith("before"):
            t["x"] = normal(B, S, D, std=2.0)
        else:
            t["y"] = normal(B, S, D)
            t["residual"] = normal(B, S, D, std=2.0)
            t["weight"] = normal(D, dtype=pt, std=0.2, mean=mean_w) if case["post"] else None
            t["gate"] = normal(B, D, dtype=pt, std=0.5) if case["gate"] else None
        if case["next"]:
            t["next_weight"] = normal(D, dtype=pt, std=0.2, mean=mean_w)
            modulated = case["gate"] or case["kind"].startswith("before")
            t["next_scale"] = normal(B, D, dtype=pt, std=0.3) if modulated else None
            t["next_shift"] = normal(B, D, dtype=pt, std=0.3) if modulated else None
        if case["kind"].endswith("backward"):
            if case["next"]:
                t["dn"] = normal(B, S, D)
            t["dr"] = normal(B, S, D)
            if not case["kind"].startswith("before"):
                # the residual that the forward pass kept, r = res_scale * residual + gate * post(y)
                t["r"] = _after_forward(t, case)[0].to(dt)
        return t
    if case["op"] == "ffn":
        M, D, F = case["tokens"], case["dim"], case["hidden"]
        t = {"x": normal(M, D), "w_gate": normal(F, D, std=1.5 / math.sqrt(D)),
             "w_up": normal(F, D, std=1.0 / math.sqrt(D))}
        if case["kind"] == "train":
            t["dh"] = normal(M, F)
        return t
    M, K, N = case["tokens"], case["dim"], case["out"]
    w = normal(N, K, dtype=torch.float32, std=1.0 / math.sqrt(K))
    w_scale = w.abs().amax(1) / 127.0
    return {"x": normal(M, K), "w8": torch.round(w / w_scale[:, None]).to(torch.int8), "w_scale": w_scale,
            "bias": normal(N, dtype=torch.float32, std=0.1) if case["bias"] else None}


def prepare(case, seed):
    return {"case": case, "t": _inputs(case, seed)}


# ---- the plain form ----------------------------------------------------------------------------

def _f(t):
    return None if t is None else t.float()


def _rms(x):
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS)
    return x * rstd, rstd


def _factor(w, scale, offset):
    """The factor on the normed row: (w + offset) * (1 + scale), broadcast over [batch, rows, dim]."""
    f = 1.0
    if w is not None:
        f = w + offset
    if scale is not None:
        f = f * (1.0 + scale[:, None, :])
    return f


def _after_forward(t, case):
    y, residual = _f(t["y"]), _f(t["residual"])
    if case["post"]:
        y = _rms(y)[0] * (_f(t["weight"]) + case["offset"])
    if case["gate"]:
        y = y * _f(t["gate"])[:, None, :]
    r = case["res_scale"] * residual + y
    if not case["next"]:
        return r, None
    return r, _before_forward(r, t, case)


def _before_forward(x, t, case):
    n = _rms(x)[0] * _factor(_f(t["next_weight"]), _f(t["next_scale"]), case["offset"])
    if t["next_shift"] is not None:
        n = n + _f(t["next_shift"])[:, None, :]
    return n


def _rms_backward(dxhat, xhat, rstd):
    return rstd * (dxhat - xhat * (dxhat * xhat).mean(-1, keepdim=True))


def _before_backward(x, dn, dr, t, case):
    """dx, dweight, dscale, dshift of the norm before a block; dr reaches x past the block."""
    xhat, rstd = _rms(x)
    w, scale = _f(t["next_weight"]), _f(t["next_scale"])
    dx = _rms_backward(dn * _factor(w, scale, case["offset"]), xhat, rstd) + dr
    per_sample = (dn * xhat).sum(1)
    dw = (per_sample if scale is None else per_sample * (1.0 + scale)).sum(0)
    if scale is None:
        return dx, dw, None, None
    return dx, dw, per_sample * (w + case["offset"]), dn.sum(1)


def _after_backward(t, case):
    y, r, dr = _f(t["y"]), _f(t["r"]), _f(t["dr"])
    out = {}
    if case["next"]:
        dr, out["dnext_weight"], out["dnext_scale"], out["dnext_shift"] = _before_backward(r, _f(t["dn"]), dr, t, case)
    out["dresidual"] = case["res_scale"] * dr
    yhat, rstd, post = y, None, y
    if case["post"]:
        w = _f(t["weight"]) + case["offset"]
        yhat, rstd = _rms(y)
        post = yhat * w
    dpost = dr
    if case["gate"]:
        out["dgate"] = (dr * post).sum(1)
        dpost = dr * _f(t["gate"])[:, None, :]
    if case["post"]:
        out["dweight"] = (dpost * yhat).sum((0, 1))
        out["dy"] = _rms_backward(dpost * w, yhat, rstd)
    else:
        out["dy"] = dpost
    return out


def _act(g, kind):
    """act(g) and its derivative."""
    if kind == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    if kind == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    a = math.sqrt(2.0 / math.pi)
    th = torch.tanh(a * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + th), 0.5 * (1.0 + th) + 0.5 * g * (1.0 - th * th) * a * (1.0 + 3 * 0.044715 * g * g)


def _cast_norm(out, t, case):
    """Row tensors in the activations' type, gradients of parameters in the parameters' type."""
    dt, pt = _DT[case["dtype"]], _DT[case["params"]]
    return {k: v.to(dt if k in ("r", "n", "dx", "dy", "dresidual") else pt) for k, v in out.items() if v is not None}


def _plain(case, t):
    if case["op"] == "norm":
        if case["kind"] == "before":
            out = {"n": _before_forward(_f(t["x"]), t, case)}
        elif case["kind"] == "after":
            r, n = _after_forward(t, case)
            out = {"r": r, "n": n}
        elif case["kind"] == "before_backward":
            dx, dw, dscale, dshift = _before_backward(_f(t["x"]), _f(t["dn"]), _f(t["dr"]), t, case)
            out = {"dx": dx, "dnext_weight": dw, "dnext_scale": dscale, "dnext_shift": dshift}
        else:
            out = _after_backward(t, case)
        return _cast_norm(out, t, case)
    dt = _DT[case["dtype"]]
    if case["op"] == "ffn":
        x, wg, wu = _f(t["x"]), _f(t["w_gate"]), _f(t["w_up"])
        g, u = x @ wg.t(), x @ wu.t()
        a, da = _act(g, case["act"])
        out = {"h": (a * u).to(dt)}
        if case["kind"] == "train":
            dh = _f(t["dh"])
            dg, du = dh * u * da, dh * a
            out["dx"] = (dg @ wg + du @ wu).to(dt)
            out["dw_gate"] = (dg.t() @ x).to(dt)
            out["dw_up"] = (du.t() @ x).to(dt)
        return out
    x = _f(t["x"])
    scale = x.abs().amax(1) / 127.0
    q = torch.where(scale[:, None] > 0, torch.round(x / scale[:, None]), torch.zeros_like(x))
    # a sum of products of 8-bit integers passes 2^24: 64 bits hold it exactly
    acc = q.double() @ t["w8"].double().t()
    y = acc * scale.double()[:, None] * t["w_scale"].double()
    if t["bias"] is not None:
        y = y + t["bias"].double()
    return {"y": y.to(dt), "q": q.to(torch.int8), "scale": scale}


# ---- the framework's operators ------------------------------------------------------------------

def _own(case, t):
    import rope_ltx3drope_amd as rla

    if case["op"] == "norm":
        kw = {"eps": _EPS, "weight_offset": case["offset"]}
        nxt = {"next_weight": t["next_weight"], "next_scale": t["next_scale"],
               "next_shift": t["next_shift"]} if case["next"] else {"next_norm": False}
        if case["kind"] == "before":
            return {"n": rla.norm_before(t["x"], t["next_weight"], t["next_scale"], t["next_shift"], **kw)}
        if case["kind"] == "after":
            r, n = rla.norm_after(t["y"], t["residual"], t["weight"], t["gate"], post_norm=case["post"],
                                  residual_scale=case["res_scale"], **nxt, **kw)
            return {"r": r, "n": n} if case["next"] else {"r": r}
        if case["kind"] == "before_backward":
            g = rla.norm_before_backward(t["dn"], t["x"], t["next_weight"], t["next_scale"], t["next_shift"],
                                         dresidual=t["dr"], **kw)
            out = {"dx": g.dx, "dnext_weight": g.dweight, "dnext_scale": g.dscale, "dnext_shift": g.dshift}
        else:
            g = rla.norm_after_backward(t["dr"], t.get("dn"), t["y"], t["r"], t["weight"], t["gate"],
                                        post_norm=case["post"], residual_scale=case["res_scale"], **nxt, **kw)
            out = {"dnext_weight": g.dnext_weight, "dnext_scale": g.dnext_scale, "dnext_shift": g.dnext_shift,
                   "dresidual": g.dresidual, "dgate": g.dgate, "dweight": g.dweight, "dy": g.dy}
            if not case["next"]:
                for k in ("dnext_weight", "dnext_scale", "dnext_shift"):
                    del out[k]
        return {k: v for k, v in out.items() if v is not None}
    if case["op"] == "ffn":
        if case["kind"] == "forward":
            return {"h": rla.gated_ffn(t["x"], t["w_gate"], t["w_up"], case["act"])}
        h, g, u = rla.gated_ffn(t["x"], t["w_gate"], t["w_up"], case["act"], save=True)
        dx, dwg, dwu = rla.gated_ffn_backward(t["dh"], t["x"], t["w_gate"], t["w_up"], g, u, case["act"])
        return {"h": h, "dx": dx, "dw_gate": dwg, "dw_up": dwu}
    q, scale = rla.q8_quantize(t["x"])
    y = rla.q8_matmul(q, scale, t["w8"], t["w_scale"], bias=t["bias"], dtype=_DT[case["dtype"]])
    return {"y": y, "q": q, "scale": scale}


def run(state):
    return (_own if own else _plain)(state["case"], state["t"])


# ---- the work that a pass cannot do without -----------------------------------------------------

def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm":
        n = case["batch"] * case["rows"] * case["dim"]
        row = n * es
        ps = 4 if case["params"] == "f32" else 2
        modulated = case["gate"] or case["kind"].startswith("before")
        vec = (case["post"] + case["next"]) * case["dim"] * ps
        vec += (case["gate"] + (2 * modulated if case["next"] else 0)) * case["batch"] * case["dim"] * ps
        if case["kind"] == "before":
            return {"bytes": 2 * row + vec, "flops": 6 * n}
        if case["kind"] == "after":
            return {"bytes": (3 + case["next"]) * row + vec, "flops": 12 * n}
        if case["kind"] == "before_backward":
            return {"bytes": 4 * row + 2 * vec, "flops": 14 * n}
        # r is needed for the next norm's gradient only, y for the post norm's or the gate's only
        reads = 1 + 2 * case["next"] + (case["post"] or case["gate"])
        return {"bytes": (reads + 2) * row + 2 * vec, "flops": 28 * n}
    if case["op"] == "ffn":
        M, D, F = case["tokens"], case["dim"], case["hidden"]
        io = M * D + 2 * F * D + M * F
        if case["kind"] == "forward":
            return {"bytes": io * es, "flops": 4 * M * D * F}
        return {"bytes": (io + M * F + M * D + 2 * F * D) * es, "flops": 12 * M * D * F}
    M, K, N = case["tokens"], case["dim"], case["out"]
    return {"bytes": M * K * es + M * K + 4 * M + N * K + 4 * N * (1 + case["bias"]) + M * N * es,
            "flops": 2 * M * K * N}


# ---- the definitions in 64 bits ------------------------------------------------------------------

def exact(case, seed):
    t = {k: (v if v is None or v.dtype == torch.int8 else v.double()) for k, v in _inputs(case, seed).items()}
    if case["op"] == "norm":
        return _exact_norm(case, t)
    if case["op"] == "ffn":
        return _exact_ffn(case, t)
    # the definition's scale and quotient are 32-bit numbers: |x| max / 127 and x / scale, each rounded
    x = _inputs(case, seed)["x"].float()
    scale = x.abs().max(dim=1).values.div(torch.full((1,), 127.0, device=x.device))
    quot = x.div(scale.clamp_min(torch.finfo(torch.float32).tiny).unsqueeze(1))
    q = quot.round().double()
    y = torch.mm(q, t["w8"].double().transpose(0, 1).contiguous())
    y.mul_(scale.double().unsqueeze(1)).mul_(t["w_scale"].unsqueeze(0))
    if t["bias"] is not None:
        y.add_(t["bias"].unsqueeze(0))
    return {"y": y, "q": q, "scale": scale.double()}


def _exact_norm(case, t):
    D = case["dim"]
    off = case["offset"]

    def inv_norm(v):
        return 1.0 / torch.sqrt(v.pow(2).sum(-1, keepdim=True) / D + _EPS)

    before = case["kind"].startswith("before")
    if not case["kind"].endswith("backward"):
        out = {}
        if before:
            r = t["x"]
        else:
            branch = t["y"]
            if case["post"]:
                branch = branch * inv_norm(branch) * (t["weight"] + off)
            if case["gate"]:
                branch = branch * t["gate"].unsqueeze(1)
            r = t["residual"] * case["res_scale"] + branch
            out["r"] = r
        if case["next"]:
            n = r * inv_norm(r) * (t["next_weight"] + off)
            if t["next_scale"] is not None:
                n = n * (t["next_scale"].unsqueeze(1) + 1.0) + t["next_shift"].unsqueeze(1)
            out["n"] = n
        return out
    out = {}
    grad = t["dr"]
    if case["next"]:
        r = t["x"] if before else t["r"]
        a = inv_norm(r)
        hat = r * a
        w = t["next_weight"] + off
        mod = 1.0 + t["next_scale"].unsqueeze(1) if t["next_scale"] is not None else torch.ones_like(w)
        out["dnext_weight"] = (t["dn"] * mod * hat).sum((0, 1))
        if t["next_scale"] is not None:
            out["dnext_scale"] = (t["dn"] * w * hat).sum(1)
            out["dnext_shift"] = t["dn"].sum(1)
        v = t["dn"] * w * mod
        grad = grad + a * v - hat * a * (v * hat).sum(-1, keepdim=True) / D
        del v, hat
    if before:
        out["dx"] = grad
        return out
    out["dresidual"] = grad * case["res_scale"]
    y = t["y"]
    a = inv_norm(y) if case["post"] else 1.0
    w = t["weight"] + off if case["post"] else 1.0
    gate = t["gate"].unsqueeze(1) if case["gate"] else 1.0
    hat = y * a
    if case["gate"]:
        out["dgate"] = (grad * hat * w).sum(1)
    if case["post"]:
        out["dweight"] = (grad * gate * hat).sum((0, 1))
        v = grad * gate * w
        out["dy"] = a * v - hat * a * (v * hat).sum(-1, keepdim=True) / D
    else:
        out["dy"] = grad * gate
    return out


def _exact_ffn(case, t):
    wg, wu, x = t["w_gate"], t["w_up"], t["x"]
    g = torch.mm(x, wg.transpose(0, 1).contiguous())
    u = torch.mm(x, wu.transpose(0, 1).contiguous())
    if case["act"] == "silu":
        sig = torch.sigmoid(g)
        a, da = g * sig, sig + g * sig * (1.0 - sig)
    elif case["act"] == "gelu":
        phi = torch.erfc(-g / math.sqrt(2.0)) / 2.0
        a, da = g * phi, phi + g * torch.exp(-g.pow(2) / 2.0) / math.sqrt(2.0 * math.pi)
    else:
        # (1 + tanh z) / 2 is the logistic function of 2 z
        z2 = math.sqrt(8.0 / math.pi) * (g + 0.044715 * g.pow(3))
        sig = torch.sigmoid(z2)
        a = g * sig
        da = sig + g * sig * (1.0 - sig) * math.sqrt(8.0 / math.pi) * (1.0 + 0.134145 * g.pow(2))
    out = {"h": a * u}
    if case["kind"] == "train":
        dg, du = t["dh"] * u * da, t["dh"] * a
        out["dx"] = torch.mm(dg, wg) + torch.mm(du, wu)
        out["dw_gate"] = torch.mm(dg.transpose(0, 1).contiguous(), x)
        out["dw_up"] = torch.mm(du.transpose(0, 1).contiguous(), x)
    return out
