"""The measured cases of the operators from the residual stream to rotated queries and keys.

- ln: layer norm before and after a block, with weight and bias, the per-sample scale and shift of a
  modulated norm and the gate on the block's output, and their backward passes;
- f8: a linear layer in 8-bit floating point (e4m3) with one scale for every 128 numbers of a row and
  every 128 x 128 block of the weights, and a training step's products of it;
- axes: rotary positions with several axes (time, height, width), any position a token, forward and
  backward.

`run` computes a case in its plain form (elementary torch operations) or, where `own` is
true, with the calls a user makes of rope_ltx3drope_amd.
"""
from __future__ import annotations

import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_F8 = torch.float8_e4m3fn
_EPS = 1e-6
_BLOCK = 128
_TOP = 448.0  # the largest e4m3 number


# ---- cases -------------------------------------------------------------------------------------

def _ln(name, kind, dtype, batch, rows, dim, params, affine, gate, modulated):
    return {"name": name, "op": "ln", "kind": kind, "dtype": dtype, "batch": batch, "rows": rows, "dim": dim,
            "params": params, "affine": affine, "gate": gate, "modulated": modulated}


def _f8(name, kind, dtype, tokens, dim, out, bias):
    return {"name": name, "op": "f8", "kind": kind, "dtype": dtype, "tokens": tokens, "dim": dim, "out": out,
            "bias": bias}


def _axes(name, kind, dtype, batch, tokens, q_heads, k_heads, head_dim, widths, pairing, frequencies, positions, fused):
    return {"name": name, "op": "axes", "kind": kind, "dtype": dtype, "batch": batch, "tokens": tokens,
            "q_heads": q_heads, "k_heads": k_heads, "head_dim": head_dim, "width_t": widths[0], "width_h": widths[1],
            "width_w": widths[2], "pairing": pairing, "frequencies": frequencies, "positions": positions,
            "fused": fused}


def listed():
    return [
        # one new token of four sequences in a text model: residual, then the next norm with weight and bias
        _ln("ln_token", "after", "bf16", 4, 1, 4096, "bf16", True, False, False),
        # a modulated norm before a block, three ragged samples of a width that no vector divides
        _ln("ln_ragged_f32", "before", "f32", 3, 1021, 2053, "f32", False, False, True),
        # a block of a diffusion transformer over a 17x34x60 grid: gate, residual, next modulated norm
        _ln("ln_grid", "after", "bf16", 2, 34680, 2048, "f32", False, True, True),
        # the same in training, a 9x34x60 grid, the norm with weight and bias: every gradient
        _ln("ln_grid_backward", "after_backward", "bf16", 2, 18360, 2048, "f32", True, True, True),
        # one token through a down projection held in 8 bits
        _f8("f8_token", "forward", "bf16", 1, 10240, 4096, False),
        # a short prompt at odd sizes, 32-bit activations, with a bias
        _f8("f8_ragged", "forward", "f32", 77, 4100, 2053, True),
        # a long prompt through an up projection
        _f8("f8_prompt", "forward", "bf16", 8192, 4096, 10240, False),
        # a training step of one layer: the weights quantised too, the output, the input's and the weights' gradients
        _f8("f8_train", "train", "bf16", 4096, 2048, 8192, False),
        # one new token of four sequences in a text model with three axes, channel i turned with i + D/2
        _axes("axes_token", "forward", "bf16", 4, 1, 16, 8, 256, (64, 96, 96), "halves", "joint", "text", True),
        # images of odd sizes packed in one sequence, 32 bits, part of each head rotated
        _axes("axes_ragged_f32", "forward", "f32", 1, 5003, 6, 3, 80, (16, 24, 24), "adjacent", "split", "packed", False),
        # queries and keys out of one projection over a 17x68x60 grid of a video
        _axes("axes_grid", "forward", "bf16", 1, 69360, 32, 8, 128, (32, 48, 48), "adjacent", "split", "grid", True),
        # the diffusion transformer's frequencies over its whole width, fractional positions, with the gradient
        _axes("axes_wide_train", "train", "bf16", 2, 18360, 1, 1, 4096, (1364, 1364, 1364), "adjacent", "wide",
              "fraction", False),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """Widths: most are multiples of 64 or 8, some are any number."""
    step = rng.choice([64, 64, 8, 1])
    return max(step, _spread(rng, lo, hi) // step * step)


def _draw_once(rng):
    op = rng.choice(["ln", "f8", "axes"])
    if op == "ln":
        kind = rng.choice(["before", "after", "before_backward", "after_backward"])
        dtype = rng.choice(["bf16", "f32"])
        return _ln("", kind, dtype, rng.randint(1, 5), _spread(rng, 1, 35000), _width(rng, 64, 8192),
                   "f32" if dtype == "f32" else rng.choice(["bf16", "f32"]), rng.random() < 0.6,
                   kind.startswith("after") and rng.random() < 0.6, rng.random() < 0.7)
    if op == "f8":
        kind = rng.choice(["forward", "forward", "train"])
        return _f8("", kind, rng.choice(["bf16", "bf16", "f32"]), _spread(rng, 1, 8192), _width(rng, 128, 10240),
                   _width(rng, 128, 10240), kind == "forward" and rng.random() < 0.5)
    kind, dtype = rng.choice(["forward", "train"]), rng.choice(["bf16", "bf16", "f32"])
    if rng.random() < 0.2:
        width = 6 * rng.randint(40, 680)
        return _axes("", kind, dtype, rng.randint(1, 3), _spread(rng, 1, 20000), 1, 1, width + rng.choice([0, 2, 4]),
                     (width // 3,) * 3, "adjacent", "wide", "fraction", rng.random() < 0.5)
    # widths of the axes: even, most of them multiples of 16 together
    step = rng.choice([8, 8, 2])
    widths = tuple(step * rng.randint(1, 64 // step) for _ in range(3))
    return _axes("", kind, dtype, rng.randint(1, 4), _spread(rng, 1, 35000), rng.choice([1, 4, 6, 16, 24, 32]),
                 rng.choice([1, 2, 3, 8]), sum(widths) + rng.choice([0, 0, 16, 2]), widths,
                 rng.choice(["adjacent", "halves"]), rng.choice(["split", "joint"]),
                 rng.choice(["text", "packed", "grid"]), rng.random() < 0.5)


def draw(rng):
    while True:
        c = _draw_once(rng)
        w = work(c)
        if w["bytes"] <= 1.1e9 and w["flops"] <= 6.5e11:
            del c["name"]
            return c


# ---- inputs ------------------------------------------------------------------------------------

def _frequencies(case):
    """Radians a unit of position, and the axis of each pair (255: a pair that is not rotated), on the host."""
    widths = (case["width_t"], case["width_h"], case["width_w"])
    if case["frequencies"] == "wide":
        # theta^(0 .. 1) pi/2, each for the three axes in turn, behind what the width leaves over
        n = widths[0] // 2
        grid = (10000.0 ** torch.linspace(0.0, 1.0, n, dtype=torch.float64) * (math.pi / 2)).float().double()
        left = case["head_dim"] // 2 - 3 * n
        axis = torch.tensor([255] * left + [0, 1, 2] * n, dtype=torch.uint8)
        return torch.cat([torch.zeros(left, dtype=torch.float64), grid.repeat_interleave(3)]), axis
    axis = torch.cat([torch.full((w // 2,), i, dtype=torch.uint8) for i, w in enumerate(widths)])
    if case["frequencies"] == "joint":
        return 10000.0 ** (-2.0 * torch.arange(sum(widths) // 2, dtype=torch.float64) / sum(widths)), axis
    return torch.cat([10000.0 ** (-2.0 * torch.arange(w // 2, dtype=torch.float64) / w) for w in widths]), axis


def _positions(case, g):
    """[3, batch, tokens]."""
    B, S = case["batch"], case["tokens"]
    at = torch.arange(S, device="cuda")
    if case["positions"] == "text":
        # the next token of sequences of any length: all axes alike
        start = torch.randint(0, 100000, (1, B, 1), generator=g, device="cuda")
        return (start + at).expand(3, B, S).contiguous()
    if case["positions"] == "packed":
        # images of 19x23 patches behind one another, each a step later than the last
        first = torch.randint(0, 1000, (B, 1), generator=g, device="cuda")
        t, rest = first + at // 437, (at % 437).expand(B, S)
        return torch.stack([t, t + rest // 23, t + rest % 23])
    t, h, w = at // 4080, at // 60 % 68, at % 60
    if case["positions"] == "grid":
        first = torch.randint(0, 64, (B, 1), generator=g, device="cuda")
        return torch.stack([first + t, h.expand(B, S), w.expand(B, S)])
    # shares of the extent, from -1 to 1, at each patch's middle
    first = torch.rand((B, 1), generator=g, device="cuda")
    t = (first + (t + 0.5) / 25.0) % 1.0
    return torch.stack([t, ((h + 0.5) / 68.0).expand(B, S), ((w + 0.5) / 60.0).expand(B, S)]) * 2.0 - 1.0


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["dtype"]]

    def normal(*shape, dtype=dt, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std + mean).to(dtype)

    if case["op"] == "ln":
        B, S, D = case["batch"], case["rows"], case["dim"]
        pt = _DT[case["params"]]
        t = {"weight": normal(D, dtype=pt, std=0.2, mean=1.0) if case["affine"] else None,
             "bias": normal(D, dtype=pt, std=0.2) if case["affine"] else None,
             "scale": normal(B, D, dtype=pt, std=0.3) if case["modulated"] else None,
             "shift": normal(B, D, dtype=pt, std=0.3) if case["modulated"] else None}
        if case["kind"].startswith("before"):
            t["x"] = normal(B, S, D, std=2.0, mean=0.5)
        else:
            t["y"] = normal(B, S, D)
            t["residual"] = normal(B, S, D, std=2.0, mean=0.5)
            t["gate"] = normal(B, D, dtype=pt, std=0.5) if case["gate"] else None
        if case["kind"].endswith("backward"):
            t["dn"] = normal(B, S, D)
            t["dr"] = normal(B, S, D)
            if not case["kind"].startswith("before"):
                # what the forward pass kept: r = residual + gate * y
                t["r"] = _ln_residual(t).to(dt)
                del t["residual"]
        return t
    if case["op"] == "f8":
        M, K, N = case["tokens"], case["dim"], case["out"]
        w = normal(N, K, std=1.0 / math.sqrt(K))
        # activations with a few loud channels, as the blocks' scales are for
        x = (normal(M, K, dtype=torch.float32) * torch.exp(normal(K, dtype=torch.float32))).to(dt)
        if case["kind"] == "train":
            return {"x": x, "w": w, "dy": normal(M, N, std=1e-3)}
        w8, w_scale = _weight_f8(w)
        return {"x": x, "w8": w8, "w_scale": w_scale,
                "bias": normal(N, dtype=torch.float32, std=0.1) if case["bias"] else None}
    B, S, Hq, Hk, D = (case[k] for k in ("batch", "tokens", "q_heads", "k_heads", "head_dim"))
    if case["fused"]:
        # views of one projection of queries, keys and values
        qkv = normal(B, S, Hq + 2 * Hk, D)
        t = {"q": qkv[:, :, :Hq], "k": qkv[:, :, Hq:Hq + Hk]}
    else:
        t = {"q": normal(B, S, Hq, D), "k": normal(B, S, Hk, D)}
    t["positions"] = _positions(case, g)
    t["frequencies"], t["axis"] = (v.cuda() for v in _frequencies(case))
    if case["kind"] == "train":
        t["dq"], t["dk"] = normal(B, S, Hq, D), normal(B, S, Hk, D)
    return t


def prepare(case, seed):
    return {"case": case, "t": _inputs(case, seed)}


# ---- the plain form ----------------------------------------------------------------------------

def _f(t):
    return None if t is None else t.float()


def _ln_residual(t):
    y = _f(t["y"])
    if t["gate"] is not None:
        y = y * _f(t["gate"])[:, None, :]
    return _f(t["residual"]) + y


def _hat(x):
    x = x - x.mean(-1, keepdim=True)
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS)
    return x * rstd, rstd


def _ln_forward(x, t):
    n = _hat(x)[0]
    if t["weight"] is not None:
        n = n * _f(t["weight"]) + _f(t["bias"])
    if t["scale"] is not None:
        n = n * (1.0 + _f(t["scale"])[:, None, :]) + _f(t["shift"])[:, None, :]
    return n


def _ln_backward(x, t):
    """Every gradient of the norm at x; dr reaches x past it."""
    dn = _f(t["dn"])
    hat, rstd = _hat(x)
    out = {}
    per_hat, per_one = (dn * hat).sum(1), dn.sum(1)
    w = _f(t["weight"])
    mod = None if t["scale"] is None else 1.0 + _f(t["scale"])
    if w is not None:
        out["dweight"] = (per_hat if mod is None else per_hat * mod).sum(0)
        out["dbias"] = (per_one if mod is None else per_one * mod).sum(0)
    if mod is not None:
        out["dscale"] = per_hat if w is None else per_hat * w + per_one * _f(t["bias"])
        out["dshift"] = per_one
    v = dn
    if w is not None:
        v = v * w
    if mod is not None:
        v = v * mod[:, None, :]
    out["dx"] = _f(t["dr"]) + rstd * (v - v.mean(-1, keepdim=True) - hat * (v * hat).mean(-1, keepdim=True))
    return out


def _plain_ln(case, t):
    if case["kind"] == "before":
        out = {"n": _ln_forward(_f(t["x"]), t)}
    elif case["kind"] == "after":
        r = _ln_residual(t)
        out = {"r": r, "n": _ln_forward(r, t)}
    elif case["kind"] == "before_backward":
        out = _ln_backward(_f(t["x"]), t)
    else:
        out = _ln_backward(_f(t["r"]), t)
        dr = out.pop("dx")
        out["dresidual"] = out["dy"] = dr
        if t["gate"] is not None:
            out["dgate"] = (dr * _f(t["y"])).sum(1)
            out["dy"] = dr * _f(t["gate"])[:, None, :]
    dt, pt = _DT[case["dtype"]], _DT[case["params"]]
    return {k: v.to(dt if k in ("r", "n", "dx", "dy", "dresidual") else pt) for k, v in out.items()}


def _padded(x, rows, cols):
    return torch.nn.functional.pad(x, (0, -x.shape[1] % cols, 0, -x.shape[0] % rows))


def _to_f8(x, scale):
    """e4m3 of x / scale, both in 32 bits; zeros where the scale is 0."""
    return torch.where(scale > 0, x / scale, torch.zeros_like(x)).clamp(-_TOP, _TOP).to(_F8)


def _rows_f8(x):
    """x in e4m3 and a scale for each 128 numbers of a row."""
    x = _f(x)
    K = x.shape[1]
    blocks = _padded(x, 1, _BLOCK).unflatten(1, (-1, _BLOCK))
    scale = blocks.abs().amax(2)
    scale = scale / torch.full_like(scale, _TOP)
    return _to_f8(blocks, scale[:, :, None]).flatten(1)[:, :K].contiguous(), scale


def _weight_f8(w):
    """w in e4m3 and a scale for each 128 x 128 block."""
    w = _f(w)
    N, K = w.shape
    blocks = _padded(w, _BLOCK, _BLOCK).unflatten(1, (-1, _BLOCK)).unflatten(0, (-1, _BLOCK))
    scale = blocks.abs().amax((1, 3))
    scale = scale / torch.full_like(scale, _TOP)
    q = _to_f8(blocks, scale[:, None, :, None]).flatten(2).flatten(0, 1)
    return q[:N, :K].contiguous(), scale


def _spread_rows(q, scale):
    return q.float() * scale.repeat_interleave(_BLOCK, 1)[:, :q.shape[1]]


def _spread_blocks(q, scale):
    full = scale.repeat_interleave(_BLOCK, 0).repeat_interleave(_BLOCK, 1)
    return q.float() * full[:q.shape[0], :q.shape[1]]


def _plain_f8(case, t):
    dt = _DT[case["dtype"]]
    q, scale = _rows_f8(t["x"])
    x = _spread_rows(q, scale)
    if case["kind"] == "forward":
        y = x @ _spread_blocks(t["w8"], t["w_scale"]).t()
        if t["bias"] is not None:
            y = y + t["bias"]
        return {"y": y.to(dt), "q": q, "scale": scale}
    w8, w_scale = _weight_f8(t["w"])
    w = _spread_blocks(w8, w_scale)
    dy = _spread_rows(*_rows_f8(t["dy"]))
    # the weights' gradient sums over tokens: blocks of 128 tokens of each column
    x_turned = _spread_rows(*_rows_f8(t["x"].t().contiguous()))
    dy_turned = _spread_rows(*_rows_f8(t["dy"].t().contiguous()))
    return {"y": (x @ w.t()).to(dt), "dx": (dy @ w).to(dt), "dw": (dy_turned @ x_turned.t()).to(dt)}


def _turned(x, cos, sin, pairing):
    """x [batch, tokens, heads, head_dim] with its pairs turned; cos and sin [batch, tokens, 1, pairs]."""
    x = _f(x)
    P = cos.shape[-1]
    if pairing == "halves":
        e, o = x[..., :P], x[..., P:2 * P]
        turned = torch.cat([e * cos - o * sin, e * sin + o * cos], -1)
    else:
        e, o = x[..., 0:2 * P:2], x[..., 1:2 * P:2]
        turned = torch.stack([e * cos - o * sin, e * sin + o * cos], -1).flatten(-2)
    return torch.cat([turned, x[..., 2 * P:]], -1)


def _plain_axes(case, t):
    # angles in 64 bits: a position of 100000 leaves 32 bits 0.004 of a radian
    rotated = t["axis"] < 3
    at = t["positions"].double()[torch.where(rotated, t["axis"], 0).long()].permute(1, 2, 0)
    angle = torch.where(rotated, at * t["frequencies"], torch.zeros_like(at))[:, :, None, :]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    dt, pairing = _DT[case["dtype"]], case["pairing"]
    out = {"q": _turned(t["q"], cos, sin, pairing).to(dt), "k": _turned(t["k"], cos, sin, pairing).to(dt)}
    if case["kind"] == "train":
        out["dq"] = _turned(t["dq"], cos, -sin, pairing).to(dt)
        out["dk"] = _turned(t["dk"], cos, -sin, pairing).to(dt)
    return out


# ---- the framework's operators ------------------------------------------------------------------

def _own(case, t):
    import rope_ltx3drope_amd as rla

    if case["op"] == "ln":
        vec = (t["weight"], t["bias"], t["scale"], t["shift"])
        kw = dict(zip(("weight", "bias", "scale", "shift"), vec))
        if case["kind"] == "before":
            return {"n": rla.layer_norm_before(t["x"], *vec, eps=_EPS)}
        if case["kind"] == "after":
            r, n = rla.layer_norm_after(t["y"], t["residual"], t["gate"], eps=_EPS, **kw)
            return {"r": r, "n": n}
        if case["kind"] == "before_backward":
            g = rla.layer_norm_before_backward(t["dn"], t["x"], *vec, dresidual=t["dr"], eps=_EPS)
        else:
            g = rla.layer_norm_after_backward(t["dr"], t["dn"], t["y"], t["r"], t["gate"], eps=_EPS, **kw)
        return {k: v for k, v in g._asdict().items() if v is not None}
    if case["op"] == "f8":
        dt = _DT[case["dtype"]]
        if case["kind"] == "forward":
            q, scale = rla.f8_quantize(t["x"])
            y = rla.f8_matmul(q, scale, t["w8"], t["w_scale"], bias=t["bias"], dtype=dt)
            return {"y": y, "q": q, "scale": scale}
        x, xs, x_turned, xs_turned = rla.f8_quantize(t["x"], turned=True)
        w, ws, w_turned, ws_turned = rla.f8_quantize_weight(t["w"], turned=True)
        y = rla.f8_matmul(x, xs, w, ws, dtype=dt)
        dy, dys, dy_turned, dys_turned = rla.f8_quantize(t["dy"], turned=True)
        dx = rla.f8_matmul(dy, dys, w_turned, ws_turned, dtype=dt)
        dw = rla.f8_matmul(dy_turned, dys_turned, x_turned, xs_turned, dtype=dt)
        return {"y": y, "dx": dx, "dw": dw}
    how = (t["positions"], t["frequencies"], t["axis"])
    q, k = rla.axes_apply_qk(t["q"], t["k"], *how, pairing=case["pairing"])
    if case["kind"] == "forward":
        return {"q": q, "k": k}
    dq, dk = rla.axes_apply_qk_backward(t["dq"], t["dk"], *how, pairing=case["pairing"])
    return {"q": q, "k": k, "dq": dq, "dk": dk}


def run(state):
    case, t = state["case"], state["t"]
    if own:
        return _own(case, t)
    return {"ln": _plain_ln, "f8": _plain_f8, "axes": _plain_axes}[case["op"]](case, t)


# ---- the work that a pass cannot do without -----------------------------------------------------

def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "ln":
        n = case["batch"] * case["rows"] * case["dim"]
        ps = 4 if case["params"] == "f32" else 2
        vec = (2 * case["affine"] * case["dim"] + (case["gate"] + 2 * case["modulated"]) * case["batch"] * case["dim"]) * ps
        rows, flops = {"before": (2, 9), "after": (4, 11), "before_backward": (4, 20),
                       "after_backward": (5 + case["gate"], 24)}[case["kind"]]
        return {"bytes": rows * n * es + vec * (1 + case["kind"].endswith("backward")), "flops": flops * n}
    if case["op"] == "f8":
        M, K, N = case["tokens"], case["dim"], case["out"]
        if case["kind"] == "train":
            return {"bytes": 2 * (M * K + N * K + M * N) * es, "flops": 6 * M * K * N}
        kb, nb = -(-K // _BLOCK), -(-N // _BLOCK)
        return {"bytes": M * K * es + M * K + 4 * M * kb + N * K + 4 * nb * kb + 4 * N * case["bias"] + M * N * es,
                "flops": 2 * M * K * N}
    S, times = case["batch"] * case["tokens"], 2 if case["kind"] == "train" else 1
    n = S * (case["q_heads"] + case["k_heads"]) * case["head_dim"] * times
    at = 3 * S * (4 if case["positions"] == "fraction" else 8)
    return {"bytes": 2 * n * es + at * times + 9 * (case["head_dim"] // 2), "flops": 3 * n}


# ---- the definitions in 64 bits ------------------------------------------------------------------

def exact(case, seed):
    t = _inputs(case, seed)
    if case["op"] == "ln":
        return _exact_ln(case, {k: None if v is None else v.double() for k, v in t.items()})
    if case["op"] == "f8":
        return _exact_f8(case, t)
    return _exact_axes(case, t)


def _exact_ln(case, t):
    D = case["dim"]
    after = case["kind"].startswith("after")
    one = torch.ones((), dtype=torch.float64, device="cuda")
    w = one if t["weight"] is None else t["weight"]
    bias = 0.0 * one if t["bias"] is None else t["bias"]
    mod = one if t["scale"] is None else (t["scale"] + 1.0).unsqueeze(1)
    gate = one if not after or t["gate"] is None else t["gate"].unsqueeze(1)
    out = {}
    if case["kind"].endswith("backward"):
        r = t["r"] if after else t["x"]
    else:
        r = t["residual"].addcmul(gate, t["y"]) if after else t["x"]
    var, mean = torch.var_mean(r, dim=-1, correction=0, keepdim=True)
    inv = 1.0 / torch.sqrt(var + _EPS)
    hat = (r - mean).mul_(inv)
    if not case["kind"].endswith("backward"):
        if after:
            out["r"] = r
        n = hat.mul_(w).add_(bias).mul_(mod)
        out["n"] = n if t["shift"] is None else n.add_(t["shift"].unsqueeze(1))
        return out
    dn = t["dn"]
    if t["weight"] is not None:
        out["dweight"] = (dn * mod * hat).sum((0, 1))
        out["dbias"] = (dn * mod).sum((0, 1))
    if t["scale"] is not None:
        out["dscale"] = (dn * (hat * w + bias)).sum(1)
        out["dshift"] = dn.sum(1)
    v = dn * w * mod
    v = v - v.sum(-1, keepdim=True) / D - hat * ((v * hat).sum(-1, keepdim=True) / D)
    total = v.mul_(inv).add_(t["dr"])
    if not after:
        out["dx"] = total
        return out
    out["dresidual"] = total
    out["dy"] = total * gate
    if t["gate"] is not None:
        out["dgate"] = (total * t["y"]).sum(1)
    return out


def _exact_blocks(x, rows):
    """(e4m3 values in 64 bits, one scale for each `rows` x 128) of x: the definition's scale, max / 448, and
    quotient, x / scale, are 32-bit numbers, each rounded."""
    R, C = x.shape
    grid = torch.zeros((-(-R // rows) * rows, -(-C // _BLOCK) * _BLOCK), dtype=torch.float64, device=x.device)
    grid[:R, :C] = x
    grid = grid.view(grid.shape[0] // rows, rows, -1, _BLOCK)
    scale = grid.abs().amax(dim=3).amax(dim=1).div(_TOP).float().double()
    v = (grid / scale.clamp_min(1e-300)[:, None, :, None]).float().double()
    # four significant bits, from 2^-6 down in steps of 2^-9; ties to even
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3.0)
    # log2 next to a power of two: the step of the power that v really is above
    step = torch.where(v.abs() >= step * 16.0, step * 2.0, step)
    step = torch.where((v.abs() < step * 8.0) & (step > 2.0 ** -9), step / 2.0, step)
    v = torch.round(v / step) * step
    return v.view(v.shape[0] * rows, -1)[:R, :C], scale


def _exact_value(x, rows):
    v, scale = _exact_blocks(x, rows)
    full = torch.repeat_interleave(torch.repeat_interleave(scale, rows, dim=0), _BLOCK, dim=1)
    return v * full[:v.shape[0], :v.shape[1]]


def _exact_f8(case, t):
    x = t["x"].double()
    if case["kind"] == "forward":
        w = t["w8"].double()
        w.mul_(torch.kron(t["w_scale"].double(), torch.ones((_BLOCK, _BLOCK), dtype=torch.float64, device="cuda"))
               [:w.shape[0], :w.shape[1]])
        q, scale = _exact_blocks(x, 1)
        y = torch.mm(_exact_value(x, 1), w.transpose(0, 1).contiguous())
        if t["bias"] is not None:
            y.add_(t["bias"].unsqueeze(0))
        return {"y": y, "q": q, "scale": scale}
    w, dy = t["w"].double(), t["dy"].double()
    w = _exact_value(w, _BLOCK)
    y = torch.mm(_exact_value(x, 1), w.transpose(0, 1).contiguous())
    dx = torch.mm(_exact_value(dy, 1), w)
    columns = _exact_value(x.transpose(0, 1).contiguous(), 1)
    dw = torch.mm(_exact_value(dy.transpose(0, 1).contiguous(), 1), columns.transpose(0, 1).contiguous())
    return {"y": y, "dx": dx, "dw": dw}


def _exact_axes(case, t):
    P = t["axis"].numel()
    angle = torch.zeros((case["batch"], case["tokens"], P), dtype=torch.float64, device="cuda")
    for a in range(3):
        angle += t["positions"][a].double().unsqueeze(-1) * (t["frequencies"] * (t["axis"] == a))
    turn = torch.polar(torch.ones_like(angle), angle).unsqueeze(2)

    def rotate(x, by):
        x = x.double()
        first = x[..., :2 * P]
        if case["pairing"] == "halves":
            z = torch.complex(first[..., :P], first[..., P:]) * by
            first = torch.cat([z.real, z.imag], -1)
        else:
            z = torch.view_as_complex(first.reshape(*first.shape[:-1], P, 2).contiguous()) * by
            first = torch.view_as_real(z).reshape(first.shape)
        return torch.cat([first, x[..., 2 * P:]], -1)

    out = {"q": rotate(t["q"], turn), "k": rotate(t["k"], turn)}
    if case["kind"] == "train":
        out["dq"], out["dk"] = rotate(t["dq"], turn.conj()), rotate(t["dk"], turn.conj())
    return out
