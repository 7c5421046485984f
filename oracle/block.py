"""The transformer-block operators from their formulas, in float64 on the CPU (torch tensors).

Every function takes and returns float64 and forms each gradient from its formula, with no
automatic differentiation; tests check the gradients against central differences.  The `bound`
functions give, next to each value, the sum of the absolute values of the terms that it is made
of: what a relative error of each term can amount to in the result.
"""
from __future__ import annotations

import math

import torch


def rstd(v, eps):
    return 1.0 / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)


def _rowwise(v):
    """A per-sample vector [batch, dim] against rows [batch, rows, dim]."""
    return v[:, None, :]


def norm_factor(weight, scale, offset, like):
    f = torch.ones_like(like)
    if weight is not None:
        f = f * (weight + offset)
    if scale is not None:
        f = f * (1.0 + _rowwise(scale))
    return f


def norm_before(x, weight, scale, shift, eps, offset):
    n = x * rstd(x, eps) * norm_factor(weight, scale, offset, x)
    return n if shift is None else n + _rowwise(shift)


def branch_factor(weight, gate, offset, like):
    f = torch.ones_like(like)
    if weight is not None:
        f = f * (weight + offset)
    if gate is not None:
        f = f * _rowwise(gate)
    return f


def norm_after(y, residual, weight, gate, post_norm, residual_scale, eps, offset):
    hat = y * rstd(y, eps) if post_norm else y
    return residual_scale * residual + hat * branch_factor(weight, gate, offset, y)


def _through_norm(v, hat, inv):
    """The gradient of x where hat = x * inv and v is that of hat."""
    return inv * (v - hat * (v * hat).mean(-1, keepdim=True))


def norm_before_backward(dn, x, weight, scale, dresidual, eps, offset):
    """dx, dweight, dscale, dshift (the last three whether or not the vector is there)."""
    inv = rstd(x, eps)
    hat = x * inv
    dx = _through_norm(dn * norm_factor(weight, scale, offset, x), hat, inv)
    if dresidual is not None:
        dx = dx + dresidual
    p1, p2 = (dn * hat).sum(1), dn.sum(1)
    w = torch.ones_like(p1) if weight is None else (weight + offset).expand_as(p1)
    s = torch.ones_like(p1) if scale is None else 1.0 + scale
    return dx, (s * p1).sum(0), w * p1, p2


def norm_after_backward(dR, y, weight, gate, post_norm, residual_scale, eps, offset):
    """dy, dresidual, dweight, dgate for the gradient dR of r."""
    inv = rstd(y, eps) if post_norm else torch.ones_like(y[..., :1])
    hat = y * inv
    q = dR * branch_factor(weight, gate, offset, y)
    dy = _through_norm(q, hat, inv) if post_norm else q
    p3 = (dR * hat).sum(1)
    w = torch.ones_like(p3) if weight is None else (weight + offset).expand_as(p3)
    g = torch.ones_like(p3) if gate is None else gate
    return dy, residual_scale * dR, (g * p3).sum(0), w * p3


def act(g, kind):
    if kind == "silu":
        return g / (1.0 + torch.exp(-g))
    if kind == "gelu":
        return 0.5 * g * (1.0 + torch.erf(g / math.sqrt(2.0)))
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)))


def act_slope(g, kind):
    if kind == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return s + g * s * (1.0 - s)
    if kind == "gelu":
        return 0.5 * (1.0 + torch.erf(g / math.sqrt(2.0))) + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    c = math.sqrt(2.0 / math.pi)
    th = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * (1.0 + th) + 0.5 * g * (1.0 - th * th) * c * (1.0 + 3 * 0.044715 * g * g)


def gated_ffn(x, w_gate, w_up, kind):
    """h, g, u."""
    g, u = x @ w_gate.T, x @ w_up.T
    return act(g, kind) * u, g, u


def gated_ffn_backward(dh, x, w_gate, w_up, g, u, kind):
    """dx, dw_gate, dw_up from the saved projections g and u."""
    dg, du = dh * u * act_slope(g, kind), dh * act(g, kind)
    return dg @ w_gate + du @ w_up, dg.T @ x, du.T @ x


def q8_quantize(x):
    """q and scale of float32 rows (numpy arithmetic in float32, each step rounded once)."""
    import numpy as np

    x = x.float().numpy()
    top = np.abs(x).max(axis=-1) if x.shape[-1] else np.zeros(x.shape[:-1], np.float32)
    scale = (top * (np.float32(1.0) / np.float32(127.0))).astype(np.float32)
    plain = np.isfinite(scale) & (scale > 0)
    safe = np.where(plain, scale, np.float32(1.0))[..., None]
    with np.errstate(invalid="ignore"):
        q = np.where(plain[..., None], np.rint((x / safe).astype(np.float32)), np.float32(0.0))
    return torch.from_numpy(np.clip(q, -127, 127).astype(np.int8)), torch.from_numpy(scale)


def q8_matmul(a, a_scale, b, b_scale, bias):
    """The product in float64 (integer sums below 2^53 are exact)."""
    y = (a.double() @ b.double().T) * a_scale.double()[:, None] * b_scale.double()
    return y if bias is None else y + bias.double()
