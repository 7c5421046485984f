"""Rotary positions with several axes from their formula, in float64 on the CPU (torch tensors)."""
from __future__ import annotations

import torch


def frequencies(widths, base, joint):
    """(frequencies, axis) of a head cut into one chunk of channels an axis, as lists."""
    total, f, axis = sum(widths), [], []
    for a, w in enumerate(widths):
        for i in range(w // 2):
            f.append(base ** (-2.0 * (len(f) if joint else i) / (total if joint else w)))
            axis.append(a)
    return f, axis


def angles(positions, freq, axis):
    """[batch, tokens, pairs] radians for positions [axes, batch, tokens]; zero where the axis does not exist."""
    out = torch.zeros(*positions.shape[1:], freq.numel(), dtype=torch.float64)
    for i in range(freq.numel()):
        if int(axis[i]) < positions.shape[0]:
            out[..., i] = positions[int(axis[i])].double() * float(freq[i])
    return out


def rotate(x, angle, axes, axis, pairing, inverse=False):
    """x [batch, tokens, heads, head_dim] in float64 with its pairs turned."""
    out = x.clone()
    P = axis.numel()
    for i in range(P):
        if int(axis[i]) >= axes:
            continue
        a, b = (2 * i, 2 * i + 1) if pairing == "adjacent" else (i, i + P)
        t = (-angle[..., i] if inverse else angle[..., i])[..., None]
        e, o = x[..., a], x[..., b]
        out[..., a] = e * torch.cos(t) - o * torch.sin(t)
        out[..., b] = e * torch.sin(t) + o * torch.cos(t)
    return out
