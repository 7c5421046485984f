"""The linear layer in 8-bit floating point from its definition, on the CPU (torch tensors).

The quantiser's scale and quotient are fp32 numbers, each rounded once, and are formed so here; products
and sums are float64.
"""
from __future__ import annotations

import torch

F8 = torch.float8_e4m3fn
TOP = torch.tensor(448.0)


def quantize(x, block_rows):
    """(e4m3 values like x, scales) with one scale for each block_rows x 128 numbers of x [rows, dim]."""
    x = x.float()
    R, C = x.shape
    down, across = -(-R // block_rows), -(-C // 128)
    q, scale = torch.zeros(R, C), torch.zeros(down, across)
    for j in range(across):
        for i in range(down):
            b = x[i * block_rows:(i + 1) * block_rows, j * 128:(j + 1) * 128]
            top = b.abs().max()
            s = torch.where(torch.isnan(b).any(), torch.tensor(float("nan")), top) / TOP
            scale[i, j] = s
            if bool(torch.isfinite(s)) and float(s) > 0:
                q[i * block_rows:(i + 1) * block_rows, j * 128:(j + 1) * 128] = (b / s).clamp(-448.0, 448.0)
    return q.to(F8), scale


def quantize_rows(x):
    """The same for block_rows = 1, all blocks at once."""
    x = x.float()
    R, C = x.shape
    b = torch.nn.functional.pad(x, (0, -C % 128)).view(R, -1, 128)
    s = b.abs().amax(2) / TOP  # amax hands a NaN on
    plain = (torch.isfinite(s) & (s > 0))[:, :, None]
    q = torch.where(plain, (b / s[:, :, None]).clamp(-448.0, 448.0), torch.zeros_like(b))
    return q.reshape(R, -1)[:, :C].to(F8), s


def spread(scale, rows, dim, block_rows):
    """A scale for every number."""
    s = scale.double().repeat_interleave(block_rows, 0).repeat_interleave(128, 1)
    return s[:rows, :dim]


def matmul(a, a_scale, b, b_scale, bias):
    """y, and the sum of the absolute values of its terms."""
    M, K = a.shape
    N = b.shape[0]
    rows = 1 if N == 1 or b_scale.shape[0] == N else 128
    x = a.double() * spread(a_scale, M, K, 1)
    w = b.double() * spread(b_scale, N, K, rows)
    y, mag = x @ w.t(), x.abs() @ w.abs().t()
    if bias is not None:
        y, mag = y + bias.double(), mag + bias.double().abs()
    return y, mag
