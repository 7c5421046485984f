"""The layer norms on rows of one value, and on rows whose spread is a few steps of fp32, against 64 bits.

Bounds.  A row's mean is formed in 64 bits: of D <= 2^14 equal fp32 numbers the sum is exact, and the quotient is
that number, so that a row of one value is zeros exactly and its variance is 0: n is the norm's term alone and
dx = (v - mean(v)) / sqrt(eps), where mean(v) is a sum of at most K = 40 operations deep.  Otherwise the mean is off by
2^-52 of the largest value, which moves hat by that over the root of the variance; what is left is rounded twice
and the variance is a sum of squares, K operations deep, under a root.
"""
from __future__ import annotations

import pytest
import torch

from tests.block_tools import U, assert_within, d, half_step, randn, tiny

pytestmark = pytest.mark.gpu

rla = pytest.importorskip("rope_ltx3drope_amd")

DEV = "cuda:0"
K = 40
EPS = 1e-6
ROOT = float(torch.tensor(EPS).double() ** -0.5)
WIDTHS = [1, 2, 3, 8, 41, 47, 61, 64, 82, 100, 512, 777, 1000, 2053, 4096, 5003, 8191, 8193, 12345, 14200, 15761, 16384]
VALUES = [0.0, 1.0, 1000.1, -3.3e7, 1.0104576503474703e8, 1541722464756.978, -1.0322083622173111e13,
          3.3976242168633284e16, 7.697086548999672e18, -1e20, 1e30, 3e38, 1e-30, -7.3e-41]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dim", WIDTHS)
def test_rows_of_one_value_are_zeros(dim, dtype):
    g = torch.Generator().manual_seed(dim)
    x = torch.tensor(VALUES, dtype=dtype)[:, None].expand(-1, dim).contiguous()
    assert not bool(rla.layer_norm_before(x.to(DEV), eps=EPS).any())
    bias, shift = randn(g, dim, dtype=dtype), randn(g, 1, dim, dtype=dtype)
    n = rla.layer_norm_before(x.to(DEV)[None], torch.full((dim,), 3.0, dtype=dtype, device=DEV), bias.to(DEV),
                              shift=shift.to(DEV), eps=EPS)
    want = d(bias) + d(shift)
    assert_within(n, want.expand(n.shape), (half_step(dtype) + 2 * U) * want.abs().expand(n.shape) + tiny(dtype), "n")
    # after a block: r = residual + gate * y is one value too
    y, gate = torch.full_like(x, 2.0)[None], torch.full((1, dim), 0.5, dtype=dtype)
    r, n = rla.layer_norm_after(y.to(DEV), x.to(DEV)[None], gate.to(DEV), eps=EPS)
    assert not bool(n.any())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dim", WIDTHS)
def test_gradients_of_rows_of_one_value(dim, dtype):
    g = torch.Generator().manual_seed(dim)
    x = torch.tensor(VALUES, dtype=dtype)[:, None].expand(-1, dim).contiguous()
    dn, w = randn(g, *x.shape, dtype=dtype), randn(g, dim, std=0.2, mean=1.0, dtype=dtype)
    got = rla.layer_norm_before_backward(dn.to(DEV), x.to(DEV), w.to(DEV), eps=EPS)
    v = d(dn) * d(w)
    want = (v - v.mean(-1, keepdim=True)) * ROOT
    tol = ROOT * ((K + 4) * U * (v.abs().mean(-1, keepdim=True) + v.abs()) + 4 * U * v.abs())
    assert_within(got.dx, want, tol + half_step(dtype) * want.abs() + tiny(dtype), "dx")
    assert not bool(got.dweight.any())  # hat is zero


@pytest.mark.parametrize("dim", [2, 8, 100, 777, 2053, 4096, 8193, 14200, 16384])
@pytest.mark.parametrize("value", [1.5, 1e3, -3.3e7, 1e13, 1.2e17])
def test_rows_whose_spread_is_a_few_steps(value, dim):
    """All elements are one fp32 number but some that lie one to three steps of it beside."""
    g = torch.Generator().manual_seed(dim)
    step = torch.randint(0, 4, (6, dim), generator=g) * (torch.rand(6, dim, generator=g) < torch.tensor(
        [1.0, 0.5, 0.1, 0.01, 0.0, 0.0])[:, None])
    step[4, 0] = step[5, -1] = 1  # one element alone
    bits = torch.tensor(value, dtype=torch.float32).view(torch.int32)
    x = (bits + step.to(torch.int32)).view(torch.float32)
    eps = 1e-30
    got = rla.layer_norm_before(x.to(DEV), eps=eps)
    # less the common value, which changes neither the mean's distance nor the spread, 64 bits hold the row exactly
    c = d(x) - d(x[:, :1])
    c = c - c.mean(-1, keepdim=True)
    inv = ((c * c).mean(-1, keepdim=True) + float(torch.tensor(eps))) ** -0.5
    want = c * inv
    off = 2.0 ** -52 * abs(value) * inv
    assert_within(got, want, off + want.abs() * (off + (K + 8) * U) + tiny(torch.float32), "n")
