"""Helpers of the transformer-block operators' tests: seeded inputs and error bounds.

Bounds are built from the arithmetic.  u = 2^-24 is half a step of fp32, relative to the value; a
result is rounded once to its type (half a step, finfo.eps / 2).  A quantity that an operator forms
by k fp32 operations from terms t_i is off by at most about k * u * sum |t_i|.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half a step below the smallest normal number: results there are not relative any more."""
    return torch.finfo(dtype).tiny * torch.finfo(dtype).eps


def randn(gen, *shape, std=1.0, mean=0.0, dtype=torch.float32):
    return (torch.randn(shape, generator=gen, dtype=torch.float32) * std + mean).to(dtype)


def d(t):
    return None if t is None else t.detach().cpu().double()


def assert_within(got, want, tol, what):
    """|got - want| <= tol everywhere (all float64 on the CPU); NaN where want is NaN only."""
    got, want = d(got), d(want)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    nan_w, nan_g = torch.isnan(want), torch.isnan(got)
    assert torch.equal(nan_w, nan_g), f"{what}: NaN at other places: {int((nan_w != nan_g).sum())}"
    err = torch.where(nan_w, torch.zeros_like(want), (got - want).abs())
    bad = err > tol
    if bool(bad.any()):
        i = int(torch.argmax((err / tol.clamp_min(1e-300) if torch.is_tensor(tol) else err / tol).reshape(-1)))
        t = float(tol.expand_as(want).reshape(-1)[i]) if torch.is_tensor(tol) else tol
        raise AssertionError(f"{what}: {int(bad.sum())} of {want.numel()} outside the bound; worst got "
                             f"{float(got.reshape(-1)[i])} want {float(want.reshape(-1)[i])} tolerance {t}")
