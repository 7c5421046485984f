"""The angles of the rotation with several axes on the GPU: unit vectors turned by them are their cosines and sines.

Bound: 9.4e-8 for the polynomials (tests/test_axes_math_host.py) and the angle's own error: position * turns is
rounded twice in 64 bits, 2^-52 of the angle.
"""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

rla = pytest.importorskip("rope_ltx3drope_amd")

DEV = "cuda:0"


@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
def test_unit_vectors(pairing):
    g = torch.Generator().manual_seed(1)
    tokens, pairs = 4096, 64
    positions = torch.randint(-1000000, 1000000, (1, tokens), generator=g)
    positions[0, :64] = torch.arange(64)
    freq = torch.rand(pairs, generator=g, dtype=torch.float64) * 10.0 ** torch.linspace(-6, 1, pairs, dtype=torch.float64)
    x = torch.zeros(tokens, 1, 2 * pairs)
    cos, sin = (slice(0, None, 2), slice(1, None, 2)) if pairing == "adjacent" else (slice(0, pairs), slice(pairs, None))
    x[..., cos] = 1.0
    args = (positions.to(DEV), freq.to(DEV), torch.zeros(pairs, dtype=torch.uint8, device=DEV))
    got = rla.axes_apply_qk(x.to(DEV), None, *args, pairing=pairing)[0].cpu().double()[:, 0]
    back = rla.axes_apply_qk_backward(x.to(DEV), None, *args, pairing=pairing)[0].cpu().double()[:, 0]
    angle = positions[0, :, None].double() * freq
    tol = 9.4e-8 + angle.abs() * 2.0 ** -51
    for turned, a in ((got, angle), (back, -angle)):
        assert bool(((turned[:, cos] - torch.cos(a)).abs() <= tol).all())
        assert bool(((turned[:, sin] - torch.sin(a)).abs() <= tol).all())
