"""Every kernel of the 8-bit floating point product's tiles on the GPU, at the sizes of tests/f8_tiles.py.

The inputs are small integers and the scales 1/2, 1 and 2, so that every sum is a multiple of 1/4 below 2^22, exact in
fp32 whatever its order (and in the 8-bit units, which keep 2^-13 of products up to 64): each output has one right
value, and one step of k left out, taken twice or scaled by another's scale changes whole tiles.  The products in
64 bits are formed on the GPU.
"""
from __future__ import annotations

import pytest
import torch

from tests import f8_tiles as ft
from tests.test_block_tiles_gpu import assert_same, integers

pytestmark = pytest.mark.gpu

rla = pytest.importorskip("rope_ltx3drope_amd")

DEV = "cuda:0"
F8 = torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def fresh():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def apart(t):
    """The same rows, as far apart as the next multiple of 128 bytes; NaN between them."""
    v = torch.full((t.shape[0], -(-t.shape[1] // 128) * 128), 0x7f, dtype=torch.uint8, device=DEV).view(F8)
    v.view(torch.uint8)[:, :t.shape[1]] = t.view(torch.uint8)
    return v[:, :t.shape[1]]


@pytest.mark.parametrize("b_rows", [False, True], ids=["blocks", "rows"])
@pytest.mark.parametrize("tokens,dim,out", ft.SIZES)
def test_tiles(tokens, dim, out, b_rows):
    gen = torch.Generator(device=DEV).manual_seed(tokens * out + dim)
    blocks = -(-dim // ft.STEP)
    a, b = (integers(gen, -8, 8, n, dim).float().to(F8) for n in (tokens, out))
    sa, sb = (2.0 ** integers(gen, -1, 1, n, blocks).float() for n in (tokens, out if b_rows else -(-out // 128)))
    bias = integers(gen, -9, 9, out).float()
    wide = lambda s: s.repeat_interleave(ft.STEP, 1)[:, :dim].double()  # noqa: E731
    w = b.double() * wide(sb if b_rows else sb.repeat_interleave(128, 0)[:out])
    want = (a.double() * wide(sa)) @ w.t().contiguous() + bias
    assert float(want.abs().max()) < 2.0 ** 22
    turned = lambda s: s.t().contiguous().t()  # noqa: E731
    for layout, operands in (("packed", (a, sa, b, sb)), ("apart", (apart(a), turned(sa), apart(b), turned(sb)))):
        for dtype in (torch.float32, torch.bfloat16):
            y = rla.f8_matmul(*operands, bias=bias, dtype=dtype)
            assert_same(y, want.to(dtype), f"{layout} {dtype}")
