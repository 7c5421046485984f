"""The quantisers of the 8-bit floating point layer on rows of more than 2^30 numbers."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

rla = pytest.importorskip("rope_ltx3drope_amd")

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def fresh():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def same_bytes(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("f", [rla.f8_quantize, rla.f8_quantize_weight], ids=["rows", "blocks"])
def test_a_row_of_more_than_two_to_the_30_numbers(f, dtype):
    """A row's bytes from 2^32 on (fp32) are those of its own numbers: its ends and its middle quantised alone give
    the same bits."""
    dim = (1 << 30) + 1032
    gen = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(1, dim, generator=gen, device=DEV, dtype=dtype)
    q, s = f(x)
    for lo, hi in ((0, 4096), (1 << 29, (1 << 29) + 4096), ((1 << 30) - 1024, dim), (1 << 30, dim)):
        part, scale = f(x[:, lo:hi].contiguous())
        assert same_bytes(q[:, lo:hi], part), lo
        assert torch.equal(s[:, lo // 128:-(-hi // 128)], scale), lo
