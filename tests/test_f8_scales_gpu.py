"""The 8-bit floating point product with scales whose product is at the ends of fp32's normal range and beyond them, as
its documentation says: exact within, off by at most a block's sum times 2^-150 below, infinite or NaN above.

The sizes take each kind of kernel: few tokens, tiles by either way of the operands, walking and split ones.
"""
from __future__ import annotations

import pytest
import torch

from tests.block_tools import U, assert_within, half_step

pytestmark = pytest.mark.gpu

rla = pytest.importorskip("rope_ltx3drope_amd")

DEV = "cuda:0"
F8 = torch.float8_e4m3fn
SIZES = [(1, 400, 70), (9, 1001, 130), (40, 512, 70), (300, 1001, 200), (100, 8192, 64), (1024, 1040, 2050),
         (2048, 528, 4100)]
TYPES = [torch.float32, torch.bfloat16]


def blocks_of(dim):
    return -(-dim // 128)


def spread(s, rows, dim):
    """A scale for every number of [rows, dim] from [rows, blocks] or one row for 128."""
    if s.shape[0] != rows:
        s = s.repeat_interleave(128, 0)[:rows]
    return s.double().repeat_interleave(128, 1)[:, :dim]


def matmul(a, b):
    return a @ b.t().contiguous()


@pytest.mark.parametrize("b_rows", [False, True], ids=["blocks", "rows"])
@pytest.mark.parametrize("M,K,N", SIZES)
def test_exact_to_the_ends_of_the_normal_range(M, K, N, b_rows):
    gen = torch.Generator(device=DEV).manual_seed(M)
    nb = N if b_rows else -(-N // 128)
    a, b = (torch.randint(-8, 9, (n, K), generator=gen, device=DEV).float().to(F8) for n in (M, N))
    # every product of scales is 2^-126, its parts as far apart as 2^-120 and 2^-6
    up = torch.randint(-6, 120, (1, blocks_of(K)), generator=gen, device=DEV).double()
    sa, sb = (2.0 ** (-126 + up)).float().expand(M, -1), (2.0 ** -up).float().expand(nb, -1)
    want = matmul(a.double(), b.double()) * 2.0 ** -126
    for dtype in TYPES:
        y = rla.f8_matmul(a, sa, b, sb, dtype=dtype)
        assert torch.equal(y.double() * 2.0 ** 126, (want * 2.0 ** 126).to(dtype).double())
    # and 2^127 of sums of -1, 0 and 1
    a = torch.zeros(M, K, device=DEV)
    at = torch.randint(0, K, (M,), generator=gen, device=DEV)
    a[torch.arange(M, device=DEV), at] = 1.0
    b = torch.randint(-1, 2, (N, K), generator=gen, device=DEV).float()
    up = up.abs()  # scales are finite themselves
    sa, sb = (2.0 ** (127 - up)).float().expand(M, -1), (2.0 ** up).float().expand(nb, -1)
    want = b.t()[at] * 2.0 ** 127
    for dtype in TYPES:
        y = rla.f8_matmul(a.to(F8), sa, b.to(F8), sb, dtype=dtype)
        assert torch.equal(y.float(), want)


@pytest.mark.parametrize("b_rows", [False, True], ids=["blocks", "rows"])
@pytest.mark.parametrize("M,K,N", SIZES)
def test_products_of_scales_below_the_normal_range(M, K, N, b_rows):
    """Scales of 2^-76 to 2^-62 multiply to 2^-152 to 2^-124."""
    gen = torch.Generator(device=DEV).manual_seed(K)
    nb = N if b_rows else -(-N // 128)
    a, b = ((torch.randn(n, K, generator=gen, device=DEV) * 40).clamp(-448, 448).to(F8) for n in (M, N))
    rand = lambda *s: torch.rand(s, generator=gen, device=DEV, dtype=torch.float64)  # noqa: E731
    sa, sb = ((2.0 ** (-76 + 14 * rand(n, blocks_of(K)))).float() for n in (M, nb))
    x, w = a.double() * spread(sa, M, K), b.double() * spread(sb, N, K)
    want, mag = matmul(x, w), matmul(x.abs(), w.abs())
    sums = matmul(a.double().abs(), b.double().abs())
    for dtype in TYPES:
        y = rla.f8_matmul(a, sa, b, sb, dtype=dtype)
        # 2^-150 for each unit of a block's sum and for each addition that ends below the normal range, beside the
        # roundings of any sum (and what the 8-bit units leave of 8 neighbours)
        tol = sums * 2.0 ** -150 + (blocks_of(K) + 17) * 2.0 ** -150 + (2 * 128 + 4 + blocks_of(K) + 17) * U * mag
        if M > 16 and dtype is torch.bfloat16:
            largest = lambda t, s: torch.nn.functional.pad(t.double().abs() * spread(s, *t.shape), (0, -K % 8)).view(  # noqa: E731
                t.shape[0], -1, 8).amax(2)
            tol = tol + 7 * 2.0 ** -13 * matmul(largest(a, sa), largest(b, sb))
        # results below bf16's (and fp32's) normal range are off by half a step of that, 2^-134 (2^-150)
        step = 2.0 ** -134 if dtype is torch.bfloat16 else 2.0 ** -150
        assert_within(y, want.cpu(), (tol + half_step(dtype) * (want.abs() + tol) + step).cpu(), f"{dtype}")


@pytest.mark.parametrize("M,K,N", SIZES)
def test_products_of_scales_above_the_range_stay_in_their_rows(M, K, N):
    gen = torch.Generator(device=DEV).manual_seed(N)
    a, b = (torch.randint(-8, 9, (n, K), generator=gen, device=DEV).float().to(F8) for n in (M, N))
    sa, sb = torch.ones(M, blocks_of(K), device=DEV), torch.full((N, blocks_of(K)), 2.0, device=DEV)
    want = matmul(a.double(), b.double()) * 2.0
    sa[0], sb[N // 2] = 2.0 ** 90, 2.0 ** 38
    for dtype in TYPES:
        y = rla.f8_matmul(a, sa, b, sb, dtype=dtype)
        assert not bool(torch.isfinite(y[0, N // 2]))
        keep = torch.arange(N, device=DEV) != N // 2
        assert torch.equal(y[1:][:, keep].double(), want[1:][:, keep].to(dtype).double())
        assert torch.equal(y[0, keep].double(), (want[0, keep] * 2.0 ** 90).to(dtype).double())
        assert torch.equal(y[1:, N // 2].double(), (want[1:, N // 2] * 2.0 ** 37).to(dtype).double())
