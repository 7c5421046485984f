"""The 8-bit floating point product at the ends of its documented sizes: sums of almost 2^21 numbers, rows almost 2^22
bytes and scales almost 2^20 numbers apart.  Sums of -1, 0 and 1 with scales of powers of two are exact in fp32."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

rla = pytest.importorskip("rope_ltx3drope_amd")

DEV = "cuda:0"
F8 = torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def fresh():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def ones(gen, *shape):
    """-1, 0 and 1 as e4m3, made from bytes: 0xb8, 0x00, 0x38."""
    v = torch.randint(0, 3, shape, generator=gen, device=DEV, dtype=torch.uint8)
    return torch.tensor([0x38, 0x00, 0xb8], dtype=torch.uint8, device=DEV)[v.int()].view(F8)


@pytest.mark.parametrize("K", [(1 << 21) - 1, (1 << 21) - 16])
@pytest.mark.parametrize("M,N", [(1, 40), (16, 40), (17, 40), (200, 130), (256, 520)])
def test_the_longest_sums(M, N, K):
    gen = torch.Generator(device=DEV).manual_seed(M)
    a, b = ones(gen, M, K), ones(gen, N, K)
    blocks = -(-K // 128)
    sa = 2.0 ** torch.randint(-1, 2, (M, blocks), generator=gen, device=DEV).float()
    sb = torch.ones(-(-N // 128), blocks, device=DEV)
    want = torch.zeros(M, N, dtype=torch.float64, device=DEV)
    for lo in range(0, K, 1 << 19):
        hi = min(K, lo + (1 << 19))
        x = a[:, lo:hi].float() * sa[:, lo // 128:-(-hi // 128)].repeat_interleave(128, 1)[:, :hi - lo]
        want += x.double() @ b[:, lo:hi].double().t().contiguous()
    assert float(want.abs().max()) < 2.0 ** 22
    for dtype in (torch.float32, torch.bfloat16):
        assert torch.equal(rla.f8_matmul(a, sa, b, sb, dtype=dtype), want.to(dtype)), dtype


@pytest.mark.parametrize("b_rows", [False, True], ids=["blocks", "rows"])
@pytest.mark.parametrize("M,K,N", [(1, 400, 70), (60, 401, 300), (300, 528, 700), (2048, 528, 2050), (2048, 529, 2050)])
def test_rows_and_scales_furthest_apart(M, K, N, b_rows):
    gen = torch.Generator(device=DEV).manual_seed(K)
    pitch, row = (1 << 22) - 16, (1 << 20) - 1
    blocks, nb = -(-K // 128), N if b_rows else -(-N // 128)

    def rows(n):
        v = torch.empty(n * pitch, dtype=torch.uint8, device=DEV).view(n, pitch)[:, :K]
        v.copy_(ones(gen, n, K).view(torch.uint8))
        return v.view(F8)

    def scales(n):
        v = torch.empty(n * row, device=DEV).view(n, row)[:, :blocks]
        return v.copy_(2.0 ** torch.randint(-1, 2, (n, blocks), generator=gen, device=DEV).float())

    a, b, sa, sb = rows(M), rows(N), scales(M), scales(nb)
    packed = [t.contiguous() for t in (a, sa, b, sb)]
    full = lambda s, n: (s if s.shape[0] == n else s.repeat_interleave(128, 0)[:n]).repeat_interleave(128, 1)[:, :K].double()  # noqa: E731
    want = (packed[0].double() * full(packed[1], M)) @ (packed[2].double() * full(packed[3], N)).t().contiguous()
    for dtype in (torch.float32, torch.bfloat16):
        assert torch.equal(rla.f8_matmul(a, sa, b, sb, dtype=dtype), want.to(dtype)), dtype
