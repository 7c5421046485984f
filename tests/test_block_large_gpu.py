"""The transformer-block operators on tensors of more than 2^32 elements: rows at both ends and around
element 2^32 against calls on those rows alone, or against 64 bits."""
from __future__ import annotations

import pytest
import torch

import workloads
from tests.test_gated_ffn_gpu import check_backward, check_forward

pytestmark = pytest.mark.gpu

rla = pytest.importorskip("rope_ltx3drope_amd")

DEV = "cuda:0"
ROWS, DIM = 1_100_003, 4096  # 4.5 G elements
PLACES = [0, (1 << 32) // DIM - 20, ROWS - 40]


@pytest.fixture(autouse=True)
def free():
    torch.cuda.empty_cache()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def rows(t, at):
    return t[at:at + 40].contiguous()


def test_norm_and_quantiser():
    x = workloads.generate_bf16_bits((ROWS, DIM), 1, DEV)
    w = torch.linspace(0.5, 1.5, DIM, device=DEV)
    n = rla.norm_before(x, w)
    for at in PLACES:
        assert torch.equal(rows(n, at), rla.norm_before(rows(x, at), w))
    r, n2 = rla.norm_after(n, x, w, next_weight=w)
    for at in PLACES:
        a, b = rla.norm_after(rows(n, at), rows(x, at), w, next_weight=w)
        assert torch.equal(rows(r, at), a) and torch.equal(rows(n2, at), b)
    del n2
    g = rla.norm_after_backward(x, n, n, r, w, next_weight=w)
    for at in PLACES:
        s = rla.norm_after_backward(rows(x, at), rows(n, at), rows(n, at), rows(r, at), w, next_weight=w)
        assert torch.equal(rows(g.dy, at), s.dy) and torch.equal(rows(g.dresidual, at), s.dresidual)
    del g, r, n
    q, scale = rla.q8_quantize(x)
    for at in PLACES:
        a, b = rla.q8_quantize(rows(x, at))
        assert torch.equal(rows(q, at), a) and torch.equal(rows(scale, at), b)


def test_q8_matmul():
    gen = torch.Generator(device=DEV).manual_seed(2)
    a = torch.randint(-127, 128, (ROWS, 48), generator=gen, device=DEV, dtype=torch.int8)
    b = torch.randint(-127, 128, (DIM, 48), generator=gen, device=DEV, dtype=torch.int8)
    sa, sb = torch.rand(ROWS, generator=gen, device=DEV), torch.rand(DIM, generator=gen, device=DEV)
    y = rla.q8_matmul(a, sa, b, sb)
    for at in PLACES:
        assert torch.equal(rows(y, at), rla.q8_matmul(rows(a, at), rows(sa, at), b, sb))


def test_gated_ffn():
    gen = torch.Generator(device=DEV).manual_seed(3)

    def randn(*shape, std=1.0):
        return (torch.randn(shape, generator=gen, device=DEV) * std).bfloat16()

    x, wg, wu = randn(ROWS, 48), randn(DIM, 48, std=0.2), randn(DIM, 48, std=0.2)
    dh = workloads.generate_bf16_bits((ROWS, DIM), 4, DEV)
    h, g, u = rla.gated_ffn(x, wg, wu, "gelu_tanh", save=True)
    dx, _, _ = rla.gated_ffn_backward(dh, x, wg, wu, g, u, "gelu_tanh", need_dw=False)
    for at in PLACES:
        t = dict(x=rows(x, at).cpu(), w_gate=wg.cpu(), w_up=wu.cpu(), dh=rows(dh, at).cpu())
        check_forward(t, "gelu_tanh", rows(h, at), rows(g, at), rows(u, at))
        check_backward(t, "gelu_tanh", rows(g, at), rows(u, at), rows(dx, at), None, None)


@pytest.mark.parametrize("tokens", [1, 2])
@pytest.mark.parametrize("out", [1 << 25, (1 << 25) + 1, (1 << 26) - 4, (1 << 26) - 3, (1 << 26) - 1])
def test_q8_matmul_of_the_most_outputs(out, tokens):
    """Every width that is taken, up to the last: sums below 2^24 and two roundings, so bit for bit."""
    gen = torch.Generator(device=DEV).manual_seed(5)
    a = torch.randint(-127, 128, (tokens, 16), generator=gen, device=DEV, dtype=torch.int8)
    b = torch.randint(-128, 128, (out, 16), generator=gen, device=DEV, dtype=torch.int8)
    sa, sb = torch.rand(tokens, generator=gen, device=DEV), torch.rand(out, generator=gen, device=DEV)
    y = rla.q8_matmul(a, sa, b, sb, dtype=torch.float32)
    for m in range(tokens):
        want = (b.float() * a[m].float()).sum(1) * sa[m] * sb
        assert torch.equal(y[m], want)
