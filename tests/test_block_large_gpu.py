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


def test_norm_vector_gradients():
    """The vectors' gradients over all rows, against 64 bits a few thousand rows at a time."""
    x, dn = (workloads.generate_bf16_bits((ROWS, DIM), seed, DEV) for seed in (6, 7))
    w = torch.linspace(0.5, 1.5, DIM, device=DEV)
    gate = torch.linspace(-1.0, 1.0, DIM, device=DEV)[None]
    b = rla.norm_before_backward(dn[None], x[None], w, gate, gate)
    dweight, dscale, dshift = (t.double() for t in b[1:])
    a = rla.norm_after_backward(dn[None], None, x[None], None, w, gate, next_norm=False)
    want, p2, terms, terms2 = (torch.zeros(DIM, dtype=torch.float64, device=DEV) for _ in range(4))
    for at in range(0, ROWS, 1 << 16):
        r, v = x[at:at + (1 << 16)].double(), dn[at:at + (1 << 16)].double()
        hat = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + 1e-6)
        want += (v * hat).sum(0)
        terms += (v * hat).abs().sum(0)
        p2 += v.sum(0)
        terms2 += v.abs().sum(0)
    # a thread's walk adds its row of 512 workgroups' (DIM / 8 threads a row, one row a workgroup at a time),
    # the join 512 parts; 40 operations for a term, and a few for the factors
    steps = (ROWS / 512 + 512 + 48) * 2.0 ** -24
    w, gate = w.double(), gate[0].double()
    for got, value, size in ((dweight, (1 + gate) * want, (1 + gate).abs() * terms), (dscale[0], w * want, w * terms),
                             (dshift[0], p2, terms2), (a.dweight.double(), gate * want, gate.abs() * terms),
                             (a.dgate[0].double(), w * want, w * terms)):
        assert bool(((got - value).abs() <= steps * size).all()), float(((got - value).abs() / size).max())


def test_gated_ffn_weight_gradients():
    """A weight's gradient over slopes of more than 2^32 elements: integers below 2^24, so exact."""
    gen = torch.Generator(device=DEV).manual_seed(8)
    x = torch.randint(-1, 2, (ROWS, 48), generator=gen, device=DEV).bfloat16()
    wg = torch.zeros(DIM, 48, dtype=torch.bfloat16, device=DEV)
    g = torch.randint(0, 2, (ROWS, DIM), generator=gen, device=DEV, dtype=torch.int8).float() * 1088.0 - 1024.0
    u = torch.ones_like(g)  # silu of 64 is 64 and its slope 1, of -1024 both are 0
    dh = torch.randint(-1, 2, (ROWS, DIM), generator=gen, device=DEV, dtype=torch.int8).bfloat16()
    _, dwg, dwu = rla.gated_ffn_backward(dh, x, wg, wg, g, u, "silu", need_dx=False)
    want = torch.zeros(DIM, 48, dtype=torch.float64, device=DEV)
    for at in range(0, ROWS, 1 << 16):
        dg = dh[at:at + (1 << 16)].double() * (g[at:at + (1 << 16)] > 0)
        want += dg.T.contiguous() @ x[at:at + (1 << 16)].double()
    assert torch.equal(dwg, want.bfloat16()) and torch.equal(dwu, (64 * want).bfloat16())


def test_norm_backward_of_the_most_samples():
    """65535 samples of the widest rows: one partial row each, 13 GB of them."""
    batch, dim = 65535, 16384
    x, dn = (workloads.generate_bf16_bits((batch, 1, dim), seed, DEV) for seed in (9, 10))
    w = torch.linspace(0.5, 1.5, dim, device=DEV)
    scale = workloads.generate_bf16_bits((batch, dim), 11, DEV).float()
    g = rla.norm_before_backward(dn, x, w, scale, scale)
    torch.cuda.synchronize()
    want, size = (torch.zeros(dim, dtype=torch.float64, device=DEV) for _ in range(2))
    for at in range(0, batch, 2048):
        part = slice(at, min(at + 2048, batch))
        one = rla.norm_before_backward(dn[part], x[part], w, scale[part], scale[part])
        assert torch.equal(g.dx[part], one.dx)
        assert torch.equal(g.dscale[part], one.dscale) and torch.equal(g.dshift[part], one.dshift)
        r, v = x[part, 0].double(), dn[part, 0].double()
        t = v * r * torch.rsqrt((r * r).mean(-1, keepdim=True) + 1e-6) * (1 + scale[part].double())
        want += t.sum(0)
        size += t.abs().sum(0)
    # 64 lanes down 65535 samples, then 16 sums; 48 operations for a term
    steps = (65536 / 64 + 16 + 48) * 2.0 ** -24
    assert bool(((g.dweight.double() - want).abs() <= steps * size).all())
