"""Every kernel of the block's matrix products on the GPU, at the sizes of tests/block_tiles.py.

The inputs are small integers, so that every sum is exact in fp32 whatever its order: each element of the
projections, of dx and of the weights' gradients has one right value, and one step of k left out, taken twice or
read from the wrong slot changes whole tiles.  The products in 64 bits are formed on the GPU.
"""
from __future__ import annotations

import pytest
import torch

from tests import block_tiles as bt
from tests.block_tools import U, half_step, tiny
from tests.test_gated_ffn_gpu import KINDS, act64, act_bounds

pytestmark = pytest.mark.gpu

rla = pytest.importorskip("rope_ltx3drope_amd")

DEV = "cuda:0"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def fresh():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def integers(gen, low, high, *shape):
    return torch.randint(low, high + 1, shape, generator=gen, device=DEV)


def product(a, b):
    """a b in 64 bits, which hold these sums exactly."""
    return a.double() @ b.double().contiguous()


def assert_same(got, want, what):
    """Every element equal (in got's type); names the first that is not and how many."""
    want = want.to(got.dtype)
    bad = got != want
    if bool(bad.any()):
        at = tuple(int(i) for i in bad.nonzero()[0])
        rows, cols = bad.any(1).sum().item(), bad.any(0).sum().item()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} differ, in {rows} rows and {cols} columns; "
                             f"first at {at}: {float(got[at])} for {float(want[at])}")


@pytest.mark.parametrize("kind,tokens,dim,hidden", [(k, *s) for k, sizes in bt.FFN.items() for s in sizes + bt.FEW])
def test_feed_forward(kind, tokens, dim, hidden):
    dtype = DTYPES[kind]
    gen = torch.Generator(device=DEV).manual_seed(tokens * hidden + dim)
    x = integers(gen, -3, 3, tokens, dim).to(dtype)
    wg, wu = (integers(gen, -2, 2, hidden, dim).to(dtype) for _ in range(2))
    act = KINDS[(tokens + dim) % 3]
    h, g, u = rla.gated_ffn(x, wg, wu, act, save=True)
    assert_same(g, product(x, wg.T), "g")
    assert_same(u, product(x, wu.T), "u")
    # h from the g and u of every element
    v, w = g.double(), u.double()
    a, tol = act64(v, act)[0], act_bounds(v, act)[0]
    want = a * w
    tol = tol * w.abs() + 2 * U * want.abs()
    tol = tol + half_step(dtype) * (want.abs() + tol) + tiny(dtype)
    off = (h.double() - want).abs() / tol
    worst = float(off.max())
    assert worst <= 1, (worst, float(v.flatten()[off.argmax()]), float(w.flatten()[off.argmax()]))
    del h, v, w, a, tol, want, off

    # silu of 64 and 128 is its argument and its slope 1, of -1024 both are 0: dg and du are integers too
    choice = torch.tensor([64.0, 128.0, -1024.0], device=DEV)
    g = choice[integers(gen, 0, 2, tokens, hidden)]
    u, dh = integers(gen, -3, 3, tokens, hidden).float(), integers(gen, -2, 2, tokens, hidden).to(dtype)
    dx, dwg, dwu = rla.gated_ffn_backward(dh, x, wg, wu, g, u, "silu")
    up = (g > 0).double()
    dg, du = dh.double() * u.double() * up, dh.double() * g.double() * up
    for t in (dx, dwg, dwu):
        assert t.dtype == dtype
    assert_same(dx, product(dg, wg) + product(du, wu), "dx")
    assert_same(dwg, product(dg.T, x), "dw_gate")
    assert_same(dwu, product(du.T, x), "dw_up")


@pytest.mark.parametrize("tokens,dim,out", bt.Q8 + bt.FEW)
def test_8_bit_layer(tokens, dim, out):
    gen = torch.Generator(device=DEV).manual_seed(tokens * out + dim)
    a, b = integers(gen, -128, 127, tokens, dim).to(torch.int8), integers(gen, -128, 127, out, dim).to(torch.int8)
    sa, sb = (torch.rand(n, generator=gen, device=DEV) * 0.02 + 1e-3 for n in (tokens, out))
    sums = product(a, b.T)
    # the sum to fp32, then two products: each rounded once, on either side
    want = sums.float() * sa[:, None] * sb
    assert_same(rla.q8_matmul(a, sa, b, sb, dtype=torch.float32), want, "y")
    assert_same(rla.q8_matmul(a, sa, b, sb), want, "y in bf16")


def test_the_integers_stay_exact():
    """The largest sums of the tests above stay within fp32's 2^24 (dx: F of 3 * 2 * 2 and of 2 * 128 * 2; dw: M of
    6 * 3 and of 256 * 3), so that no order of them rounds; dg and du (at most 6 and 256) fit bf16's 8 bits."""
    for sizes in bt.FFN.values():
        for tokens, dim, hidden in sizes + bt.FEW:
            assert dim * 3 * 2 < 2 ** 24
            assert hidden * (3 * 2 * 2 + 2 * 128 * 2) < 2 ** 24
            assert tokens * 256 * 3 < 2 ** 24
