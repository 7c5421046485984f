"""Scales of the 8-bit floating point layer whose leading dimensions hold some of size 1, of any strides there: one new
token of each sequence, its scales out of those of many tokens."""
from __future__ import annotations

import pytest
import torch

from tests.block_tools import U

pytestmark = pytest.mark.gpu

rla = pytest.importorskip("rope_ltx3drope_amd")

DEV = "cuda:0"


def same_bytes(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("batch,tokens", [(4, 7), (1, 5), (3, 1), (40, 3)])
def test_one_token_of_each_sequence(batch, tokens):
    gen = torch.Generator(device=DEV).manual_seed(batch)
    x = torch.randn(batch, tokens, 400, generator=gen, device=DEV)
    w, ws = rla.f8_quantize_weight(torch.randn(70, 400, generator=gen, device=DEV))
    q, s = rla.f8_quantize(x)
    full = rla.f8_matmul(q, s, w, ws, dtype=torch.float32)
    wide = lambda v: v.double().repeat_interleave(128, -1)[..., :400]  # noqa: E731
    mag = (q.double().abs() * wide(s)) @ (w.double().abs() * wide(ws)).t().contiguous()
    for scales in (s, s.contiguous()):
        for t in range(tokens):
            one, scale = q[:, t:t + 1].contiguous(), scales[:, t:t + 1]
            got = rla.f8_matmul(one, scale, w, ws, dtype=torch.float32)
            want = rla.f8_matmul(one, scale.contiguous(), w, ws, dtype=torch.float32)
            assert torch.equal(got, want)
            # the same sums among those of many tokens, which may be split otherwise: both are within their roundings
            assert bool(((got - full[:, t:t + 1]).abs() <= 2 * (2 * 128 + 4 + 4 + 17) * U * mag[:, t:t + 1]).all())
    # and scales that go there
    out = torch.full((batch, tokens, 4), 7.0, device=DEV)
    for t in range(tokens):
        x1 = x[:, t:t + 1].contiguous()
        q1, s1 = rla.f8_quantize(x1, scale_out=out[:, t:t + 1])
        assert same_bytes(q1, q[:, t:t + 1]) and torch.equal(out[:, t], s[:, t])
    assert torch.equal(out, s)


def test_dimensions_that_are_not_one_are_refused():
    q, s = rla.f8_quantize(torch.randn(4, 6, 200, device=DEV))
    w, ws = rla.f8_quantize_weight(torch.randn(30, 200, device=DEV))
    with pytest.raises(rla.Ltx3dRopeUnsupported) as e:
        rla.f8_matmul(q[:, :3].contiguous(), s[:, :3], w, ws)
    assert e.value.reason == "NOT_CONTIGUOUS"
    five = s.reshape(2, 1, 2, 1, 6, 2)
    got = rla.f8_matmul(q.view(2, 1, 2, 1, 6, 200), five, w, ws)
    assert torch.equal(got.view(4, 6, 30), rla.f8_matmul(q, s, w, ws))
