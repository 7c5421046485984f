"""The rotation with several axes on tokens of 2 and 4 GB, whose heads and channels make 2^20 workgroups and more."""
from __future__ import annotations

import pytest
import torch

from tests.test_axes_gpu import check

pytestmark = pytest.mark.gpu

rla = pytest.importorskip("rope_ltx3drope_amd")

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def fresh():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("heads,head_dim,pairs,pairing,tokens", [(16384, 65534, 32767, "halves", 2),
                                                                 (32768, 65536, 32768, "adjacent", 1),
                                                                 (8200, 65535, 1, "adjacent", 2)])
def test_tokens_of_more_workgroups_than_a_small_launch(heads, head_dim, pairs, pairing, tokens):
    gen = torch.Generator(device=DEV).manual_seed(heads)
    q = torch.randn(tokens, heads, head_dim, generator=gen, device=DEV, dtype=torch.bfloat16)
    positions = torch.randint(0, 1000, (2, tokens), generator=gen, device=DEV)
    freq = torch.rand(pairs, generator=gen, device=DEV, dtype=torch.float64)
    axis = torch.randint(0, 2, (pairs,), generator=gen, device=DEV).to(torch.uint8)
    out, none = rla.axes_apply_qk(q, None, positions, freq, axis, pairing=pairing)
    assert none is None
    for lo in range(0, heads, 4096):  # some heads at a time: the same bits
        part, _ = rla.axes_apply_qk(q[:, lo:lo + 4096].contiguous(), None, positions, freq, axis, pairing=pairing)
        assert torch.equal(out[:, lo:lo + 4096], part), lo
    del part
    # and some heads against the formula: a few hundred pairs, whose channels stand side by side in a small head
    some = torch.randint(0, pairs, (min(pairs, 200),), generator=gen, device=DEV)
    at = (lambda i: (i, i + pairs)) if pairing == "halves" else (lambda i: (2 * i, 2 * i + 1))
    channels = torch.stack(at(some), 1).reshape(-1)
    cut = lambda t: t[:, ::1013][..., channels].cpu()[None]  # noqa: E731
    check(cut(q), cut(out), positions.cpu()[:, None], freq[some].cpu(), axis[some].cpu(), "adjacent", False, "heads")
