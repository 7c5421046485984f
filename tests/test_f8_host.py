"""CPU tests of the 8-bit floating point linear layer: the oracle's rounding by hand, and the C ABI's refusals,
which come before anything touches a GPU."""
from __future__ import annotations

import ctypes
import os

import pytest
import torch

import oracle.f8 as of

rla = pytest.importorskip("rope_ltx3drope_amd")
from rope_ltx3drope_amd import _lib  # noqa: E402

if not os.path.exists(_lib.LIB_PATH):
    pytest.skip("libltx3drope.so not built (python -m rope_ltx3drope_amd.build)", allow_module_level=True)

L = _lib.lib()
FAKE = 1 << 26  # an aligned address that no rule below dereferences


def nearest(v):
    """e4m3 by definition: the nearest of all its finite values, ties to the even mantissa."""
    every = torch.arange(256, dtype=torch.uint8).view(of.F8).double()
    codes = torch.arange(256)
    keep = torch.isfinite(every)
    every, codes = every[keep], codes[keep]
    out = torch.empty(v.numel(), dtype=torch.float64)
    for i, x in enumerate(v.double().reshape(-1)):
        gap = (every - x).abs()
        best = torch.nonzero(gap == gap.min()).reshape(-1)
        even = [int(b) for b in best if int(codes[b]) % 2 == 0]
        out[i] = every[even[0] if even else int(best[0])]
    return out.view(v.shape)


def test_the_oracle_rounds_to_the_nearest_value():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(3, 200, generator=g) * torch.exp(torch.randn(200, generator=g) * 2)
    q, s = of.quantize(x, 1)
    assert s.shape == (3, 2)
    for r in range(3):
        for b, (lo, hi) in enumerate(((0, 128), (128, 200))):
            assert float(s[r, b]) == float(x[r, lo:hi].abs().max() / torch.tensor(448.0))
            assert torch.equal(q[r, lo:hi].double(), nearest(x[r, lo:hi] / s[r, b]))
    q2, s2 = of.quantize_rows(x)
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)
    q, s = of.quantize(x, 128)
    assert s.shape == (1, 2) and float(s[0, 1]) == float(x[:, 128:].abs().max() / torch.tensor(448.0))


def test_gradients_of_the_layer_against_differences():
    """y = x w^T is bilinear: its slope along a direction is exact, and dx = dy w, dw = dy^T x give it."""
    g = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    x, w, dy, vx, vw = r(5, 7), r(6, 7), r(5, 6), r(5, 7), r(6, 7)
    loss = lambda x, w: float(((x @ w.t()) * dy).sum())  # noqa: E731
    dx, dw = dy @ w, dy.t() @ x
    h = 1e-3
    assert abs((loss(x + h * vx, w) - loss(x - h * vx, w)) / (2 * h) - float((dx * vx).sum())) < 1e-9
    assert abs((loss(x, w + h * vw) - loss(x, w - h * vw)) / (2 * h) - float((dw * vw).sum())) < 1e-9


def quantize_status(**kw):
    c = dict(dtype=0, blocks=0, rows=200, dim=300, turned_pitch=256, scale_strides=(3, 1), scale_turned_strides=(2, 1), x=FAKE, q=FAKE * 2, scale=FAKE * 3,
             q_turned=FAKE * 4, scale_turned=FAKE * 5)
    c.update(kw)
    for n in ("scale_strides", "scale_turned_strides"):
        c[n] = (_lib.i64 * 2)(*c[n])
    reason = ctypes.c_int(-1)
    return L.ltx3drope_f8_quantize(_lib.F8Quantize(**c), None, reason), _lib.REASONS[reason.value]


@pytest.mark.parametrize("kw", [dict(blocks=2), dict(blocks=-1), dict(q_turned=None), dict(scale_turned=None),
                                dict(turned_pitch=199), dict(scale_strides=(-1, 1)), dict(scale_turned_strides=(1, -1))])
def test_quantize_invalid(kw):
    assert quantize_status(**kw)[0] == _lib.E_INVALID
    assert L.ltx3drope_f8_quantize(None, None, None) == _lib.E_INVALID


@pytest.mark.parametrize("kw,reason", [
    (dict(dtype=2), "DTYPE"), (dict(dim=0), "NONPOSITIVE_DIM"), (dict(rows=-1), "NONPOSITIVE_DIM"),
    (dict(dim=1 << 31), "TOO_LARGE"), (dict(rows=1 << 31, turned_pitch=1 << 31), "TOO_LARGE"),
    (dict(turned_pitch=1 << 32), "TOO_LARGE"), (dict(rows=1 << 26, dim=1 << 12, turned_pitch=1 << 26), "TOO_LARGE"),
    (dict(x=None), "NULLPTR"), (dict(q=None), "NULLPTR"), (dict(scale=None), "NULLPTR"), (dict(x=FAKE + 1), "ALIGN"),
    (dict(scale=FAKE * 3 + 2), "ALIGN"), (dict(scale_turned=FAKE * 5 + 1), "ALIGN"), (dict(q=FAKE), "OVERLAP"),
    (dict(q=FAKE + 239996), "OVERLAP"), (dict(q_turned=FAKE * 2 + 59999), "OVERLAP"), (dict(scale=FAKE * 4), "OVERLAP"),
    (dict(scale_turned=FAKE * 4 + 300 * 256 - 4), "OVERLAP"), (dict(), "NOT_DEVICE_PTR"),
    (dict(q=FAKE + 240000), "NOT_DEVICE_PTR"), (dict(scale_turned=FAKE * 4 + 300 * 256), "NOT_DEVICE_PTR"),
    (dict(q_turned=None, scale_turned=None, turned_pitch=0), "NOT_DEVICE_PTR"), (dict(blocks=1), "NOT_DEVICE_PTR"),
    (dict(scale_strides=(1 << 31, 1)), "TOO_LARGE"), (dict(scale_strides=(2, 1)), "OVERLAP"),
    (dict(scale_strides=(1, 199)), "OVERLAP"), (dict(scale_strides=(0, 1)), "OVERLAP"),
    (dict(scale_turned_strides=(1, 1)), "OVERLAP"), (dict(scale_strides=(1, 200)), "NOT_DEVICE_PTR"),
    (dict(scale_turned_strides=(1, 300)), "NOT_DEVICE_PTR"),
    # 200 rows of 3 blocks, the blocks 1000 apart: the last scale is number 2199
    (dict(scale_strides=(1, 1000), q=FAKE * 3 + 2199 * 4 + 3), "OVERLAP"),
    (dict(scale_strides=(1, 1000), q=FAKE * 3 + 2200 * 4), "NOT_DEVICE_PTR"),
])
def test_quantize_refusals(kw, reason):
    assert quantize_status(**kw) == (_lib.E_UNSUPPORTED, reason)


def test_quantize_empty():
    assert quantize_status(rows=0, x=None, q=None, scale=None, q_turned=None, scale_turned=None) == (_lib.OK, "OK")


def call(**kw):
    c = dict(dtype=0, b_rows=0, tokens=100, dim=300, out=200, a_pitch=300, b_pitch=300, a_scale_strides=(3, 1),
             b_scale_strides=(3, 1), a=FAKE, b=FAKE * 2,
             a_scale=FAKE * 3, b_scale=FAKE * 4, y=FAKE * 5, workspace=FAKE * 6, workspace_bytes=1 << 24)
    c.update(kw)
    for n in ("a_scale_strides", "b_scale_strides"):
        c[n] = (_lib.i64 * 2)(*c[n])
    return _lib.F8Matmul(**c)


def status(**kw):
    reason = ctypes.c_int(-1)
    return L.ltx3drope_f8_matmul(call(**kw), None, reason), _lib.REASONS[reason.value]


@pytest.mark.parametrize("kw", [dict(b_rows=2), dict(a_pitch=299), dict(b_pitch=0), dict(workspace_bytes=-1),
                                dict(a_scale_strides=(1, -1)), dict(b_scale_strides=(-3, 1)),
                                dict(tokens=100, dim=8192, out=64, a_pitch=8192, b_pitch=8192, workspace_bytes=16)])
def test_matmul_invalid(kw):
    assert status(**kw)[0] == _lib.E_INVALID
    assert L.ltx3drope_f8_matmul(None, None, None) == _lib.E_INVALID
    assert L.ltx3drope_f8_matmul_workspace(None) == _lib.E_INVALID


@pytest.mark.parametrize("kw,reason", [
    (dict(dtype=2), "DTYPE"), (dict(dim=0), "NONPOSITIVE_DIM"), (dict(tokens=-1), "NONPOSITIVE_DIM"),
    (dict(out=-1), "NONPOSITIVE_DIM"), (dict(dim=1 << 21, a_pitch=1 << 21, b_pitch=1 << 21), "TOO_LARGE"),
    (dict(a_pitch=1 << 22), "TOO_LARGE"), (dict(b_pitch=1 << 40), "TOO_LARGE"), (dict(tokens=1 << 26), "TOO_LARGE"),
    (dict(out=1 << 26), "TOO_LARGE"), (dict(tokens=1 << 18, out=1 << 17), "TOO_LARGE"),
    (dict(a_scale_strides=(1 << 20, 1)), "TOO_LARGE"), (dict(b_scale_strides=(1, 1 << 31)), "TOO_LARGE"),
    (dict(a_scale_strides=(1, 5000), y=FAKE * 3 + 10099 * 4), "OVERLAP"),
    (dict(a_scale_strides=(1, 5000), y=FAKE * 3 + 10100 * 4), "NOT_DEVICE_PTR"),
    (dict(a=None), "NULLPTR"), (dict(b=None), "NULLPTR"), (dict(a_scale=None), "NULLPTR"),
    (dict(b_scale=None), "NULLPTR"), (dict(y=None), "NULLPTR"), (dict(y=FAKE * 5 + 2), "ALIGN"),
    (dict(a_scale=FAKE * 3 + 1), "ALIGN"), (dict(bias=FAKE * 7 + 2), "ALIGN"), (dict(y=FAKE), "OVERLAP"),
    (dict(y=FAKE * 2 + 59996), "OVERLAP"), (dict(bias=FAKE * 5), "OVERLAP"), (dict(y=FAKE * 4 + 20), "OVERLAP"),
    (dict(y=FAKE * 4 + 24), "NOT_DEVICE_PTR"), (dict(b_rows=1, y=FAKE * 4 + 200 * 12 - 4), "OVERLAP"),
    (dict(b_rows=1, y=FAKE * 4 + 200 * 12), "NOT_DEVICE_PTR"),
    # rows further apart: the last one ends at 199 * 320 + 300
    (dict(b_pitch=320, y=FAKE * 2 + 63976), "OVERLAP"), (dict(b_pitch=320, y=FAKE * 2 + 63980), "NOT_DEVICE_PTR"),
    (dict(), "NOT_DEVICE_PTR"),
])
def test_matmul_refusals(kw, reason):
    assert status(**kw) == (_lib.E_UNSUPPORTED, reason)


def test_matmul_empty_and_workspace():
    none = dict(a=None, b=None, a_scale=None, b_scale=None, y=None, workspace=None, workspace_bytes=0)
    for kw in (dict(tokens=0), dict(out=0)):
        assert status(**none, **kw) == (_lib.OK, "OK")
    size = lambda **kw: L.ltx3drope_f8_matmul_workspace(call(**kw))  # noqa: E731
    assert size(tokens=0) == 0 and size(tokens=16, dim=1 << 16, a_pitch=1 << 16, b_pitch=1 << 16) == 0
    assert size(tokens=100, dim=8192, out=64, a_pitch=8192, b_pitch=8192) > 0
    assert size(dtype=7) == _lib.E_UNSUPPORTED and size(b_rows=3) == _lib.E_INVALID


def test_descriptors_as_bytes():
    for cls, packed in ((_lib.F8Quantize, _lib.F8_QUANTIZE_BYTES), (_lib.F8Matmul, _lib.F8_BYTES)):
        values = list(range(1, len(cls._fields_) + 3))  # two fields of two numbers
        raw = packed.pack(*values)
        s = cls.from_buffer_copy(raw)
        flat = []
        for n, _ in cls._fields_:
            v = getattr(s, n)
            flat += list(v) if hasattr(v, "__len__") else [v]
        assert len(raw) == ctypes.sizeof(cls) and flat == values
