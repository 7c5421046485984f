"""CPU tests of the layer norms: the oracle's gradients against central differences, and the C ABI's
refusals, which come before anything touches a GPU."""
from __future__ import annotations

import ctypes
import os

import pytest
import torch

import oracle.block as ob
from tests.test_block_host import check_differences

rla = pytest.importorskip("rope_ltx3drope_amd")
from rope_ltx3drope_amd import _lib  # noqa: E402

if not os.path.exists(_lib.LIB_PATH):
    pytest.skip("libltx3drope.so not built (python -m rope_ltx3drope_amd.build)", allow_module_level=True)

L = _lib.lib()
FAKE = 1 << 20  # an aligned address that no rule below dereferences


def test_gradients_of_the_oracle():
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    B, S, D = 2, 3, 10
    y, res, gate, w, bias, sc, sh, dr, dn = r(B, S, D), r(B, S, D), r(B, D), r(D), r(D), r(B, D), r(B, D), \
        r(B, S, D), r(B, S, D)

    def f(y, res, gate, w, bias, sc, sh):
        x = ob.layer_norm_residual(y, res, gate)
        return (x * dr).sum() + (ob.layer_norm_before(x, w, bias, sc, sh, 1e-3) * dn).sum()

    x = ob.layer_norm_residual(y, res, gate)
    dR, dw, dbias, dsc, dsh = ob.layer_norm_before_backward(dn, x, w, bias, sc, dr, 1e-3)
    dy, dres, dgate = ob.layer_norm_after_backward(dR, y, gate)
    args, grads = (y, res, gate, w, bias, sc, sh), [dy, dres, dgate, dw, dbias, dsc, dsh]
    check_differences(f, args, grads)
    # each gradient's own mistakes are found: the mean left in, the bias left out of the scale's
    for i, wrong in ((1, dres + 1e-3), (5, dsc - bias * dn.sum(1)), (3, dw * 1.001)):
        with pytest.raises(AssertionError):
            check_differences(f, args, grads[:i] + [wrong] + grads[i + 1:])


def test_the_oracle_against_torch():
    g = torch.Generator().manual_seed(4)
    x, w, b = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((2, 5, 33), (33,), (33,)))
    want = torch.nn.functional.layer_norm(x, (33,), w, b, 1e-5)
    assert torch.allclose(ob.layer_norm_before(x, w, b, None, None, 1e-5), want, rtol=1e-13, atol=1e-13)


def call(**kw):
    c = dict(dtype=0, param_dtype=0, after=1, batch=2, rows=3, dim=64, eps=1e-6, y=FAKE, residual=FAKE * 2, r=FAKE * 3,
             n=FAKE * 4)
    c.update(kw)
    return _lib.LayerNorm(**c)


def status(**kw):
    reason = ctypes.c_int(-1)
    return L.ltx3drope_layer_norm(call(**kw), None, reason), _lib.REASONS[reason.value]


@pytest.mark.parametrize("kw", [dict(eps=0.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(eps=-1.0),
                                dict(after=2), dict(after=-1), dict(reserved=1), dict(after=0),
                                dict(after=0, y=None), dict(after=0, y=None, r=None, gate=FAKE * 5)])
def test_invalid(kw):
    assert status(**kw)[0] == _lib.E_INVALID


@pytest.mark.parametrize("kw,reason", [
    (dict(dtype=2), "DTYPE"), (dict(param_dtype=1), "DTYPE"), (dict(dtype=1, param_dtype=3), "DTYPE"),
    (dict(dim=0), "NONPOSITIVE_DIM"), (dict(rows=-1), "NONPOSITIVE_DIM"), (dict(batch=-1), "NONPOSITIVE_DIM"),
    (dict(dim=16385), "TOO_LARGE"), (dict(batch=1 << 16, rows=1 << 15), "TOO_LARGE"),
    (dict(batch=65536, rows=1, shift=FAKE * 5), "TOO_LARGE"),
    (dict(y=None), "NULLPTR"), (dict(n=None), "NULLPTR"), (dict(r=None), "NULLPTR"), (dict(residual=None), "NULLPTR"),
    (dict(y=FAKE + 2), "ALIGN"), (dict(bias=FAKE * 5 + 1), "ALIGN"), (dict(n=FAKE * 3), "OVERLAP"),
    (dict(r=FAKE * 2 + 64), "OVERLAP"), (dict(scale=FAKE * 4), "OVERLAP"), (dict(), "NOT_DEVICE_PTR"),
    (dict(r=FAKE * 2, n=FAKE), "NOT_DEVICE_PTR"),  # exactly over the inputs: passes the overlap rule
    (dict(after=0, y=None, r=None), "NOT_DEVICE_PTR"),
])
def test_refusals(kw, reason):
    assert status(**kw) == (_lib.E_UNSUPPORTED, reason)


def test_empty_calls_look_at_no_pointer():
    for kw in (dict(rows=0), dict(batch=0)):
        assert status(y=None, residual=None, r=None, n=None, **kw) == (_lib.OK, "OK")
    assert L.ltx3drope_layer_norm(None, None, None) == _lib.E_INVALID
    assert L.ltx3drope_layer_norm_backward(None, None, None) == _lib.E_INVALID
    assert L.ltx3drope_layer_norm_backward_workspace(None) == _lib.E_INVALID


def backward_call(**kw):
    c = dict(dtype=0, param_dtype=0, after=1, batch=2, rows=3, dim=64, eps=1e-6, dr=FAKE, dn=FAKE * 2, y=FAKE * 3,
             r=FAKE * 4, gate=FAKE * 5, dgate=FAKE * 6, dresidual=FAKE * 7, dy=FAKE * 8, workspace=FAKE * 9,
             workspace_bytes=1 << 20)
    c.update(kw)
    return _lib.LayerNormBackward(**c)


@pytest.mark.parametrize("kw,want", [
    (dict(workspace_bytes=16), (_lib.E_INVALID, "OK")), (dict(gate=None), (_lib.E_INVALID, "OK")),
    (dict(dweight=FAKE * 10), (_lib.E_INVALID, "OK")), (dict(dscale=FAKE * 10), (_lib.E_INVALID, "OK")),
    (dict(workspace_bytes=-1), (_lib.E_INVALID, "OK")), (dict(after=0), (_lib.E_INVALID, "OK")),
    (dict(dn=None), (_lib.E_UNSUPPORTED, "NULLPTR")), (dict(y=None), (_lib.E_UNSUPPORTED, "NULLPTR")),
    (dict(r=None), (_lib.E_UNSUPPORTED, "NULLPTR")), (dict(dresidual=None), (_lib.E_UNSUPPORTED, "NULLPTR")),
    (dict(dy=None), (_lib.E_UNSUPPORTED, "NULLPTR")), (dict(workspace=None), (_lib.E_UNSUPPORTED, "NULLPTR")),
    (dict(workspace=FAKE * 9 + 8), (_lib.E_UNSUPPORTED, "ALIGN")),
    (dict(workspace=FAKE * 3), (_lib.E_UNSUPPORTED, "OVERLAP")), (dict(dy=FAKE * 7), (_lib.E_UNSUPPORTED, "OVERLAP")),
    (dict(dshift=FAKE * 6), (_lib.E_UNSUPPORTED, "OVERLAP")),
    (dict(), (_lib.E_UNSUPPORTED, "NOT_DEVICE_PTR")),
    (dict(dgate=None, y=None, workspace=None, workspace_bytes=0), (_lib.E_UNSUPPORTED, "NOT_DEVICE_PTR")),
    (dict(rows=0, dgate=None, dresidual=None, dy=None, dn=None, r=None, y=None, workspace=None, workspace_bytes=0),
     (_lib.OK, "OK")),
])
def test_backward_refusals(kw, want):
    reason = ctypes.c_int(-1)
    assert (L.ltx3drope_layer_norm_backward(backward_call(**kw), None, reason), _lib.REASONS[reason.value]) == want


def test_workspace_sizes():
    size = lambda **kw: L.ltx3drope_layer_norm_backward_workspace(backward_call(**kw))  # noqa: E731
    assert size(dgate=None) == 0 and size(rows=0) == 0 and size(batch=0) == 0
    assert size() == 3 * 2 * 3 * 64 * 4  # three sums of two samples, a workgroup a row
    assert size(eps=0.0) == _lib.E_INVALID and size(dim=1 << 20) == _lib.E_UNSUPPORTED


def test_descriptors_as_bytes():
    """The packed bytes are the structures: fields of both at the same offsets."""
    for cls, packed in ((_lib.LayerNorm, _lib.LAYER_NORM_BYTES), (_lib.LayerNormBackward, _lib.LAYER_NORM_BACKWARD_BYTES)):
        values = list(range(1, len(cls._fields_) + 1))
        raw = packed.pack(*values)
        s = cls.from_buffer_copy(raw)
        assert len(raw) == ctypes.sizeof(cls)
        assert [getattr(s, n) for n, _ in cls._fields_] == values
