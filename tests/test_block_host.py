"""CPU tests of the transformer-block operators: the oracle's gradients against central differences,
and the C ABI's refusals, which come before anything touches a GPU."""
from __future__ import annotations

import ctypes
import os

import pytest
import torch

import oracle.block as ob

rla = pytest.importorskip("rope_ltx3drope_amd")
from rope_ltx3drope_amd import _lib  # noqa: E402

if not os.path.exists(_lib.LIB_PATH):
    pytest.skip("libltx3drope.so not built (python -m rope_ltx3drope_amd.build)", allow_module_level=True)

L = _lib.lib()


def slope(f, args, i, direction, h=1e-5):
    def at(s):
        moved = list(args)
        moved[i] = moved[i] + s * direction
        return f(*moved)

    return float((at(h) - at(-h)) / (2 * h))


def check_differences(f, args, grads, seed=0):
    """The gradient of the scalar f along a random direction of each argument.  In float64 with h = 1e-5
    truncation (h^2) and rounding (1e-16 / h) are both about 1e-10 of the terms' sum: 1e-6 covers it."""
    gen = torch.Generator().manual_seed(seed)
    for i, g in enumerate(grads):
        if g is None:
            continue
        v = torch.randn(args[i].shape, generator=gen, dtype=torch.float64)
        want = slope(f, args, i, v)
        got = float((g * v).sum())
        assert abs(got - want) <= 1e-6 * (1 + float((g * v).abs().sum())), (i, got, want)


@pytest.mark.parametrize("offset,res_scale,post", [(0.0, 1.0, True), (1.0, 0.5, True), (1.0, 2.0, False)])
def test_norm_gradients_of_the_oracle(offset, res_scale, post):
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    B, S, D = 2, 3, 10
    y, res, w, gate, nw, ns, nb, dr, dn = r(B, S, D), r(B, S, D), r(D), r(B, D), r(D), r(B, D), r(B, D), r(B, S, D), \
        r(B, S, D)

    def f(y, res, w, gate, nw, ns, nb):
        x = ob.norm_after(y, res, w, gate, post, res_scale, 1e-3, offset)
        return (x * dr).sum() + (ob.norm_before(x, nw, ns, nb, 1e-3, offset) * dn).sum()

    x = ob.norm_after(y, res, w, gate, post, res_scale, 1e-3, offset)
    dR, dnw, dns, dnb = ob.norm_before_backward(dn, x, nw, ns, dr, 1e-3, offset)
    dy, dres, dw, dgate = ob.norm_after_backward(dR, y, w, gate, post, res_scale, 1e-3, offset)
    check_differences(f, (y, res, w, gate, nw, ns, nb), (dy, dres, dw, dgate, dnw, dns, dnb))
    # the oracle's own mistakes are found: a wrong offset or a lost projection fails the same check
    with pytest.raises(AssertionError):
        check_differences(f, (y, res, w, gate, nw, ns, nb), (dy + 1e-3 * y, dres, dw, dgate, dnw, dns, dnb))


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh"])
def test_ffn_gradients_of_the_oracle(kind):
    g = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    x, wg, wu, dh = r(4, 6), r(7, 6), r(7, 6), r(4, 7)

    def f(x, wg, wu):
        return (ob.gated_ffn(x, wg, wu, kind)[0] * dh).sum()

    _, gg, uu = ob.gated_ffn(x, wg, wu, kind)
    check_differences(f, (x, wg, wu), ob.gated_ffn_backward(dh, x, wg, wu, gg, uu, kind))


# ---- refusals of the norm --------------------------------------------------------------------------

FAKE = 1 << 20  # an aligned address that no rule below dereferences


def norm_call(**kw):
    c = dict(dtype=0, param_dtype=0, after=1, post_norm=1, next_norm=1, batch=2, rows=3, dim=64, eps=1e-6,
             weight_offset=0.0, residual_scale=1.0, y=FAKE, residual=FAKE * 2, r=FAKE * 3, n=FAKE * 4)
    c.update(kw)
    return _lib.Norm(**c)


def norm_status(**kw):
    reason = ctypes.c_int(-1)
    return L.ltx3drope_norm(norm_call(**kw), None, reason), _lib.REASONS[reason.value]


@pytest.mark.parametrize("kw", [dict(eps=0.0), dict(eps=float("nan")), dict(eps=-1.0), dict(weight_offset=float("inf")),
                                dict(residual_scale=float("nan")), dict(after=2), dict(post_norm=-1),
                                dict(next_norm=3), dict(reserved=1), dict(after=0), dict(next_norm=0),
                                dict(after=0, y=None, r=None, post_norm=0, next_norm=0, n=None),
                                dict(after=0, y=None, r=None, post_norm=0, residual_scale=2.0),
                                dict(after=0, y=None, r=FAKE, post_norm=0)])
def test_norm_invalid(kw):
    assert norm_status(**kw)[0] == _lib.E_INVALID


@pytest.mark.parametrize("kw,reason", [
    (dict(dtype=2), "DTYPE"), (dict(param_dtype=1), "DTYPE"), (dict(dtype=1, param_dtype=3), "DTYPE"),
    (dict(dim=0), "NONPOSITIVE_DIM"), (dict(rows=-1), "NONPOSITIVE_DIM"), (dict(batch=-1), "NONPOSITIVE_DIM"),
    (dict(dim=16385), "TOO_LARGE"), (dict(batch=1 << 16, rows=1 << 15), "TOO_LARGE"),
    (dict(batch=65536, rows=1, gate=FAKE * 5), "TOO_LARGE"),
    (dict(y=None), "NULLPTR"), (dict(n=None), "NULLPTR"), (dict(r=None), "NULLPTR"), (dict(residual=None), "NULLPTR"),
    (dict(y=FAKE + 2), "ALIGN"), (dict(next_weight=FAKE * 5 + 1), "ALIGN"), (dict(n=FAKE * 3), "OVERLAP"),
    (dict(r=FAKE * 2 + 64), "OVERLAP"), (dict(weight=FAKE * 4), "OVERLAP"), (dict(), "NOT_DEVICE_PTR"),
    (dict(r=FAKE * 2, n=FAKE), "NOT_DEVICE_PTR"),  # exactly over the inputs: passes the overlap rule
])
def test_norm_refusals(kw, reason):
    assert norm_status(**kw) == (_lib.E_UNSUPPORTED, reason)


def test_norm_empty_calls_look_at_no_pointer():
    for kw in (dict(rows=0), dict(batch=0)):
        assert norm_status(y=None, residual=None, r=None, n=None, **kw) == (_lib.OK, "OK")
    assert L.ltx3drope_norm(None, None, None) == _lib.E_INVALID


def backward_call(**kw):
    c = dict(dtype=0, param_dtype=0, after=1, post_norm=1, next_norm=1, batch=2, rows=3, dim=64, eps=1e-6,
             weight_offset=0.0, residual_scale=1.0, dr=FAKE, dn=FAKE * 2, y=FAKE * 3, r=FAKE * 4,
             weight=FAKE * 5, dweight=FAKE * 6, dresidual=FAKE * 7, dy=FAKE * 8, workspace=FAKE * 9,
             workspace_bytes=1 << 20)
    c.update(kw)
    return _lib.NormBackward(**c)


@pytest.mark.parametrize("kw,want", [
    (dict(workspace_bytes=16), (_lib.E_INVALID, "OK")), (dict(weight=None), (_lib.E_INVALID, "OK")),
    (dict(dgate=FAKE * 10), (_lib.E_INVALID, "OK")), (dict(next_norm=0), (_lib.E_INVALID, "OK")),
    (dict(dn=None), (_lib.E_UNSUPPORTED, "NULLPTR")), (dict(y=None), (_lib.E_UNSUPPORTED, "NULLPTR")),
    (dict(dy=None), (_lib.E_UNSUPPORTED, "NULLPTR")), (dict(workspace=None), (_lib.E_UNSUPPORTED, "NULLPTR")),
    (dict(workspace=FAKE * 9 + 8), (_lib.E_UNSUPPORTED, "ALIGN")),
    (dict(workspace=FAKE * 3), (_lib.E_UNSUPPORTED, "OVERLAP")), (dict(dy=FAKE * 7), (_lib.E_UNSUPPORTED, "OVERLAP")),
    (dict(dim=16385), (_lib.E_UNSUPPORTED, "TOO_LARGE")), (dict(), (_lib.E_UNSUPPORTED, "NOT_DEVICE_PTR")),
])
def test_norm_backward_refusals(kw, want):
    reason = ctypes.c_int(-1)
    st = L.ltx3drope_norm_backward(backward_call(**kw), None, reason)
    assert (st, _lib.REASONS[reason.value]) == want


def test_norm_workspace_sizes():
    size = L.ltx3drope_norm_backward_workspace
    assert size(backward_call(dweight=None)) == 0
    assert size(backward_call(rows=0)) == 0
    assert size(backward_call()) == 3 * 6 * 64 * 4  # 6 rows, a workgroup each, no per-sample vector
    assert size(backward_call(gate=FAKE, dgate=FAKE)) == 3 * 2 * 3 * 64 * 4
    assert size(backward_call(batch=1, rows=100000, dim=2048)) == 3 * 512 * 2048 * 4
    assert size(backward_call(eps=0.0)) == _lib.E_INVALID and size(None) == _lib.E_INVALID


# ---- refusals of the feed-forward block and the 8-bit linear layer -----------------------------------

def ffn_call(**kw):
    c = dict(dtype=1, activation=0, tokens=4, dim=64, hidden=32, x=FAKE, w_gate=FAKE * 2, w_up=FAKE * 3, h=FAKE * 4)
    c.update(kw)
    return _lib.GatedFfn(**c)


@pytest.mark.parametrize("kw,want", [
    (dict(activation=3), (_lib.E_INVALID, "OK")), (dict(activation=-1), (_lib.E_INVALID, "OK")),
    (dict(g=FAKE * 5), (_lib.E_INVALID, "OK")),
    (dict(tokens=17, dim=4096), (_lib.E_INVALID, "OK")),  # sums to be split, no workspace
    (dict(tokens=17, dim=4096, workspace_bytes=-1), (_lib.E_INVALID, "OK")),
    (dict(tokens=17, dim=4096, workspace_bytes=1 << 20), (_lib.E_UNSUPPORTED, "NULLPTR")),
    (dict(dtype=2), (_lib.E_UNSUPPORTED, "DTYPE")), (dict(dim=0), (_lib.E_UNSUPPORTED, "NONPOSITIVE_DIM")),
    (dict(tokens=-1), (_lib.E_UNSUPPORTED, "NONPOSITIVE_DIM")), (dict(dim=1 << 21), (_lib.E_UNSUPPORTED, "TOO_LARGE")),
    (dict(hidden=1 << 20), (_lib.E_UNSUPPORTED, "TOO_LARGE")), (dict(tokens=1 << 21), (_lib.E_UNSUPPORTED, "TOO_LARGE")),
    (dict(tokens=1 << 20, hidden=1 << 19), (_lib.E_UNSUPPORTED, "TOO_LARGE")),
    (dict(x=None), (_lib.E_UNSUPPORTED, "NULLPTR")), (dict(h=None), (_lib.E_UNSUPPORTED, "NULLPTR")),
    (dict(x=FAKE + 1), (_lib.E_UNSUPPORTED, "ALIGN")), (dict(h=FAKE + 64), (_lib.E_UNSUPPORTED, "OVERLAP")),
    (dict(g=FAKE * 4, u=FAKE * 5), (_lib.E_UNSUPPORTED, "OVERLAP")), (dict(), (_lib.E_UNSUPPORTED, "NOT_DEVICE_PTR")),
    (dict(tokens=0, x=None, h=None), (_lib.OK, "OK")), (dict(hidden=0, x=None, h=None), (_lib.OK, "OK")),
])
def test_ffn_refusals(kw, want):
    reason = ctypes.c_int(-1)
    st = L.ltx3drope_gated_ffn(ffn_call(**kw), None, reason)
    assert (st, _lib.REASONS[reason.value]) == want


def ffn_backward_call(**kw):
    c = dict(dtype=1, activation=0, tokens=4, dim=64, hidden=32, dh=FAKE, x=FAKE * 2, w_gate=FAKE * 3, w_up=FAKE * 4,
             g=FAKE * 5, u=FAKE * 6, dx=FAKE * 7, dw_gate=FAKE * 8, dw_up=FAKE * 9, workspace=FAKE * 10,
             workspace_bytes=1 << 19)
    c.update(kw)
    return _lib.GatedFfnBackward(**c)


@pytest.mark.parametrize("kw,want", [
    (dict(dw_up=None), (_lib.E_INVALID, "OK")), (dict(workspace_bytes=64), (_lib.E_INVALID, "OK")),
    (dict(activation=9), (_lib.E_INVALID, "OK")), (dict(dtype=5), (_lib.E_UNSUPPORTED, "DTYPE")),
    (dict(workspace=None), (_lib.E_UNSUPPORTED, "NULLPTR")), (dict(g=None), (_lib.E_UNSUPPORTED, "NULLPTR")),
    (dict(x=None), (_lib.E_UNSUPPORTED, "NULLPTR")), (dict(w_up=None), (_lib.E_UNSUPPORTED, "NULLPTR")),
    (dict(workspace=FAKE * 10 + 4), (_lib.E_UNSUPPORTED, "ALIGN")), (dict(dx=FAKE), (_lib.E_UNSUPPORTED, "OVERLAP")),
    (dict(dx=None, dw_gate=None, dw_up=None), (_lib.OK, "OK")), (dict(), (_lib.E_UNSUPPORTED, "NOT_DEVICE_PTR")),
])
def test_ffn_backward_refusals(kw, want):
    reason = ctypes.c_int(-1)
    st = L.ltx3drope_gated_ffn_backward(ffn_backward_call(**kw), None, reason)
    assert (st, _lib.REASONS[reason.value]) == want


def test_product_workspace_sizes():
    # few tiles and long sums are split; many tiles, short sums and few tokens are not
    assert L.ltx3drope_gated_ffn_workspace(ffn_call(tokens=16, dim=4096)) == 0
    assert L.ltx3drope_gated_ffn_workspace(ffn_call(tokens=17)) == 0
    assert L.ltx3drope_gated_ffn_workspace(ffn_call(tokens=17, dim=4096)) > 0
    assert L.ltx3drope_gated_ffn_workspace(ffn_call(tokens=8192, dim=4096, hidden=8192)) == 0
    assert L.ltx3drope_gated_ffn_backward_workspace(ffn_backward_call(tokens=0)) == 0
    assert L.ltx3drope_gated_ffn_backward_workspace(ffn_backward_call()) > 0
    assert L.ltx3drope_q8_matmul_workspace(q8_call(tokens=65)) == 0
    assert L.ltx3drope_q8_matmul_workspace(q8_call(tokens=17, dim=4096)) > 0
    for f in (L.ltx3drope_gated_ffn_workspace, L.ltx3drope_gated_ffn_backward_workspace,
              L.ltx3drope_q8_matmul_workspace):
        assert f(None) == _lib.E_INVALID


def q8_call(**kw):
    c = dict(dtype=1, reserved=0, tokens=4, dim=64, out=8, a=FAKE, b=FAKE * 2, a_scale=FAKE * 3, b_scale=FAKE * 4,
             y=FAKE * 5)
    c.update(kw)
    return _lib.Q8Matmul(**c)


@pytest.mark.parametrize("kw,want", [
    (dict(reserved=1), (_lib.E_INVALID, "OK")), (dict(tokens=17, dim=4096), (_lib.E_INVALID, "OK")),
    (dict(dtype=2), (_lib.E_UNSUPPORTED, "DTYPE")), (dict(dim=0), (_lib.E_UNSUPPORTED, "NONPOSITIVE_DIM")),
    (dict(dim=131072), (_lib.E_UNSUPPORTED, "TOO_LARGE")), (dict(out=1 << 26), (_lib.E_UNSUPPORTED, "TOO_LARGE")),
    (dict(tokens=1 << 20, out=1 << 20), (_lib.E_UNSUPPORTED, "TOO_LARGE")),
    (dict(a_scale=None), (_lib.E_UNSUPPORTED, "NULLPTR")), (dict(y=None), (_lib.E_UNSUPPORTED, "NULLPTR")),
    (dict(bias=FAKE * 6 + 2), (_lib.E_UNSUPPORTED, "ALIGN")), (dict(y=FAKE), (_lib.E_UNSUPPORTED, "OVERLAP")),
    (dict(out=0, a=None), (_lib.OK, "OK")), (dict(tokens=0, a=None), (_lib.OK, "OK")),
    (dict(), (_lib.E_UNSUPPORTED, "NOT_DEVICE_PTR")),
])
def test_q8_matmul_refusals(kw, want):
    reason = ctypes.c_int(-1)
    st = L.ltx3drope_q8_matmul(q8_call(**kw), None, reason)
    assert (st, _lib.REASONS[reason.value]) == want


@pytest.mark.parametrize("args,want", [
    ((2, 3, 8, FAKE, FAKE * 2, FAKE * 3), (_lib.E_UNSUPPORTED, "DTYPE")),
    ((0, 3, 0, FAKE, FAKE * 2, FAKE * 3), (_lib.E_UNSUPPORTED, "NONPOSITIVE_DIM")),
    ((0, 1 << 31, 8, FAKE, FAKE * 2, FAKE * 3), (_lib.E_UNSUPPORTED, "TOO_LARGE")),
    ((0, 3, 8, None, FAKE * 2, FAKE * 3), (_lib.E_UNSUPPORTED, "NULLPTR")),
    ((0, 3, 8, FAKE + 2, FAKE * 2, FAKE * 3), (_lib.E_UNSUPPORTED, "ALIGN")),
    ((0, 3, 8, FAKE, FAKE, FAKE * 3), (_lib.E_UNSUPPORTED, "OVERLAP")),
    ((0, 3, 8, FAKE, FAKE * 2, FAKE * 3), (_lib.E_UNSUPPORTED, "NOT_DEVICE_PTR")),
    ((0, 0, 8, None, None, None), (_lib.OK, "OK")),
])
def test_q8_quantize_refusals(args, want):
    reason = ctypes.c_int(-1)
    st = L.ltx3drope_q8_quantize(*args, None, reason)
    assert (st, _lib.REASONS[reason.value]) == want


@pytest.mark.parametrize("call", [
    lambda: rla.gated_ffn(torch.zeros(4, 8), torch.zeros(6, 8), torch.zeros(6, 8)),
    lambda: rla.q8_quantize(torch.zeros(4, 8)),
    lambda: rla.q8_matmul(torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4), torch.zeros(6, 8, dtype=torch.int8),
                          torch.zeros(6)),
    lambda: rla.norm_before(torch.zeros(2, 3, 8)),
    lambda: rla.norm_after(torch.zeros(2, 3, 8), torch.zeros(2, 3, 8)),
    lambda: rla.norm_before_backward(torch.zeros(2, 3, 8), torch.zeros(2, 3, 8)),
])
def test_host_tensors_are_refused(call):
    with pytest.raises(rla.Ltx3dRopeUnsupported) as e:
        call()
    assert e.value.reason == "NOT_DEVICE_PTR"


@pytest.mark.parametrize("tokens", [0, 3, 4032, 1 << 20, 1 << 62])
@pytest.mark.parametrize("hidden", [1 << 61, 1 << 62, (1 << 62) + (1 << 20), (1 << 63) - 32, (1 << 63) - 1])
def test_sizes_whose_products_pass_64_bits_are_refused(tokens, hidden):
    reason = ctypes.c_int(-1)
    for call, size, make in ((L.ltx3drope_gated_ffn, L.ltx3drope_gated_ffn_workspace, ffn_call),
                             (L.ltx3drope_gated_ffn_backward, L.ltx3drope_gated_ffn_backward_workspace,
                              ffn_backward_call)):
        for kw in (dict(tokens=tokens, hidden=hidden), dict(tokens=hidden, dim=hidden)):
            assert call(make(**kw), None, reason) == _lib.E_UNSUPPORTED
            assert _lib.REASONS[reason.value] == "TOO_LARGE"
            assert size(make(**kw)) == _lib.E_UNSUPPORTED
    for kw in (dict(tokens=tokens, out=hidden), dict(tokens=hidden, dim=hidden)):
        assert L.ltx3drope_q8_matmul(q8_call(**kw), None, reason) == _lib.E_UNSUPPORTED
        assert _lib.REASONS[reason.value] == "TOO_LARGE"


def test_widest_8_bit_layers():
    """The last width that is taken passes the checks of sizes; the next one does not."""
    reason = ctypes.c_int(-1)
    for out, tokens, want in (((1 << 26) - 1, 1, "NOT_DEVICE_PTR"), (1 << 26, 1, "TOO_LARGE"),
                              ((1 << 26) - 1, 64, "NOT_DEVICE_PTR"), ((1 << 26) - 1, 256, "TOO_LARGE")):
        far = dict(a=FAKE, a_scale=FAKE * 2, b=FAKE << 8, b_scale=FAKE << 16, y=FAKE << 20)
        assert L.ltx3drope_q8_matmul(q8_call(tokens=tokens, dim=16, out=out, **far), None, reason) == _lib.E_UNSUPPORTED
        assert _lib.REASONS[reason.value] == want, (out, tokens)


@pytest.mark.parametrize("rows,dim", [(1 << 24, 1 << 24), (1 << 18, 1 << 30), (1 << 30, 1 << 18)])
def test_quantiser_of_2_to_the_48_elements_is_refused(rows, dim):
    reason = ctypes.c_int(-1)
    args = (FAKE, 1 << 58, 1 << 60, None, reason)  # apart from each other at any of these sizes
    assert L.ltx3drope_q8_quantize(0, rows, dim, *args) == _lib.E_UNSUPPORTED
    assert _lib.REASONS[reason.value] == "TOO_LARGE"
    assert L.ltx3drope_q8_quantize(0, rows - 1, dim, *args) == _lib.E_UNSUPPORTED
    assert _lib.REASONS[reason.value] == "NOT_DEVICE_PTR"
