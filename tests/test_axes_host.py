"""CPU tests of the rotary positions with several axes: the oracle against the complex form and against
differences, the frequencies, and the C ABI's refusals, which come before anything touches a GPU."""
from __future__ import annotations

import ctypes
import itertools
import os
import random

import pytest
import torch

import oracle.axes as oa

rla = pytest.importorskip("rope_ltx3drope_amd")
from rope_ltx3drope_amd import _lib  # noqa: E402

if not os.path.exists(_lib.LIB_PATH):
    pytest.skip("libltx3drope.so not built (python -m rope_ltx3drope_amd.build)", allow_module_level=True)

L = _lib.lib()
FAKE = 1 << 24  # an aligned address that no rule below dereferences


@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
def test_oracle_against_the_complex_form(pairing):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(2, 3, 2, 14, generator=g, dtype=torch.float64)
    pos = torch.randint(0, 1000, (3, 2, 3), generator=g)
    f, axis = oa.frequencies([4, 2, 6], 100.0, False)
    f, axis = torch.tensor(f, dtype=torch.float64), torch.tensor(axis)
    angle = oa.angles(pos, f, axis)
    got = oa.rotate(x, angle, 3, axis, pairing)
    turn = torch.exp(1j * angle)[:, :, None, :]
    if pairing == "adjacent":
        z = torch.complex(x[..., 0:12:2], x[..., 1:12:2]) * turn
        want = torch.stack([z.real, z.imag], -1).flatten(-2)
    else:
        z = torch.complex(x[..., :6], x[..., 6:12]) * turn
        want = torch.cat([z.real, z.imag], -1)
    assert torch.allclose(got[..., :12], want, rtol=0, atol=1e-13)
    assert torch.equal(got[..., 12:], x[..., 12:])
    # the inverse rotation is the gradient: for a linear map <dy, R x> = <R^T dy, x>, and R^T undoes R
    dy = torch.randn(x.shape, generator=g, dtype=torch.float64)
    back = oa.rotate(dy, angle, 3, axis, pairing, inverse=True)
    assert abs(float((dy * got).sum() - (back * x).sum())) < 1e-11
    assert torch.allclose(oa.rotate(got, angle, 3, axis, pairing, inverse=True), x, rtol=0, atol=1e-13)
    # a pair without an axis stays
    part = torch.where(torch.arange(6) % 2 == 0, axis, torch.tensor(255))
    got = oa.rotate(x, oa.angles(pos, f, part), 3, part, pairing)
    for i in (1, 3, 5):
        for c in ((2 * i, 2 * i + 1) if pairing == "adjacent" else (i, i + 6)):
            assert torch.equal(got[..., c], x[..., c])


@pytest.mark.parametrize("joint", [False, True])
@pytest.mark.parametrize("widths,base", [((32, 48, 48), 10000.0), ((2,), 1e6), ((16, 24), 500.0), ((2, 4, 6, 8), 3.5)])
def test_frequencies(widths, base, joint):
    n = sum(widths) // 2
    f, a = (ctypes.c_double * n)(), (ctypes.c_uint8 * n)()
    assert L.ltx3drope_axes_frequencies(len(widths), (_lib.i64 * len(widths))(*widths), base, int(joint), f, a) == 0
    want, axis = oa.frequencies(widths, base, joint)
    assert list(a) == axis
    for x, y in zip(f, want):
        assert abs(x - y) <= 2.0 ** -51 * y  # two correctly used powers, each within an ulp


@pytest.mark.parametrize("axes,widths,base,joint", [(0, (2,), 10.0, 0), (256, (2,) * 256, 10.0, 0), (1, (3,), 10.0, 0),
                                                    (2, (2, 0), 10.0, 0), (1, (65538,), 10.0, 0), (1, (2,), 0.0, 0),
                                                    (1, (2,), float("nan"), 0), (1, (2,), 10.0, 2)])
def test_frequencies_invalid(axes, widths, base, joint):
    n = 65538
    f, a = (ctypes.c_double * n)(), (ctypes.c_uint8 * n)()
    assert L.ltx3drope_axes_frequencies(axes, (_lib.i64 * len(widths))(*widths), base, joint, f, a) == _lib.E_INVALID
    assert L.ltx3drope_axes_frequencies(1, (_lib.i64 * 1)(2), 10.0, 0, None, a) == _lib.E_INVALID


def call(**kw):
    B, S, Hq, Hk, D = 2, 3, 4, 2, 16
    c = dict(dtype=0, pairing=0, inverse=0, position_type=0, frequency_type=0, axes=3, batch=B, tokens=S, q_heads=Hq,
             k_heads=Hk, head_dim=D, pairs=8, q_strides=(S * Hq * D, Hq * D, D), k_strides=(S * Hk * D, Hk * D, D),
             q_out_strides=(S * Hq * D, Hq * D, D), k_out_strides=(S * Hk * D, Hk * D, D),
             position_strides=(B * S, S, 1), q=FAKE, k=FAKE * 2, q_out=FAKE * 3, k_out=FAKE * 4, positions=FAKE * 5,
             frequencies=FAKE * 6, axis=FAKE * 7)
    c.update(kw)
    for n in ("q_strides", "k_strides", "q_out_strides", "k_out_strides", "position_strides"):
        c[n] = (_lib.i64 * 3)(*c[n])
    return _lib.Axes(**c)


def status(**kw):
    reason = ctypes.c_int(-1)
    return L.ltx3drope_axes_apply(call(**kw), None, reason), _lib.REASONS[reason.value]


@pytest.mark.parametrize("kw", [dict(pairing=2), dict(inverse=-1), dict(position_type=3), dict(frequency_type=2),
                                dict(axes=0), dict(axes=256), dict(q_strides=(-1, 64, 16)),
                                dict(position_strides=(6, 3, -1)), dict(k_heads=0)])
def test_invalid(kw):
    assert status(**kw)[0] == _lib.E_INVALID
    assert L.ltx3drope_axes_apply(None, None, None) == _lib.E_INVALID


@pytest.mark.parametrize("kw,reason", [
    (dict(dtype=2), "DTYPE"), (dict(head_dim=0), "NONPOSITIVE_DIM"), (dict(pairs=0), "NONPOSITIVE_DIM"),
    (dict(tokens=-1), "NONPOSITIVE_DIM"), (dict(pairs=9), "SPLIT_SUM"), (dict(head_dim=15), "SPLIT_SUM"),
    (dict(batch=65536), "TOO_LARGE"), (dict(tokens=1 << 31), "TOO_LARGE"), (dict(q_heads=65537), "TOO_LARGE"),
    (dict(head_dim=65537), "TOO_LARGE"), (dict(q_strides=(1 << 62, 64, 16)), "TOO_LARGE"),
    (dict(q_strides=(1 << 58, 1 << 57, 16)), "TOO_LARGE"), (dict(position_strides=(1 << 60, 1, 1)), "TOO_LARGE"),
    (dict(q=None), "NULLPTR"), (dict(q_out=None), "NULLPTR"), (dict(k=None), "NULLPTR"), (dict(k_out=None), "NULLPTR"),
    (dict(positions=None), "NULLPTR"), (dict(frequencies=None), "NULLPTR"), (dict(axis=None), "NULLPTR"),
    (dict(q=FAKE + 2), "ALIGN"), (dict(positions=FAKE * 5 + 4), "ALIGN"), (dict(frequencies=FAKE * 6 + 4), "ALIGN"),
    (dict(q_out=FAKE + 4), "OVERLAP"), (dict(k_out=FAKE * 3), "OVERLAP"), (dict(q_out=FAKE * 2), "OVERLAP"),
    (dict(q_out=FAKE * 5), "OVERLAP"), (dict(k_out=FAKE * 7), "OVERLAP"), (dict(k_out=FAKE), "OVERLAP"),
    (dict(q_out_strides=(192, 64, 15)), "OVERLAP"), (dict(q_out_strides=(0, 64, 16)), "OVERLAP"),
    (dict(q_out_strides=(192, 32, 16)), "OVERLAP"),
    # the same address with other strides is not the input itself
    (dict(q_out=FAKE, q_out_strides=(48, 16, 96)), "OVERLAP"),
    (dict(), "NOT_DEVICE_PTR"), (dict(q_out=FAKE, k_out=FAKE * 2), "NOT_DEVICE_PTR"),
    (dict(k=None, k_out=None, k_heads=0), "NOT_DEVICE_PTR"), (dict(q_strides=(0, 0, 0)), "NOT_DEVICE_PTR"),
    (dict(position_type=1, positions=FAKE * 5 + 4), "NOT_DEVICE_PTR"),
    (dict(frequency_type=1, frequencies=FAKE * 6 + 4), "NOT_DEVICE_PTR"),
])
def test_refusals(kw, reason):
    assert status(**kw) == (_lib.E_UNSUPPORTED, reason)


def fused(order, heads=(4, 2, 2), **kw):
    """q and k as views of one projection of q, k and v heads, in place."""
    H, S, B, D, es = sum(heads), 3, 2, 16, 4
    if order == "token":  # [B, S, H, D]
        strides, step = (S * H * D, H * D, D), D
    else:  # [B, H, S, D]
        strides, step = (H * S * D, D, S * D), S * D
    k = FAKE + heads[0] * step * es
    return dict(q=FAKE, q_out=FAKE, k=k, k_out=k, q_strides=strides, k_strides=strides, q_out_strides=strides,
                k_out_strides=strides, **kw)


@pytest.mark.parametrize("order", ["token", "head"])
def test_views_of_one_projection_in_place(order):
    assert status(**fused(order))[1] == "NOT_DEVICE_PTR"
    assert status(**fused(order, tokens=1))[1] == "NOT_DEVICE_PTR"
    assert status(**fused(order, batch=1))[1] == "NOT_DEVICE_PTR"
    # one head short: k's first head is q's last
    c = fused(order)
    step = (16 if order == "token" else 48) * 4
    assert status(**dict(c, k=c["k"] - step, k_out=c["k"] - step))[1] == "OVERLAP"
    # one head too far: k's last head is the next row's q
    last = fused(order, heads=(4, 2, 0))
    assert status(**last)[1] == "NOT_DEVICE_PTR"
    assert status(**dict(last, k=last["k"] + step, k_out=last["k"] + step))[1] == ("OVERLAP")


def elements(p, strides, sizes, width, es):
    return [p + es * (sum(i * s for i, s in zip(at, strides)) + c)
            for at in itertools.product(*[range(n) for n in sizes]) for c in range(width)]


def test_no_shared_element_is_let_through():
    """Random small strides and addresses: whatever shares an element of an output is refused."""
    rng = random.Random(5)
    seen = {"OVERLAP": 0, "NOT_DEVICE_PTR": 0}
    for _ in range(4000):
        B, S, Hq, Hk, D, es = rng.randint(1, 2), rng.randint(1, 3), rng.randint(1, 3), rng.randint(1, 2), 2, 4
        def strides():
            return tuple(rng.choice([0, 1, 2, 4, 6, 8, 10, 12, 16, 24, 32, 36]) for _ in range(3))
        sq, sk = strides(), strides()
        share = rng.random() < 0.6
        so, sko = (sq, sq if share else sk) if rng.random() < 0.7 else (strides(), strides())
        if share:
            sk = sq
        q = FAKE
        k = q + es * rng.randint(0, 60)
        qo = q if rng.random() < 0.5 else q + es * rng.randint(0, 80)
        ko = k if rng.random() < 0.5 else q + es * rng.randint(0, 80)
        st = status(batch=B, tokens=S, q_heads=Hq, k_heads=Hk, head_dim=D, pairs=1, q=q, k=k, q_out=qo, k_out=ko,
                    q_strides=sq, k_strides=sk, q_out_strides=so, k_out_strides=sko)[1]
        seen[st] += 1
        if st == "OVERLAP":
            continue
        qe, ke = (elements(p, s, (B, S, h), D, es) for p, s, h in ((q, sq, Hq), (k, sk, Hk)))
        qoe, koe = (elements(p, s, (B, S, h), D, es) for p, s, h in ((qo, so, Hq), (ko, sko, Hk)))
        assert len(set(qoe)) == len(qoe) and len(set(koe)) == len(koe)
        assert not set(qoe) & set(koe)
        assert not set(qoe) & set(ke) and not set(koe) & set(qe)
        assert not set(qoe) & set(qe) or qoe == qe
        assert not set(koe) & set(ke) or koe == ke
    assert min(seen.values()) > 100, seen


def test_empty_calls_look_at_no_pointer():
    none = dict(q=None, k=None, q_out=None, k_out=None, positions=None, frequencies=None, axis=None)
    for kw in (dict(batch=0), dict(tokens=0), dict(q_heads=0, k_heads=0)):
        assert status(**none, **kw) == (_lib.OK, "OK")


def test_descriptor_as_bytes():
    values = list(range(1, 35))
    raw = _lib.AXES_BYTES.pack(*values)
    s = _lib.Axes.from_buffer_copy(raw)
    assert len(raw) == ctypes.sizeof(_lib.Axes)
    flat = []
    for n, _ in _lib.Axes._fields_:
        v = getattr(s, n)
        flat += list(v) if hasattr(v, "__len__") else [v]
    assert flat == values


def test_binding_refuses_before_the_gpu():
    q = torch.zeros(4, 2, 8)
    f, a, pos = torch.ones(4, dtype=torch.float64), torch.zeros(4, dtype=torch.uint8), torch.zeros(1, 4, dtype=torch.int64)

    def reason(*args, **kw):
        with pytest.raises(rla.Ltx3dRopeUnsupported) as e:
            rla.axes_apply_qk(*args, **kw)
        return e.value.reason

    assert reason(q, q, pos, f, a) == "NOT_DEVICE_PTR"
    assert reason(q[0], None, pos, f, a) == "SHAPE_MISMATCH"
    with pytest.raises(ValueError):
        rla.axes_apply_qk(q, q, pos, f, a, pairing="neighbours")
    with pytest.raises(ValueError):
        rla.axes_apply_qk(q, None, pos, f, a, k_out=q)
