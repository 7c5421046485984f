"""Rotary positions with several axes on the GPU against oracle.axes in 64 bits.

Bounds.  The angle is two products in 64 bits, 2^-52 of it, and what is left of it after its whole turns is
exact to 2^-53 of a turn; sine and cosine are within 2e-7 (the reduced angle is rounded to fp32, 4.7e-8 at
pi/4; the Taylor sums leave 2e-9 and their rounding 1.3e-7).  A rotated channel is a sum of two products.
"""
from __future__ import annotations

import math

import pytest
import torch

import oracle.axes as oa
from tests.block_tools import U, assert_within, d, half_step, randn, tiny

pytestmark = pytest.mark.gpu

rla = pytest.importorskip("rope_ltx3drope_amd")
from rope_ltx3drope_amd import _lib  # noqa: E402

DEV = "cuda:0"
TYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(autouse=True)
def fresh():
    assert torch.cuda.is_available()
    _lib.lib()
    rla.stats_reset()
    yield
    torch.cuda.synchronize()


def check(x, got, positions, freq, axis, pairing, inverse, what):
    """x, got [batch, tokens, heads, head_dim]; positions [axes, batch, tokens]."""
    axes = positions.shape[0]
    angle = oa.angles(positions, freq, axis)
    xs = d(x)
    want = oa.rotate(xs, angle, axes, axis, pairing, inverse)
    P = axis.numel()
    # |e| + |o| of each channel's pair, and its angle's own error
    both, slack = torch.zeros_like(xs), torch.zeros_like(xs)
    for i in range(P):
        if int(axis[i]) >= axes:
            continue
        a, b = (2 * i, 2 * i + 1) if pairing == "adjacent" else (i, i + P)
        m = xs[..., a].abs() + xs[..., b].abs()
        both[..., a] = both[..., b] = m
        slack[..., a] = slack[..., b] = m * (2.0 ** -50 * angle[..., i].abs()[..., None])
    tol = both * (2e-7 + 3 * U) + slack
    assert_within(got, want, tol + half_step(x.dtype) * want.abs() + torch.where(both > 0, tiny(x.dtype), 0.0), what)
    # what is not rotated is there bit for bit
    still = torch.ones(x.shape[-1], dtype=torch.bool)
    for i in range(P):
        if int(axis[i]) < axes:
            for c in ((2 * i, 2 * i + 1) if pairing == "adjacent" else (i, i + P)):
                still[c] = False
    bits = torch.int32 if x.dtype is torch.float32 else torch.int16
    assert torch.equal(got.cpu()[..., still].contiguous().view(bits), x.cpu()[..., still].contiguous().view(bits))


def make(B, S, Hq, Hk, D, P, axes, dtype, seed, positions="int", spare=0):
    g = torch.Generator().manual_seed(seed)
    q, k = randn(g, B, S, Hq, D, dtype=dtype), randn(g, B, S, Hk, D, dtype=dtype)
    axis = torch.randint(0, axes, (P,), generator=g).to(torch.uint8)
    if spare:
        axis[::spare] = 255
        axis[1::2 * spare] = axes
    freq = torch.rand(P, generator=g, dtype=torch.float64) ** 3
    if positions == "float":
        pos = torch.rand(axes, B, S, generator=g) * 2 - 1
        freq *= 15000.0
    else:
        pos = torch.randint(-5, 200000, (axes, B, S), generator=g)
    return q, k, pos, freq, axis


def run(q, k, pos, freq, axis, pairing, **kw):
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    args = (dev(pos), dev(freq), dev(axis))
    qo, ko = rla.axes_apply_qk(dev(q), dev(k), *args, pairing=pairing, **kw)
    check(q, qo, pos, freq.double(), axis, pairing, False, "q")
    dq, dk = rla.axes_apply_qk_backward(dev(q), dev(k), *args, pairing=pairing)
    check(q, dq, pos, freq.double(), axis, pairing, True, "dq")
    if k is not None:
        check(k, ko, pos, freq.double(), axis, pairing, False, "k")
        check(k, dk, pos, freq.double(), axis, pairing, True, "dk")
    return qo, ko


PAIRINGS = ["adjacent", "halves"]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pairing", PAIRINGS)
@pytest.mark.parametrize("D,P", [(2, 1), (3, 1), (16, 8), (16, 4), (8, 4), (24, 8), (20, 6), (64, 32), (80, 32), (122, 61),
                                 (128, 64), (128, 60), (256, 128), (96, 16), (250, 100), (512, 256), (520, 260),
                                 (1032, 512), (2050, 1024)])
def test_widths(D, P, pairing, dtype):
    """Head widths and rotated parts around every boundary of the kernels' shapes."""
    run(*make(2, 5, 3, 2, D, P, 3, dtype, D + P, spare=5 if P > 10 else 0), pairing)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pairing", PAIRINGS)
@pytest.mark.parametrize("B,S,Hq,Hk", [(1, 1, 1, 1), (4, 1, 16, 8), (1, 700, 1, 1), (3, 67, 5, 1), (1, 4, 70, 9),
                                       (300, 2, 2, 2), (1, 5000, 2, 1), (1, 9, 300, 1)])
def test_sizes(B, S, Hq, Hk, pairing, dtype):
    """One token, many samples, more tokens than a grid takes at once, one head and hundreds."""
    run(*make(B, S, Hq, Hk, 32, 16, 3, dtype, S + Hq), pairing)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pairing", PAIRINGS)
@pytest.mark.parametrize("B,S,Hq,Hk,D,P,axes", [(1, 16385, 3, 1, 64, 32, 3), (2, 8193, 2, 0, 20, 6, 1), (3, 6001, 1, 1, 16, 4, 30),
                                                (1, 16399, 1, 1, 6, 3, 70), (1, 3001, 1, 1, 1366, 683, 3),
                                                (1, 5003, 1, 0, 400, 150, 2)])
def test_many_tokens_of_few_channels(B, S, Hq, Hk, D, P, axes, pairing, dtype):
    """Tokens enough that a wavefront takes several, the last one fewer."""
    run(*make(B, S, Hq, Hk, D, P, axes, dtype, S), pairing)


@pytest.mark.parametrize("dtype", TYPES)
def test_strides_that_no_index_passes(dtype):
    """One head, one sample, one axis: their strides are any numbers."""
    q, k, pos, freq, axis = make(1, 9, 1, 5, 16, 8, 1, dtype, 1)
    axis[:] = 0
    far = 1 << 61
    wide = q.to(DEV).as_strided(q.shape, (far, 16, far + 1, 1))
    at = pos.to(DEV).as_strided(pos.shape, (far - 1, far, 1))
    got, got_k = rla.axes_apply_qk(wide, k.to(DEV), at, freq.to(DEV), axis.to(DEV))
    check(q, got, pos, freq, axis, "adjacent", False, "q")
    check(k, got_k, pos, freq, axis, "adjacent", False, "k")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("S,Hk", [(5, 70), (20000, 3)])
def test_keys_alone(S, Hk, dtype):
    q, k, pos, freq, axis = make(1, S, 0, Hk, 24, 8, 2, dtype, S)
    q_out, k_out = rla.axes_apply_qk(q.to(DEV), k.to(DEV), pos.to(DEV), freq.to(DEV), axis.to(DEV))
    assert q_out.shape == q.shape
    check(k, k_out, pos, freq, axis, "adjacent", False, "k")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("S", [1, 3, 500])
@pytest.mark.parametrize("D", [16, 4096, 4098, 8192, 1000])
def test_whole_width_as_one_head(D, S, dtype):
    """One head as wide as the model, frequencies over all of it, a few pairs left as they are."""
    q, k, pos, freq, axis = make(1, S, 1, 1, D, D // 2, 3, dtype, D, "float")
    axis[:2] = 255
    run(q, k, pos, freq, axis, "adjacent")


@pytest.mark.parametrize("pairing", PAIRINGS)
@pytest.mark.parametrize("D", [1000, 66000 // 8 * 8 - 464])
def test_long_parts_that_pass_through(D, pairing):
    run(*make(1, 3, 2, 1, D, 8, 2, torch.bfloat16, D), pairing)


@pytest.mark.parametrize("axes", [1, 2, 3, 4, 200, 255])
def test_axes_counts(axes):
    run(*make(2, 6, 2, 2, 128, 64, axes, torch.float32, axes, spare=7), "adjacent")


@pytest.mark.parametrize("ptype", [torch.int64, torch.int32, torch.float32])
@pytest.mark.parametrize("ftype", [torch.float64, torch.float32])
def test_position_and_frequency_types(ptype, ftype):
    q, k, pos, freq, axis = make(2, 9, 2, 1, 64, 32, 3, torch.float32, 3)
    run(q, k, pos.to(ptype), freq.to(ftype), axis, "halves")


def test_far_positions():
    """Positions up to 2^40: the angle's 64 bits still hold it to 2^-50 of itself."""
    q, k, pos, freq, axis = make(1, 64, 1, 1, 32, 16, 2, torch.float32, 4)
    run(q, k, pos * (1 << 22), freq, axis, "adjacent")


def test_every_quarter_and_border():
    """Angles next to every multiple of pi / 4, from both sides, and exactly 0."""
    steps = torch.arange(-40, 41, dtype=torch.float64)
    freq = torch.tensor([math.pi / 4, math.nextafter(math.pi / 4, 0), math.pi / 4 * (1 + 1e-9), 0.0], dtype=torch.float64)
    q = torch.tensor([1.0, 0.0]).repeat(1, 81, 1, 4)
    pos = steps.to(torch.int64).view(1, 1, 81)
    qo, _ = run(q, None, pos, freq, torch.zeros(4, dtype=torch.uint8), "adjacent")
    assert torch.equal(qo[..., 6:].cpu(), q[..., 6:])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pairing", PAIRINGS)
def test_strided_views(pairing, dtype):
    """q and k out of one projection, heads before tokens, positions token by token, outputs of any strides, and in
    place: always the contiguous call's bits."""
    q, k, pos, freq, axis = make(2, 37, 4, 2, 64, 32, 3, dtype, 9)
    how = (freq.to(DEV), axis.to(DEV))
    P = pos.to(DEV)
    want = rla.axes_apply_qk(q.to(DEV), k.to(DEV), P, *how, pairing=pairing)
    check(q, want[0], pos, freq, axis, pairing, False, "q")

    def same(got):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])

    def fused(order):
        shape = (2, 37, 8, 64) if order == "token" else (2, 8, 37, 64)
        buf = torch.full(shape, 3.0, dtype=dtype, device=DEV)
        view = buf if order == "token" else buf.transpose(1, 2)
        vq, vk = view[:, :, :4], view[:, :, 4:6]
        vq.copy_(q)
        vk.copy_(k)
        return buf, view, vq, vk

    for order in ("token", "head"):
        buf, view, vq, vk = fused(order)
        got = rla.axes_apply_qk(vq, vk, P, *how, pairing=pairing)
        assert got[0].is_contiguous() and got[1].is_contiguous()
        same(got)
        got = rla.axes_apply_qk(vq, vk, P, *how, pairing=pairing, inplace=True)
        assert got[0].data_ptr() == vq.data_ptr()
        same(got)
        assert bool((view[:, :, 6:] == 3.0).all())  # the values beside them
    # positions as [batch, tokens, axes]
    same(rla.axes_apply_qk(q.to(DEV), k.to(DEV), P.permute(1, 2, 0).contiguous().permute(2, 0, 1), *how, pairing=pairing))
    # an odd offset and odd strides: no 16-byte vector
    odd = torch.zeros(2, 37, 4, 67, dtype=dtype, device=DEV)[..., 1:65]
    odd.copy_(q)
    out = torch.full((2, 37, 4, 69), 7.0, dtype=dtype, device=DEV)
    got = rla.axes_apply_qk(odd, k.to(DEV), P, *how, pairing=pairing, q_out=out[..., 3:67])
    check(q, got[0], pos, freq, axis, pairing, False, "q of odd strides")
    assert bool((out[..., :3] == 7).all()) and bool((out[..., 67:] == 7).all())
    # one sample's positions for all
    one = rla.axes_apply_qk(q.to(DEV), k.to(DEV), P[:, 0].contiguous(), *how, pairing=pairing)
    both = rla.axes_apply_qk(q.to(DEV), k.to(DEV), P[:, :1].expand(3, 2, 37), *how, pairing=pairing)
    assert torch.equal(one[0], both[0]) and torch.equal(one[1], both[1])
    # without a batch
    flat = rla.axes_apply_qk(q[0].to(DEV), k[0].to(DEV), P[:, 0], *how, pairing=pairing)
    assert torch.equal(flat[0], want[0][0]) and torch.equal(flat[1], want[1][0])
    # q alone
    alone, nothing = rla.axes_apply_qk(q.to(DEV), None, P, *how, pairing=pairing)
    assert nothing is None and torch.equal(alone, want[0])
    # broadcast inputs
    wide = q[:, :, :1].to(DEV).expand(2, 37, 4, 64)
    got = rla.axes_apply_qk(wide, k.to(DEV), P, *how, pairing=pairing)
    assert torch.equal(got[0][:, :, 3], want[0][:, :, 0])


def test_the_grid_kernels_rotation():
    """Integer positions on a (T, H, W) grid with the tables' frequencies: the values of apply_qk to within both bounds."""
    split, grid = (8, 12, 12), (3, 5, 7)
    g = torch.Generator().manual_seed(2)
    q, k = (randn(g, 2, *grid, 3, 32).to(DEV) for _ in range(2))
    want = rla.forward_pair(q, k, split)
    f, a = rla.axes_frequencies(split, device=DEV)
    pos = torch.stack(torch.meshgrid(*[torch.arange(n) for n in grid], indexing="ij")).view(3, -1).to(DEV)
    got = rla.axes_apply_qk(q.view(2, 105, 3, 32), k.view(2, 105, 3, 32), pos, f, a)
    for x, y, z in zip(got, want, (q, k)):
        size = d(z).view(2, 105, 3, 16, 2).abs().sum(-1, keepdim=True).expand(-1, -1, -1, -1, 2).reshape(2, 105, 3, 32)
        assert_within(x, d(y).view(2, 105, 3, 32), size * (2e-7 + 8 * U) + tiny(torch.float32), "against apply_qk")


def test_rotate_half_with_one_axis():
    """One axis in halves with the frequencies of a cos/sin cache: neox_apply_qk's values, whose every product is
    rounded to fp32."""
    g = torch.Generator().manual_seed(6)
    q, k = randn(g, 50, 4, 64).to(DEV), randn(g, 50, 2, 64).to(DEV)
    f, a = rla.axes_frequencies((64,), device=DEV)
    pos = torch.randint(0, 4096, (50,), generator=g).to(DEV)
    angle = torch.arange(4096, dtype=torch.float64)[:, None] * f.cpu()
    cache = torch.cat([angle.cos(), angle.sin()], 1).float().to(DEV)
    want = rla.neox_apply_qk(q, k, pos, cache)
    got = rla.axes_apply_qk(q, k, pos[None], f, a, pairing="halves")
    for x, y, z in zip(got, want, (q, k)):
        size = (d(z)[..., :32].abs() + d(z)[..., 32:].abs()).repeat(1, 1, 2)
        assert_within(x, d(y), size * (2e-7 + 8 * U) + tiny(torch.float32), "against neox_apply_qk")


def test_the_frequency_grid():
    """dit_freq_grid's frequencies for three axes in turn over a whole width, with fractional positions."""
    n = 341
    grid = rla.dit_freq_grid(10000.0, 6 * n, 6, True, device=DEV)
    freq = torch.cat([torch.zeros(1, device=DEV), grid.repeat_interleave(3)])
    axis = torch.tensor([255] + [0, 1, 2] * n, dtype=torch.uint8)
    g = torch.Generator().manual_seed(7)
    q, pos = randn(g, 1, 21, 1, 2 * (3 * n + 1), dtype=torch.bfloat16), torch.rand(3, 1, 21, generator=g) * 2 - 1
    run(q, q, pos, freq.cpu(), axis, "adjacent")


def test_special_values_stay_in_their_pair():
    """Infinities and NaN reach their own pair only, and not what passes through."""
    for dtype in TYPES:
        for pairing in PAIRINGS:
            for D in (32, 34):  # vectors, and single elements
                q, _, pos, freq, axis = make(1, 6, 2, 1, D, 12, 2, dtype, D)
                axis[3] = 255
                how = (pos.to(DEV), freq.to(DEV), axis.to(DEV))
                clean = rla.axes_apply_qk(q.to(DEV), None, *how, pairing=pairing)[0].cpu()
                a, b = (6, 7) if pairing == "adjacent" else (3, 15)  # pair 3, left as it is
                c, e = (10, 11) if pairing == "adjacent" else (5, 17)
                q[0, 2, 1, a], q[0, 2, 1, b], q[0, 2, 1, D - 1] = float("inf"), float("nan"), float("-inf")
                q[0, 4, 0, c] = float("nan")
                got = rla.axes_apply_qk(q.to(DEV), None, *how, pairing=pairing)[0].cpu()
                assert got[0, 2, 1, a] == float("inf") and torch.isnan(got[0, 2, 1, b])
                assert got[0, 2, 1, D - 1] == float("-inf")
                assert torch.isnan(got[0, 4, 0, c]) and torch.isnan(got[0, 4, 0, e])
                touched = torch.zeros(q.shape, dtype=torch.bool)
                touched[0, 2, 1, [a, b, D - 1]] = True
                touched[0, 4, 0, [c, e]] = True
                assert torch.equal(got[~touched], clean[~touched])


def test_positions_that_are_not_finite():
    """An infinite or undefined position gives NaN to its own token and axis only."""
    q, _, pos, freq, axis = make(1, 4, 2, 1, 32, 16, 2, torch.float32, 8, "float")
    how = (freq.to(DEV), axis.to(DEV))
    clean = rla.axes_apply_qk(q.to(DEV), None, pos.to(DEV), *how)[0].cpu()
    pos[0, 0, 1], pos[1, 0, 3] = float("inf"), float("nan")
    got = rla.axes_apply_qk(q.to(DEV), None, pos.to(DEV), *how)[0].cpu()
    on = axis.repeat_interleave(2).long()
    assert torch.equal(got[0, [0, 2]], clean[0, [0, 2]])
    assert torch.isnan(got[0, 1][:, on == 0]).all() and torch.equal(got[0, 1][:, on == 1], clean[0, 1][:, on == 1])
    assert torch.isnan(got[0, 3][:, on == 1]).all() and torch.equal(got[0, 3][:, on == 0], clean[0, 3][:, on == 0])


def test_gradient_against_differences():
    """The map is linear: its difference along a direction is the map of that direction, and the backward its
    transpose, <dy, R v> = <R^T dy, v>."""
    q, k, pos, freq, axis = make(2, 5, 3, 2, 40, 16, 3, torch.float32, 11)
    how = (pos.to(DEV), freq.to(DEV), axis.to(DEV))
    g = torch.Generator().manual_seed(1)
    v, dy = randn(g, *q.shape), randn(g, *q.shape)
    f = lambda x: d(rla.axes_apply_qk(x.to(DEV), k.to(DEV), *how)[0])  # noqa: E731
    slope = ((f(q + 2 ** -6 * v) - f(q - 2 ** -6 * v)) * 2.0 ** 5 * d(dy)).sum()
    back = d(rla.axes_apply_qk_backward(dy.to(DEV), k.to(DEV), *how)[0])
    # each of the 1200 terms carries about four roundings of values near 3, over 2^-5
    assert abs(float(slope) - float((back * d(v)).sum())) <= 4 * 4 * 3 * U * 2 ** 5 * 1200 ** 0.5 * 3


def test_other_stream_and_graph():
    q, k, pos, freq, axis = make(2, 40, 4, 2, 64, 32, 3, torch.bfloat16, 12)
    q, k, pos, freq, axis = (t.to(DEV) for t in (q, k, pos, freq, axis))

    def step(**kw):
        a = rla.axes_apply_qk(q, k, pos, freq, axis, **kw)
        return a + rla.axes_apply_qk_backward(*a, pos, freq, axis, **kw)

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(4):
        gen = torch.Generator().manual_seed(100 + i)
        q.copy_(randn(gen, *q.shape))
        k.copy_(randn(gen, *k.shape))
        pos.copy_(torch.randint(0, 5000, pos.shape, generator=gen))
        eager = step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, outs)), i


def test_refusals_on_the_device():
    q, k, pos, freq, axis = (t.to(DEV) for t in make(2, 5, 3, 2, 16, 8, 3, torch.float32, 1))

    def refused(why, *args, **kw):
        with pytest.raises(rla.Ltx3dRopeUnsupported) as e:
            rla.axes_apply_qk(*args, **kw)
        assert e.value.reason == why, e.value.reason

    refused("SHAPE_MISMATCH", q, k[:, :4], pos, freq, axis)
    refused("SHAPE_MISMATCH", q, k[..., :8], pos, freq, axis)
    refused("SHAPE_MISMATCH", q, k, pos[:, :1], freq, axis)
    refused("SHAPE_MISMATCH", q, k, pos, freq[:4], axis)
    refused("DTYPE", q, k.bfloat16(), pos, freq, axis)
    refused("DTYPE", q.half(), k.half(), pos, freq, axis)
    refused("DTYPE", q, k, pos.double(), freq, axis)
    refused("DTYPE", q, k, pos, freq, axis.long())
    refused("NOT_DEVICE_PTR", q, k, pos.cpu(), freq, axis)
    refused("NOT_CONTIGUOUS", q.transpose(2, 3).contiguous().transpose(2, 3), k, pos, freq, axis)
    refused("NOT_CONTIGUOUS", q, k, pos, torch.ones(16, dtype=torch.float64, device=DEV)[::2], axis)
    refused("SPLIT_SUM", q[..., :8], k[..., :8], pos, freq, axis)
    refused("OUTPUT_MISMATCH", q, k, pos, freq, axis, q_out=k)
    refused("OVERLAP", q, k, pos, freq, axis, q_out=torch.zeros(1, 5, 3, 16, device=DEV).expand(2, 5, 3, 16))
    refused("OVERLAP", q, q, pos, freq, axis, inplace=True)
    assert rla.stats()["fast_launches"] == 0
    with pytest.raises(ValueError):
        rla.axes_apply_qk(q, k, pos, freq, axis, inplace=True, q_out=torch.empty_like(q))


def test_empty_calls():
    q, k, pos, freq, axis = (t.to(DEV) for t in make(2, 5, 3, 2, 16, 8, 3, torch.float32, 1))
    a, b = rla.axes_apply_qk(q[:, :0], k[:, :0], pos[:, :, :0], freq, axis)
    assert a.shape == (2, 0, 3, 16) and b.shape == (2, 0, 2, 16)
    a, b = rla.axes_apply_qk(q[:, :, :0], k, pos, freq, axis)
    assert a.numel() == 0 and torch.equal(b, rla.axes_apply_qk(k, None, pos, freq, axis)[0])


@pytest.mark.parametrize("pairing", PAIRINGS)
def test_more_than_two_to_the_32_elements(pairing):
    """Offsets that pass 32 bits: the last tokens of 2^20 + 77 against the same tokens alone."""
    S, H, D = (1 << 20) + 77, 33, 128
    q = torch.empty(1, S, H, D, dtype=torch.bfloat16, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(2)
    tail = torch.randn(90, H, D, generator=gen, device=DEV).bfloat16()
    q[0, :-90] = 1.0
    q[0, -90:] = tail
    pos = torch.arange(S, device=DEV).repeat(3, 1)
    f, a = rla.axes_frequencies((32, 48, 48), device=DEV)
    out, _ = rla.axes_apply_qk(q, None, pos, f, a, pairing=pairing)
    assert torch.equal(out[0, -90:], rla.axes_apply_qk(tail, None, pos[:, -90:], f, a, pairing=pairing)[0])
    mid = rla.axes_apply_qk(q[0, 700000:700050], None, pos[:, 700000:700050], f, a, pairing=pairing)[0]
    assert torch.equal(out[0, 700000:700050], mid)
    del out
    rla.axes_apply_qk(q, None, pos, f, a, pairing=pairing, inplace=True)
    assert torch.equal(q[0, 700000:700050], mid)
