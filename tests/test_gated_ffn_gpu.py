"""The gated feed-forward block on the GPU, forward and backward, against oracle.block in 64 bits.

Bounds.  A sum of K products on the matrix cores is off by at most a step of fp32 (2 u) of the running
sum an addition: (K + 2) * 2 u * sum |terms|.  The activations go through the hardware's exponential
and reciprocal: their logistic function of z is within (|z| + 8) u, relative; gelu's erf within 8 u.
What the backward pass keeps between its products (dg, du) is rounded once to the rows' type.
"""
from __future__ import annotations

import math

import pytest
import torch

import oracle.block as ob
from tests.block_tools import U, assert_within, d, half_step, randn, tiny

pytestmark = pytest.mark.gpu

rla = pytest.importorskip("rope_ltx3drope_amd")
from rope_ltx3drope_amd import _lib  # noqa: E402

DEV = "cuda:0"
KINDS = ["silu", "gelu", "gelu_tanh"]
TYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(autouse=True)
def fresh():
    assert torch.cuda.is_available()
    _lib.lib()
    rla.stats_reset()
    yield
    torch.cuda.synchronize()


def inputs(M, D, F, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return dict(x=randn(g, M, D, dtype=dtype), w_gate=randn(g, F, D, std=2.0 / math.sqrt(D), dtype=dtype),
                w_up=randn(g, F, D, std=1.0 / math.sqrt(D), dtype=dtype), dh=randn(g, M, F, dtype=dtype))


def z_bound(g):
    """The larger of the logistic functions' arguments, and the factor on its slope."""
    return 1.6 * g.abs() + 0.0715 * g.abs() ** 3, 1.6 * (1.0 + 0.135 * g * g)


def check_forward(t, kind, h, g=None, u=None):
    x, wg, wu = d(t["x"]), d(t["w_gate"]), d(t["w_up"])
    hs, D = half_step(t["x"].dtype), x.shape[1]
    want, wantg, wantu = ob.gated_ffn(x, wg, wu, kind)
    g_tol = (D + 2) * 2 * U * (x.abs() @ wg.abs().T)
    u_tol = (D + 2) * 2 * U * (x.abs() @ wu.abs().T)
    z, _ = z_bound(wantg)
    a = ob.act(wantg, kind).abs()
    a_tol = 1.2 * g_tol + (z + 8) * U * a + 8 * U * wantg.abs()
    tol = a_tol * (wantu.abs() + u_tol) + a * u_tol + 2 * U * want.abs()
    assert_within(h, want, tol + hs * (want.abs() + tol) + tiny(t["x"].dtype), "h")
    if g is not None:
        assert g.dtype == torch.float32 and u.dtype == torch.float32
        assert_within(g, wantg, g_tol, "g")
        assert_within(u, wantu, u_tol, "u")


def check_backward(t, kind, g, u, dx, dwg, dwu):
    x, wg, wu, dh, g, u = (d(v) for v in (t["x"], t["w_gate"], t["w_up"], t["dh"], g, u))
    dt = t["x"].dtype
    hs, (M, D), F = half_step(dt), x.shape, wg.shape[0]
    want_dx, want_dwg, want_dwu = ob.gated_ffn_backward(dh, x, wg, wu, g, u, kind)
    z, slope_factor = z_bound(g)
    dg, du = dh * u * ob.act_slope(g, kind), dh * ob.act(g, kind)
    slope_tol = (z + 16) * U * (1 + 2 * g.abs() * slope_factor)
    dg_tol = (dh * u).abs() * slope_tol + (hs + 4 * U) * dg.abs() + tiny(dt)
    du_tol = dh.abs() * ((z + 8) * U * ob.act(g, kind).abs() + 8 * U * g.abs()) + (hs + 4 * U) * du.abs() + tiny(dt)
    dga, dua = dg.abs() + dg_tol, du.abs() + du_tol
    if dx is not None:
        tol = dg_tol @ wg.abs() + du_tol @ wu.abs() + (2 * F + 2) * 2 * U * (dga @ wg.abs() + dua @ wu.abs())
        assert_within(dx, want_dx, tol + hs * (want_dx.abs() + tol) + tiny(dt), "dx")
    if dwg is not None:
        for got, want, tol0, mag, name in ((dwg, want_dwg, dg_tol, dga, "dw_gate"), (dwu, want_dwu, du_tol, dua, "dw_up")):
            tol = tol0.T @ x.abs() + (M + 2) * 2 * U * (mag.T @ x.abs())
            assert_within(got, want, tol + hs * (want.abs() + tol) + tiny(dt), name)


def run(M, D, F, dtype, kind, seed):
    t = inputs(M, D, F, dtype, seed)
    dev = {k: v.to(DEV) for k, v in t.items()}
    h, g, u = rla.gated_ffn(dev["x"], dev["w_gate"], dev["w_up"], kind, save=True)
    check_forward(t, kind, h, g, u)
    assert torch.equal(h, rla.gated_ffn(dev["x"], dev["w_gate"], dev["w_up"], kind))
    grads = rla.gated_ffn_backward(dev["dh"], dev["x"], dev["w_gate"], dev["w_up"], g, u, kind)
    check_backward(t, kind, g, u, *grads)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 33, 64, 65, 100, 127, 128, 129, 257, 300])
def test_token_counts(M, dtype):
    run(M, 136, 200, dtype, KINDS[M % 3], M)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [1, 3, 7, 11, 77])
@pytest.mark.parametrize("D", [1, 3, 7, 8, 24, 31, 63, 64, 65, 100, 129, 200, 520, 1032])
def test_widths(D, M, dtype):
    run(M, D, 48, dtype, KINDS[D % 3], 100 + D)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [1, 4, 5, 140])
@pytest.mark.parametrize("F", [1, 2, 3, 5, 15, 16, 17, 63, 64, 66, 100, 127, 128, 130, 257])
def test_hidden_widths(F, M, dtype):
    run(M, 72, F, dtype, KINDS[F % 3], 200 + F)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,D,F", [(2048, 128, 3200), (2047, 72, 3201), (2300, 2304, 1152), (300, 2056, 700),
                                   (1025, 4096, 64), (1, 8200, 30), (3, 4104, 257), (12, 5000, 33), (70, 8200, 20), (1700, 640, 65), (90, 1025, 1700)])
def test_large_tiles(M, D, F, dtype):
    """Enough tiles for the large ones; long sums; odd edges of both."""
    run(M, D, F, dtype, "silu", 300 + M)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", KINDS)
def test_activations_over_their_range(kind, dtype):
    """Projections from -40 to 40 through an identity-like weight: the activations' tails, both directions."""
    F = 256
    values = torch.linspace(-40, 40, 64 * 70).reshape(70, 64).to(dtype)
    t = dict(x=values, w_gate=torch.zeros(F, 64, dtype=dtype), w_up=torch.zeros(F, 64, dtype=dtype))
    for i in range(64):
        t["w_gate"][i, i] = 1
        t["w_up"][i, 63 - i] = 1
    t["dh"] = randn(torch.Generator().manual_seed(1), 70, F, dtype=dtype)
    dev = {k: v.to(DEV) for k, v in t.items()}
    h, g, u = rla.gated_ffn(dev["x"], dev["w_gate"], dev["w_up"], kind, save=True)
    assert torch.equal(g[:, :64].cpu(), values.float())
    check_forward(t, kind, h, g, u)
    check_backward(t, kind, g, u, *rla.gated_ffn_backward(dev["dh"], dev["x"], dev["w_gate"], dev["w_up"], g, u, kind))


@pytest.mark.parametrize("dtype", TYPES)
def test_unaligned_tensors(dtype):
    """Tensors that start one element past a 16-byte boundary."""
    for M in (1, 4, 10, 100):
        t = inputs(M, 64, 80, dtype, 9)

        def shifted(v):
            b = torch.empty(v.numel() + 1, dtype=v.dtype, device=DEV)[1:].view(v.shape)
            b.copy_(v)
            return b

        dev = {k: shifted(v) for k, v in t.items()}
        h, g, u = rla.gated_ffn(dev["x"], dev["w_gate"], dev["w_up"], "gelu", save=True)
        check_forward(t, "gelu", h, g, u)
        check_backward(t, "gelu", g, u, *rla.gated_ffn_backward(dev["dh"], dev["x"], dev["w_gate"], dev["w_up"],
                                                                shifted(g), shifted(u), "gelu"))


def test_leading_dimensions_and_parts_left_out():
    t = inputs(12, 64, 96, torch.bfloat16, 2)
    dev = {k: v.to(DEV) for k, v in t.items()}
    h, g, u = rla.gated_ffn(dev["x"].view(3, 4, 64), dev["w_gate"], dev["w_up"], save=True)
    assert h.shape == (3, 4, 96)
    check_forward(t, "silu", h.view(12, 96))
    args = (dev["dh"].view(3, 4, 96), dev["x"].view(3, 4, 64), dev["w_gate"], dev["w_up"], g, u)
    dx, dwg, dwu = rla.gated_ffn_backward(*args)
    a = rla.gated_ffn_backward(*args, need_dw=False)
    b = rla.gated_ffn_backward(*args, need_dx=False)
    assert torch.equal(a[0], dx) and a[1] is None and a[2] is None
    assert b[0] is None and torch.equal(b[1], dwg) and torch.equal(b[2], dwu)
    assert rla.gated_ffn_backward(*args, need_dx=False, need_dw=False) == (None, None, None)


def test_rows_behind_the_output_are_left_alone():
    for M in (1, 4, 8, 90):
        t = inputs(M, 64, 100, torch.bfloat16, 4)
        dev = {k: v.to(DEV) for k, v in t.items()}
        big = torch.full((M + 2, 100), 7.0, dtype=torch.bfloat16, device=DEV)
        rla.gated_ffn(dev["x"], dev["w_gate"], dev["w_up"], out=big[1:M + 1])
        assert bool((big[0] == 7).all()) and bool((big[M + 1] == 7).all())
        check_forward(t, "silu", big[1:M + 1])


def test_a_row_of_nan_stays_its_own():
    for M in (3, 6, 130):
        t = inputs(M, 64, 64, torch.bfloat16, 5)
        dev = {k: v.to(DEV) for k, v in t.items()}
        want = rla.gated_ffn(dev["x"], dev["w_gate"], dev["w_up"])
        dev["x"][2] = float("nan")
        got = rla.gated_ffn(dev["x"], dev["w_gate"], dev["w_up"])
        assert torch.isnan(got[2]).all()
        keep = [i for i in range(M) if i != 2]
        assert torch.equal(got[keep], want[keep])


def test_empty_calls():
    x, w = torch.empty(0, 32, device=DEV), torch.ones(8, 32, device=DEV)
    h, g, u = rla.gated_ffn(x, w, w, save=True)
    assert h.shape == (0, 8)
    dx, dwg, dwu = rla.gated_ffn_backward(h, x, w, w, g, u)
    assert dx.shape == (0, 32) and bool((dwg == 0).all()) and bool((dwu == 0).all())
    x, w = torch.ones(5, 32, device=DEV), torch.empty(0, 32, device=DEV)
    h, g, u = rla.gated_ffn(x, w, w, save=True)
    dx, _, _ = rla.gated_ffn_backward(h, x, w, w, g, u)
    assert h.shape == (5, 0) and bool((dx == 0).all())


def test_gradients_against_differences():
    """Central differences of the fp32 kernel along one direction of each argument."""
    for M in (7, 70):
        t = inputs(M, 40, 56, torch.float32, 21)
        dev = {k: v.to(DEV) for k, v in t.items()}
        _, g, u = rla.gated_ffn(dev["x"], dev["w_gate"], dev["w_up"], "gelu_tanh", save=True)
        grads = rla.gated_ffn_backward(dev["dh"], dev["x"], dev["w_gate"], dev["w_up"], g, u, "gelu_tanh")
        gen = torch.Generator().manual_seed(3)
        step = 2.0 ** -8
        for name, grad in zip(("x", "w_gate", "w_up"), grads):
            v = torch.randn(dev[name].shape, generator=gen).to(DEV) / math.sqrt(40)

            def loss(s):
                moved = dict(dev)
                moved[name] = dev[name] + s * v
                return float((d(rla.gated_ffn(moved["x"], moved["w_gate"], moved["w_up"], "gelu_tanh")) *
                              d(dev["dh"])).sum())

            diff = (loss(step) - loss(-step)) / (2 * step)
            slope = float((d(grad) * d(v)).sum())
            # rounding: M * 56 outputs of size ~4 with sums of 40 terms, 2^-24 each, random in sign; the
            # truncation step^2 / 6 * third derivative, the projections moving by about 3 a unit
            noise = math.sqrt(M * 56 * 40) * 4 * 2.0 ** -24 / step
            assert abs(diff - slope) <= 4 * noise + step * step * 27 * math.sqrt(M * 56), (name, diff, slope)


def test_other_stream_and_graph():
    t = inputs(130, 200, 264, torch.bfloat16, 8)
    dev = {k: v.to(DEV) for k, v in t.items()}
    odd = {k: v.to(DEV) for k, v in inputs(70, 2051, 90, torch.bfloat16, 8).items()}

    def step():
        outs = []
        for v in (dev, odd):  # the second's sums are split: a workspace in the forward as well
            h, g, u = rla.gated_ffn(v["x"], v["w_gate"], v["w_up"], "gelu", save=True)
            outs += [h, *rla.gated_ffn_backward(v["dh"], v["x"], v["w_gate"], v["w_up"], g, u, "gelu")]
        return outs

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for v in (dev, odd):
        h, g, u = rla.gated_ffn(v["x"], v["w_gate"], v["w_up"], "gelu", save=True, stream=side)
        got += [h, *rla.gated_ffn_backward(v["dh"], v["x"], v["w_gate"], v["w_up"], g, u, "gelu", stream=side)]
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(4):
        gen = torch.Generator().manual_seed(50 + i)
        for v in (dev, odd):
            v["x"].copy_(randn(gen, *v["x"].shape, dtype=torch.bfloat16))
            v["dh"].copy_(randn(gen, *v["dh"].shape, dtype=torch.bfloat16))
        eager = step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, outs):
            assert torch.equal(a, b), i


def test_refusals_on_the_device():
    x, w = torch.zeros(4, 32, device=DEV), torch.zeros(16, 32, device=DEV)

    def refused(reason, f):
        with pytest.raises(rla.Ltx3dRopeUnsupported) as e:
            f()
        assert e.value.reason == reason

    refused("SHAPE_MISMATCH", lambda: rla.gated_ffn(x, w, w[:8]))
    refused("SHAPE_MISMATCH", lambda: rla.gated_ffn(x, w[:, :31].contiguous(), w))
    refused("DTYPE", lambda: rla.gated_ffn(x.half(), w.half(), w.half()))
    refused("DTYPE", lambda: rla.gated_ffn(x, w.bfloat16(), w))
    refused("NOT_DEVICE_PTR", lambda: rla.gated_ffn(x, w.cpu(), w))
    refused("NOT_CONTIGUOUS", lambda: rla.gated_ffn(torch.zeros(4, 64, device=DEV)[:, :32], w, w))
    buf = torch.zeros(4 * 32 + 4 * 16, device=DEV)
    refused("OVERLAP", lambda: rla.gated_ffn(buf[:128].view(4, 32), w, w, out=buf[100:164].view(4, 16)))
    with pytest.raises(ValueError):
        rla.gated_ffn(x, w, w, "relu")
    assert rla.stats()["fast_launches"] == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,D,F", [(5, 8, 8161), (5, 200, 8200), (8, 64, 8192), (9, 72, 8192), (15, 136, 8200), (16, 520, 8161),
                                   (16, 128, 16391), (17, 200, 8200), (33, 392, 8200), (64, 136, 8161), (100, 264, 8200),
                                   (128, 320, 4100), (129, 264, 8200)])
def test_few_tokens_of_wide_blocks(M, D, F, dtype):
    """Tiles with three steps on their way, sums of one step to some, where they begin and end."""
    run(M, D, F, dtype, "silu", M * F + D)


def test_few_tokens_repeat_their_bits():
    t = {k: v.to(DEV) for k, v in inputs(16, 1024, 8200, torch.bfloat16, 5).items()}
    first = rla.gated_ffn(t["x"], t["w_gate"], t["w_up"])
    for i in range(20):
        assert torch.equal(rla.gated_ffn(t["x"], t["w_gate"], t["w_up"]), first), i
    for m in (5, 9, 15):  # rows do not depend on their neighbours
        assert torch.equal(rla.gated_ffn(t["x"][:m], t["w_gate"], t["w_up"]), first[:m]), m


def act64(v, kind):
    """act(v) and its slope in 64 bits, to full relative precision on both sides."""
    if kind == "gelu":
        c, phi = torch.erfc(-v / math.sqrt(2.0)) / 2.0, torch.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)
        return v * c, c + v * phi, c.abs(), (v * phi).abs()
    k, cubic = (1.0, 0.0) if kind == "silu" else (math.sqrt(8.0 / math.pi), 0.044715)
    s = torch.sigmoid(k * (v + cubic * v ** 3))
    inner = torch.where((s == 0) | (s == 1), torch.zeros_like(s), k * (1.0 + 3 * cubic * v * v))
    t = torch.sigmoid(-k * (v + cubic * v ** 3))  # 1 - s
    return v * s, s + v * s * t * inner, s, (v * s * t * inner).abs()


def act_bounds(v, kind):
    """What act(v) and its slope in fp32 may be off by.

    gelu: the argument is off by 2 u relative (constant, product), which moves erfc(x) by (2 x^2 + 1) times
    as much, and erfcf itself is within 16 ulp; the density's exponent g^2 / 2 by 3 u relative.  Below 2^-126
    an ulp is 2^-149 whatever the value: half of 16 of those, and half of one for the halving, is below 2^-145.
    The others: z by 6 u (gelu_tanh) and z log2(e) by 2 u relative, exp2, 1 + and the reciprocal by 5 u:
    k |z| u + 8 u, the first weighed with 1 - s as e^-z is in 1 + e^-z.  Below 2^-126 the reciprocal may be 0."""
    a, slope, s, rest = act64(v, kind)
    if kind == "gelu":
        c_tol = (2 * v * v + 40) * U * s + 2.0 ** -145
        return v.abs() * c_tol + 2 * U * a.abs(), c_tol + rest * (2 * v * v + 8) * U + 2 * U * (s + rest)
    per, z = (2, v.abs()) if kind == "silu" else (8, 1.6 * v.abs() + 0.0715 * v.abs() ** 3)
    inner = 1.0 if kind == "silu" else 1.6 * (1.0 + 0.135 * v * v)
    t = (1.0 - s).clamp_min(0)
    s_tol = s * (t * (per * z + 2) + 8) * U + 2.0 ** -126
    away = t * s_tol + s * (s_tol + U)
    away = torch.where((s == 0) | (s == 1), torch.zeros_like(s), v.abs() * inner * away)
    return v.abs() * s_tol + 2 * U * a.abs(), s_tol + away + 10 * U * (s + rest)


def check_act(values, kind, dtype):
    """h = act(v) and its slope through one hidden unit: g = v and u = 1 exactly."""
    x = torch.stack([values, torch.ones_like(values)], 1).to(DEV)
    wg, wu = torch.tensor([[1.0, 0.0]], dtype=dtype, device=DEV), torch.tensor([[0.0, 1.0]], dtype=dtype, device=DEV)
    h, g, u = rla.gated_ffn(x, wg, wu, kind, save=True)
    assert torch.equal(g[:, 0].cpu(), values.float()) and bool((u == 1).all())
    dx, _, _ = rla.gated_ffn_backward(torch.ones_like(h), x, wg, wu, g, u, kind, need_dw=False)
    a, slope, _, _ = act64(d(values), kind)
    a_tol, slope_tol = act_bounds(d(values), kind)
    hs = half_step(dtype)
    for got, want, tol, what in ((h[:, 0], a, a_tol, "act"), (dx[:, 0], slope, slope_tol, "slope"),
                                 (dx[:, 1], a, a_tol, "act in dx")):
        assert_within(got, want, tol + hs * (want.abs() + tol) + tiny(dtype), what)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [3, 16, 1500])
@pytest.mark.parametrize("kind,low,high", [("silu", -80.0, 20.0), ("gelu", -12.5, 8.0), ("gelu_tanh", -9.5, 8.0)])
def test_activation_tails_relative_to_their_values(kind, low, high, M, dtype):
    check_act(torch.linspace(low, high, M).to(dtype), kind, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", KINDS)
def test_activations_of_huge_projections(kind, dtype):
    """Far out act(v) is v or 0 and its slope 1 or 0, also where v^2 and v^3 pass fp32's range."""
    v = torch.tensor([1e3, 1e6, 1e13, 1e15, 5e18, 3e19, 1e20, 1e30, 3e38])
    check_act(torch.cat([v, -v]).to(dtype), kind, dtype)


def test_through_an_autograd_function():
    """Calls are not recorded; a Function around one and its backward pass gives the leaves their gradients."""

    class Block(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, wg, wu):
            h, g, u = rla.gated_ffn(x, wg, wu, "gelu", save=True)
            ctx.save_for_backward(x, wg, wu, g, u)
            return h

        @staticmethod
        def backward(ctx, dh):
            return rla.gated_ffn_backward(dh, *ctx.saved_tensors, "gelu")

    t = inputs(40, 72, 88, torch.bfloat16, 13)
    leaves = [t[k].to(DEV).requires_grad_() for k in ("x", "w_gate", "w_up")]
    assert not rla.gated_ffn(*leaves, "gelu").requires_grad
    h = Block.apply(*leaves)
    h.backward(t["dh"].to(DEV))
    _, g, u = rla.gated_ffn(*leaves, "gelu", save=True)
    check_forward(t, "gelu", h)
    check_backward(t, "gelu", g, u, *[v.grad for v in leaves])
