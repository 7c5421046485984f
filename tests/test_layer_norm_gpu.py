"""The layer norms before and after a block on the GPU, forward and backward, against oracle.block in 64 bits.

Bounds.  A sum over a row is made of at most 16 terms a thread, 6 steps of a wavefront's sum and 16 of a
workgroup's: K = 40 fp32 operations bound it, and the few operations after it.  The mean is off by at most
E = K u mean|x|.  What the kernel holds is x less that mean: c + (at most E), its own mean off by K u times
its size; the variance is a sum of squares of that size.  A sum over rows takes at most `rows`
additions down a thread's walk and 64 more when the partial sums are joined.
"""
from __future__ import annotations

import pytest
import torch

import oracle.block as ob
from tests.block_tools import U, assert_within, d, half_step, randn, tiny

pytestmark = pytest.mark.gpu

rla = pytest.importorskip("rope_ltx3drope_amd")
from rope_ltx3drope_amd import _lib  # noqa: E402

DEV = "cuda:0"
K = 40
EPS = 1e-6


@pytest.fixture(autouse=True)
def fresh():
    assert torch.cuda.is_available()
    _lib.lib()
    rla.stats_reset()
    yield
    torch.cuda.synchronize()


class Case:
    """Inputs of one call, on the CPU in their own types, and their copies on the GPU."""

    def __init__(self, batch, rows, dim, dtype, pdtype, seed, weight=True, bias=True, gate=True, modulated=True,
                 mean=0.5, std=2.0, eps=EPS):
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.pdtype, self.rows, self.dim, self.batch = dtype, pdtype, rows, dim, batch
        self.eps = float(torch.tensor(eps))  # as the call takes it
        size = (batch, rows, dim)
        self.y, self.residual = randn(g, *size, std=std / 2, dtype=dtype), randn(g, *size, std=std, mean=mean, dtype=dtype)
        self.dr, self.dn = randn(g, *size, dtype=dtype), randn(g, *size, dtype=dtype)
        vec = lambda *s, std, mean=0.0: randn(g, *s, std=std, mean=mean, dtype=pdtype)  # noqa: E731
        self.weight = vec(dim, std=0.2, mean=1.0) if weight else None
        self.bias = vec(dim, std=0.3) if bias else None
        self.gate = vec(batch, dim, std=0.5) if gate else None
        self.scale = vec(batch, dim, std=0.3) if modulated else None
        self.shift = vec(batch, dim, std=0.3) if modulated else None

    def dev(self, name):
        t = getattr(self, name)
        return None if t is None else t.to(DEV)

    def kw(self):
        return dict(eps=self.eps, **{n: self.dev(n) for n in ("weight", "bias", "scale", "shift")})


def hat_bound(x, eps):
    """hat(x), its bound, its size with the mean's error in it, and 1/std with its relative bound."""
    hat, inv = ob.layer_norm_parts(x, eps)
    E = K * U * x.abs().mean(-1, keepdim=True)
    size = inv * ((x - x.mean(-1, keepdim=True)).abs() + E)
    # mean(d^2) and e^2 are at most mean(size^2) in units of the variance
    rel = 2 * K * U * (size * size).mean(-1, keepdim=True).clamp_min(1.0)
    tol = 4 * U * size + K * U * size.mean(-1, keepdim=True) + rel * hat.abs()
    return hat, tol, size, inv, rel


def term(c, x):
    """bias * (1 + scale) + shift, and the sum of its terms' magnitudes."""
    t, mag = torch.zeros_like(x), torch.zeros_like(x)
    s = 1.0 if c.scale is None else 1.0 + d(c.scale)[:, None, :]
    if c.bias is not None:
        t, mag = t + d(c.bias) * s, mag + (d(c.bias) * s).abs()
    if c.shift is not None:
        t, mag = t + d(c.shift)[:, None, :], mag + d(c.shift).abs()[:, None, :]
    return t, mag


def check_n(c, x, x_tol, got):
    """The norm at x, which the kernel holds to within x_tol."""
    hat, tol, _, inv, _ = hat_bound(x, c.eps)
    # an error of x moves the element, the mean and, through the variance, the whole row
    moved = inv * (x_tol + x_tol.mean(-1, keepdim=True))
    tol = tol + moved + hat.abs() * (hat.abs() * moved).mean(-1, keepdim=True)
    f = ob.norm_factor(d(c.weight), d(c.scale), 0.0, x).abs()
    _, mag = term(c, x)
    want = ob.layer_norm_before(x, d(c.weight), d(c.bias), d(c.scale), d(c.shift), c.eps)
    assert_within(got, want, f * tol + 6 * U * (f * hat.abs() + mag) + half_step(c.dtype) * want.abs() + tiny(c.dtype),
                  "n")


def check_after(c, r_got, n_got):
    y, res = d(c.y), d(c.residual)
    r = ob.layer_norm_residual(y, res, d(c.gate))
    tol = 2 * U * (res.abs() + (r - res).abs())
    assert_within(r_got, r, tol + half_step(c.dtype) * r.abs() + tiny(c.dtype), "r")
    check_n(c, r, tol, n_got)


def sum_tol(terms_abs, terms_tol, rows, axes):
    return terms_tol.sum(axes) + (rows + 64 + K) * U * terms_abs.sum(axes)


def check_backward(c, x, g, after):
    """g: the gradients by name; x: the norm's input (r, or the input before)."""
    xs, dn, dr = d(x), d(c.dn), d(c.dr)
    hs, ph = half_step(c.dtype), half_step(c.pdtype)
    dR, dw, dbias, dscale, dshift = ob.layer_norm_before_backward(dn, xs, d(c.weight), d(c.bias), d(c.scale), dr, c.eps)
    hat, hat_tol, size, inv, rel = hat_bound(xs, c.eps)
    v = (dn * ob.norm_factor(d(c.weight), d(c.scale), 0.0, xs))
    va = v.abs()
    mean = lambda t: t.mean(-1, keepdim=True)  # noqa: E731
    proj = mean(v * hat)
    # sum v d and e sum v, each of terms of size v * size
    proj_tol = mean(va * hat_tol) + 2 * K * U * mean(va * size) + 2 * K * U * mean(va) * mean(size) + rel * mean(va * size)
    inner = va + mean(va) + hat.abs() * mean(va * size)
    tol = inv * (8 * U * inner + K * U * mean(va) + hat.abs() * proj_tol + hat_tol * proj.abs() + rel * inner)
    dR_tol = tol + 4 * U * (dr.abs() + dR.abs())
    t = dn.abs() * size
    p1_tol, p2_tol = sum_tol(t, dn.abs() * hat_tol, c.rows, 1), sum_tol(dn.abs(), 0 * dn, c.rows, 1)
    s = torch.ones_like(xs[:, 0]) if c.scale is None else (1 + d(c.scale)).abs()
    w = torch.ones_like(xs[:, 0]) if c.weight is None else d(c.weight).expand_as(xs[:, 0]).abs()
    b = torch.zeros_like(xs[:, 0]) if c.bias is None else d(c.bias).expand_as(xs[:, 0]).abs()
    many = (c.batch + 68) * U
    if c.weight is not None:
        bound = (s * p1_tol).sum(0) + many * (s * t.sum(1)).sum(0)
        assert_within(g["weight"], dw, bound + ph * dw.abs() + tiny(c.pdtype), "dweight")
    if c.bias is not None:
        bound = (s * p2_tol).sum(0) + many * (s * dn.abs().sum(1)).sum(0)
        assert_within(g["bias"], dbias, bound + ph * dbias.abs() + tiny(c.pdtype), "dbias")
    if c.scale is not None:
        bound = w * p1_tol + b * p2_tol + 4 * U * (w * t.sum(1) + b * dn.abs().sum(1))
        assert_within(g["scale"], dscale, bound + ph * dscale.abs() + tiny(c.pdtype), "dscale")
    if c.shift is not None:
        assert_within(g["shift"], dshift, p2_tol + ph * dshift.abs() + tiny(c.pdtype), "dshift")
    assert_within(g["res"], dR, dR_tol + hs * dR.abs() + tiny(c.dtype), "dresidual")
    if not after:
        return
    y = d(c.y)
    dy, _, dgate = ob.layer_norm_after_backward(dR, y, d(c.gate))
    ga = torch.ones_like(y) if c.gate is None else d(c.gate).abs()[:, None, :]
    assert_within(g["y"], dy, ga * dR_tol + (hs + 2 * U) * dy.abs() + tiny(c.dtype), "dy")
    if c.gate is not None:
        bound = sum_tol((dR * y).abs(), dR_tol * y.abs(), c.rows, 1)
        assert_within(g["gate"], dgate, bound + ph * dgate.abs() + tiny(c.pdtype), "dgate")


def run_all(c):
    """Both forwards and both backwards of a case."""
    x = d(c.residual)
    check_n(c, x, torch.zeros_like(x), rla.layer_norm_before(c.dev("residual"), **c.kw()))
    r, n = rla.layer_norm_after(c.dev("y"), c.dev("residual"), c.dev("gate"), **c.kw())
    check_after(c, r, n)
    g = rla.layer_norm_after_backward(c.dev("dr"), c.dev("dn"), c.dev("y"), r, c.dev("gate"), **c.kw())
    check_backward(c, r, dict(res=g.dresidual, y=g.dy, gate=g.dgate, weight=g.dweight, bias=g.dbias, scale=g.dscale,
                              shift=g.dshift), True)
    b = rla.layer_norm_before_backward(c.dev("dn"), c.dev("residual"), dresidual=c.dev("dr"), **c.kw())
    check_backward(c, c.residual, dict(res=b.dx, weight=b.dweight, bias=b.dbias, scale=b.dscale, shift=b.dshift), False)
    return g, b


TYPES = [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32)]


@pytest.mark.parametrize("dtype,pdtype", TYPES)
@pytest.mark.parametrize("dim", [1, 2, 7, 8, 63, 64, 72, 511, 512, 520, 1000, 2048, 2053, 4096, 4100, 8192, 8193, 8200,
                                 16383, 16384])
def test_widths(dim, dtype, pdtype):
    """Widths around every boundary of the kernels' shapes, ragged rows, several samples."""
    run_all(Case(3, 5, dim, dtype, pdtype, dim))


@pytest.mark.parametrize("dtype,pdtype", TYPES)
@pytest.mark.parametrize("batch,rows,dim", [(1, 1, 4096), (4, 1, 4096), (1, 517, 264), (2, 1500, 96), (7, 3, 1920),
                                            (1, 9000, 64), (300, 2, 130), (33, 70, 40)])
def test_row_counts(batch, rows, dim, dtype, pdtype):
    """One row, more rows than a grid takes at once, many samples."""
    run_all(Case(batch, rows, dim, dtype, pdtype, 1000 + rows))


@pytest.mark.parametrize("dtype,pdtype", TYPES)
@pytest.mark.parametrize("weight,bias,gate,mod", [(w, b, g, m) for w in (0, 1) for b in (0, 1) for g in (0, 1)
                                                  for m in (0, 1)])
def test_parts_left_out(weight, bias, gate, mod, dtype, pdtype):
    """Every combination of weight, bias, gate and modulation."""
    g, b = run_all(Case(2, 9, 648, dtype, pdtype, 7, bool(weight), bool(bias), bool(gate), bool(mod)))
    assert [t is not None for t in g[2:]] == [bool(v) for v in (gate, weight, bias, mod, mod)]
    assert [t is not None for t in b[1:]] == [bool(v) for v in (weight, bias, mod, mod)]


@pytest.mark.parametrize("dim", [64, 2048, 2053])
@pytest.mark.parametrize("mean", [30.0, 3e3, -1e6])
def test_means_beside_which_the_spread_is_small(mean, dim):
    """A mean of up to a million times the spread (where fp32 holds the mean to 0.06 of it)."""
    run_all(Case(2, 7, dim, torch.float32, torch.float32, dim, mean=mean, std=1.0))


def test_rows_of_one_value():
    """No spread at all: hat is zero to within the mean's rounding, and nothing is NaN."""
    for value in (0.0, 1.0, 1000.1, -3.3e7, 1e30):
        x = torch.full((3, 777), value, device=DEV)
        n = rla.layer_norm_before(x, eps=EPS)
        # x less its own mean is exact to a step of |x| K u; its mean is off by K u of that
        assert float(n.abs().max()) <= 1000 * (K * U) ** 2 * abs(value) * 2
        b = rla.layer_norm_before_backward(x, x, eps=EPS)
        assert bool(torch.isfinite(b.dx).all())


@pytest.mark.parametrize("dtype,pdtype", TYPES)
@pytest.mark.parametrize("dim", [64, 2053, 4096, 16384])
@pytest.mark.parametrize("scale", [2.0 ** 55, 2.0 ** 61, 2.0 ** -40])
def test_rows_whose_squares_add_up_past_fp32(scale, dim, dtype, pdtype):
    """The variance is finite in fp32 (around 2e37 for the larger scale) where the sum of the squares, or one of
    them alone, is not; and rows far below 1.  The scaling is exact, so the bounds are those of any row."""
    c = Case(2, 5, dim, dtype, pdtype, dim + 1)
    c.y, c.residual = c.y * scale, c.residual * scale
    run_all(c)


def test_sums_that_pass_fp32():
    """mean(|x|) is finite and the sum of a row is not: 2048 values around 2^126."""
    gen = torch.Generator().manual_seed(1)
    x = torch.randint(-8, 9, (3, 2048), generator=gen).float() * 2.0 ** 103 + 2.0 ** 126
    n = rla.layer_norm_before(x.to(DEV))
    # (x - mean)^2 passes fp32: zeros, never NaN
    assert bool((n == 0).all())
    y = torch.randint(-8, 9, (3, 2048), generator=gen).float() * 2.0 ** 58 + 2.0 ** 80
    got = rla.layer_norm_before(y.to(DEV))
    want, tol, *_ = hat_bound(d(y), EPS)
    assert_within(got, want, tol + 6 * U * want.abs() + tiny(torch.float32), "n")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_unaligned_rows(dtype):
    """Row tensors that start one element past a 16-byte boundary."""
    c = Case(2, 11, 1024, dtype, torch.float32, 5)

    def shifted(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
        v = buf[1:].view(t.shape)
        v.copy_(t)
        assert v.data_ptr() % 16 != 0 and v.is_contiguous()
        return v

    r, n = rla.layer_norm_after(shifted(c.y), shifted(c.residual), c.dev("gate"), **c.kw())
    check_after(c, r, n)
    g = rla.layer_norm_after_backward(shifted(c.dr), shifted(c.dn), shifted(c.y), shifted(r.cpu()), c.dev("gate"),
                                      **c.kw())
    check_backward(c, r, dict(res=g.dresidual, y=g.dy, gate=g.dgate, weight=g.dweight, bias=g.dbias, scale=g.dscale,
                              shift=g.dshift), True)


def test_vectors_off_16_bytes():
    """Aligned rows with vectors that start one element past a 16-byte boundary: the aligned call's bits."""
    c = Case(2, 6, 1024, torch.bfloat16, torch.float32, 8)
    kw = c.kw()

    def shifted(t):
        v = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)[1:].view(t.shape)
        v.copy_(t)
        return v

    odd = {k: shifted(v) if torch.is_tensor(v) else v for k, v in kw.items()}
    args = (c.dev("y"), c.dev("residual"))
    a, b = rla.layer_norm_after(*args, c.dev("gate"), **kw), rla.layer_norm_after(*args, shifted(c.gate), **odd)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_two_dimensional_rows_and_vector():
    c = Case(1, 6, 256, torch.bfloat16, torch.float32, 3)
    kw = c.kw()
    a = rla.layer_norm_before(c.dev("residual"), **kw)
    flat = dict(kw, scale=kw["scale"][0], shift=kw["shift"][0])
    assert torch.equal(a[0], rla.layer_norm_before(c.dev("residual")[0], **flat))


def test_special_rows():
    """Zero rows, infinities and NaN stay in their own row; the rows beside them are as without them."""
    c = Case(1, 8, 512, torch.float32, torch.float32, 4)
    y, res, gate = c.dev("y"), c.dev("residual"), c.dev("gate")
    r0, n0 = rla.layer_norm_after(y, res, gate, **c.kw())
    y2, res2 = y.clone(), res.clone()
    y2[0, 1] = 0.0
    res2[0, 1] = 0.0
    y2[0, 3, 17] = float("nan")
    y2[0, 5, 100] = float("inf")
    r, n = rla.layer_norm_after(y2, res2, gate, **c.kw())
    for row in (0, 2, 4, 6, 7):
        assert torch.equal(r[0, row], r0[0, row]) and torch.equal(n[0, row], n0[0, row])
    assert bool((r[0, 1] == 0).all())
    x = torch.zeros(1, 1, 512, dtype=torch.float64)
    t, mag = term(c, x)
    assert_within(n[0, 1], t[0, 0], 4 * U * mag[0, 0], "n of a zero row")
    assert torch.isnan(n[0, 3]).all() and torch.isnan(n[0, 5]).all()
    assert torch.isinf(r[0, 5, 100]) and int(torch.isnan(r[0, 3]).sum()) == 1


def test_outputs_over_inputs():
    for dtype in (torch.float32, torch.bfloat16):
        c = Case(2, 13, 2048, dtype, torch.float32, 9)
        r0, n0 = rla.layer_norm_after(c.dev("y"), c.dev("residual"), c.dev("gate"), **c.kw())
        y, res = c.dev("y"), c.dev("residual")
        r, n = rla.layer_norm_after(y, res, c.dev("gate"), r_out=res, n_out=y, **c.kw())
        assert r.data_ptr() == res.data_ptr() and torch.equal(r, r0) and torch.equal(n, n0)
        x = c.dev("residual")
        want = rla.layer_norm_before(x, **c.kw())
        rla.layer_norm_before(x, out=x, **c.kw())
        assert torch.equal(x, want)


def test_rows_behind_the_outputs_are_left_alone():
    c = Case(1, 3, 520, torch.bfloat16, torch.bfloat16, 2)
    big = torch.full((1, 5, 520), 7.0, dtype=torch.bfloat16, device=DEV)
    rla.layer_norm_before(c.dev("residual"), out=big[:, 1:4], **c.kw())
    assert bool((big[:, 0] == 7).all()) and bool((big[:, 4] == 7).all()) and not bool((big[:, 1:4] == 7).all())


def test_empty_calls():
    x = torch.empty(2, 0, 64, device=DEV)
    w, v = torch.ones(64, device=DEV), torch.ones(2, 64, device=DEV)
    assert rla.layer_norm_before(x, w, w, v, v).shape == x.shape
    g = rla.layer_norm_after_backward(x, x, x, x, v, weight=w, bias=w, scale=v, shift=v)
    for t in (g.dgate, g.dweight, g.dbias, g.dscale, g.dshift):
        assert bool((t == 0).all())
    x0, v0 = torch.empty(0, 3, 64, device=DEV), torch.empty(0, 64, device=DEV)
    g = rla.layer_norm_before_backward(x0, x0, w, w, v0, v0)
    assert bool((g.dweight == 0).all()) and bool((g.dbias == 0).all()) and g.dscale.shape == (0, 64)


def test_without_a_gradient_past_the_norm():
    c = Case(2, 9, 264, torch.bfloat16, torch.float32, 15)
    c.dr = torch.zeros_like(c.dr)
    a = rla.layer_norm_after_backward(c.dev("dr"), c.dev("dn"), c.dev("y"), c.dev("residual"), c.dev("gate"), **c.kw())
    b = rla.layer_norm_after_backward(None, c.dev("dn"), c.dev("y"), c.dev("residual"), c.dev("gate"), **c.kw())
    for s, t in zip(a, b):
        assert torch.equal(s, t)
    # without a gate y is not needed
    g = rla.layer_norm_after_backward(c.dev("dr"), c.dev("dn"), None, c.dev("residual"), **c.kw())
    assert g.dgate is None and torch.equal(g.dy, g.dresidual)


def test_equal_calls_give_equal_bits():
    c = Case(2, 700, 1024, torch.bfloat16, torch.float32, 6)
    outs = [rla.layer_norm_after_backward(c.dev("dr"), c.dev("dn"), c.dev("y"), c.dev("residual"), c.dev("gate"),
                                          **c.kw()) for _ in range(4)]
    for o in outs[1:]:
        for a, b in zip(outs[0], o):
            assert torch.equal(a, b)


def test_gradients_against_differences():
    """Central differences of the fp32 kernel along one direction against its own gradients."""
    c = Case(2, 6, 96, torch.float32, torch.float32, 11)
    names = ["y", "residual", "gate", "weight", "bias", "scale", "shift"]
    base = {n: c.dev(n) for n in names}
    gen = torch.Generator().manual_seed(1)
    dirs = {n: torch.randn(base[n].shape, generator=gen).to(DEV) for n in names}
    dr, dn = c.dev("dr"), c.dev("dn")

    def forward(v):
        return rla.layer_norm_after(v["y"], v["residual"], v["gate"], weight=v["weight"], bias=v["bias"],
                                    scale=v["scale"], shift=v["shift"], eps=EPS)

    def loss(step, only):
        r, n = forward({n: base[n] + (step * dirs[n] if n == only else 0) for n in names})
        return float((d(r) * d(dr)).sum() + (d(n) * d(dn)).sum())

    r, _ = forward(base)
    g = rla.layer_norm_after_backward(dr, dn, base["y"], r, base["gate"], weight=base["weight"], bias=base["bias"],
                                      scale=base["scale"], shift=base["shift"], eps=EPS)
    grads = dict(y=g.dy, residual=g.dresidual, gate=g.dgate, weight=g.dweight, bias=g.dbias, scale=g.dscale,
                 shift=g.dshift)
    h = 2.0 ** -9
    # each of the 2304 products r*dr, n*dn carries about 8 roundings of 2^-24 of size ~4, random in sign
    noise = 8 * 2.0 ** -24 * 4 * 2304 ** 0.5 / h
    for n in names:
        slope = float((d(grads[n]) * d(dirs[n])).sum())
        diff = (loss(h, n) - loss(-h, n)) / (2 * h)
        # truncation: h^2/6 of the third derivative, below about 60 times the gradient's size here
        assert abs(diff - slope) <= 4 * noise + 10 * h * h * float(d(grads[n]).norm()) * 6, (n, diff, slope)


def test_other_stream_and_graph():
    """The calls on a side stream, then captured and replayed with new inputs against eager calls."""
    c = Case(2, 40, 1024, torch.bfloat16, torch.float32, 12)
    args = {n: c.dev(n) for n in ("y", "residual", "gate", "dr", "dn")}
    kw = c.kw()

    def step(**more):
        r, n = rla.layer_norm_after(args["y"], args["residual"], args["gate"], **kw, **more)
        return (r, n) + tuple(rla.layer_norm_after_backward(args["dr"], args["dn"], args["y"], r, args["gate"], **kw,
                                                            **more))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(stream=side)
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
        gen = torch.Generator().manual_seed(100 + i)
        for k in ("y", "residual", "dr", "dn"):
            args[k].copy_(randn(gen, *args[k].shape, dtype=torch.bfloat16))
        eager = step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, outs):
            assert torch.equal(a, b), i


def test_refusals_on_the_device():
    x = torch.zeros(2, 3, 64, device=DEV)
    w = torch.ones(64, device=DEV)
    buf = torch.zeros(7 * 64, device=DEV)

    def refused(reason, f):
        with pytest.raises(rla.Ltx3dRopeUnsupported) as e:
            f()
        assert e.value.reason == reason

    refused("OVERLAP", lambda: rla.layer_norm_before(buf[:384].view(2, 3, 64), out=buf[64:448].view(2, 3, 64)))
    refused("NOT_DEVICE_PTR", lambda: rla.layer_norm_before(x, w.cpu()))
    refused("NOT_CONTIGUOUS", lambda: rla.layer_norm_before(torch.zeros(2, 3, 128, device=DEV)[..., :64], w))
    refused("SHAPE_MISMATCH", lambda: rla.layer_norm_before(x, torch.ones(65, device=DEV)))
    refused("SHAPE_MISMATCH", lambda: rla.layer_norm_before(x, w, w, torch.ones(3, 64, device=DEV)))
    refused("SHAPE_MISMATCH", lambda: rla.layer_norm_after(x, x[:1]))
    refused("DTYPE", lambda: rla.layer_norm_before(x, w, w.bfloat16()))
    refused("DTYPE", lambda: rla.layer_norm_before(x.half(), w.half()))
    refused("TOO_LARGE", lambda: rla.layer_norm_before(torch.zeros(1, 1, 16385, device=DEV)))
    with pytest.raises(rla.Ltx3dRopeError) as e:
        rla.layer_norm_before(x, w, eps=0.0)
    assert e.value.status == _lib.E_INVALID
    assert rla.stats()["fast_launches"] == 0


def test_more_than_two_to_the_32_elements():
    """2^21 + 5 rows of 2056: offsets pass 32 bits.  The last rows against the same rows alone, and the weight's
    gradient, whose every term is a small integer times 2^-k, against the count."""
    rows, dim = (1 << 21) + 5, 2056
    x = torch.empty(1, rows, dim, dtype=torch.bfloat16, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(2)
    tail = torch.randn(64, dim, generator=gen, device=DEV).bfloat16()
    x.view(-1)[: rows * dim - 64 * dim].fill_(1.0)
    x[0, -64:] = tail
    n = rla.layer_norm_before(x)
    alone = rla.layer_norm_before(tail)
    assert torch.equal(n[0, -64:], alone)
    assert bool((n[0, : 1 << 12] == 0).all()) and bool((n[0, (1 << 20): (1 << 20) + 4096] == 0).all())
    b = torch.zeros(dim, device=DEV)
    g = rla.layer_norm_before_backward(x, n, None, b)
    # dbias: the sum of dn = 1 over rows - 64 rows, and the tail's
    want = rows - 64 + d(tail).sum(0)
    assert_within(g.dbias, want, (rows / 512 + 600) * U * (rows + d(tail).abs().sum(0)), "dbias")
