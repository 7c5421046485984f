"""The norms before and after a block on the GPU, forward and backward, against oracle.block in 64 bits.

Bounds.  A sum of squares over a row is made of at most 16 products a thread, 6 steps of a wavefront's
sum and 16 of a workgroup's: K_ROW = 40 fp32 operations bound it, its reciprocal root (half the
relative error, and 2 u of its own) and the few products after it.  A sum over rows takes at most
`rows` additions down a thread's walk and 64 more when the partial sums are joined.
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
K_ROW = 40
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

    def __init__(self, batch, rows, dim, dtype, pdtype, seed, post=True, weight=True, gate=True, next_norm=True,
                 modulated=True, offset=0.0, res_scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.pdtype, self.post, self.next_norm = dtype, pdtype, post, next_norm
        self.offset, self.res_scale, self.rows, self.dim, self.batch = offset, res_scale, rows, dim, batch
        rowsz = (batch, rows, dim)
        self.y, self.residual = randn(g, *rowsz, dtype=dtype), randn(g, *rowsz, std=2.0, dtype=dtype)
        self.dr, self.dn = randn(g, *rowsz, dtype=dtype), randn(g, *rowsz, dtype=dtype)
        vec = lambda *s, std, mean=0.0: randn(g, *s, std=std, mean=mean, dtype=pdtype)  # noqa: E731
        self.weight = vec(dim, std=0.2, mean=1.0 - offset) if weight else None
        self.gate = vec(batch, dim, std=0.5) if gate else None
        self.nw = vec(dim, std=0.2, mean=1.0 - offset) if next_norm else None
        self.ns = vec(batch, dim, std=0.3) if next_norm and modulated else None
        self.nb = vec(batch, dim, std=0.3) if next_norm and modulated else None
        if not next_norm:
            self.dn = None

    def dev(self, name):
        t = getattr(self, name)
        return None if t is None else t.to(DEV)

    def kw(self):
        return dict(eps=EPS, weight_offset=self.offset)

    def after_kw(self):
        k = dict(post_norm=self.post, residual_scale=self.res_scale, next_norm=self.next_norm, **self.kw())
        if self.next_norm:
            k.update(next_weight=self.dev("nw"), next_scale=self.dev("ns"), next_shift=self.dev("nb"))
        return k


def check_before(c, got):
    x = d(c.residual)
    want = ob.norm_before(x, d(c.nw), d(c.ns), d(c.nb), EPS, c.offset)
    mag = ob.norm_before(x.abs(), None, None, None, EPS, 0) * ob.norm_factor(d(c.nw), d(c.ns), c.offset, x).abs()
    if c.nb is not None:
        mag = mag + d(c.nb).abs()[:, None, :]
    assert_within(got, want, K_ROW * U * mag + half_step(c.dtype) * want.abs() + tiny(c.dtype), "n")


def r_and_bound(c):
    """r in 64 bits and what its fp32 form may be off by."""
    y, res = d(c.y), d(c.residual)
    r = ob.norm_after(y, res, d(c.weight), d(c.gate), c.post, c.res_scale, EPS, c.offset)
    hat = y * ob.rstd(y, EPS) if c.post else y
    mag = (c.res_scale * res).abs() + (hat * ob.branch_factor(d(c.weight), d(c.gate), c.offset, y)).abs()
    return r, K_ROW * U * mag


def check_after(c, r_got, n_got):
    r, tol = r_and_bound(c)
    assert_within(r_got, r, tol + half_step(c.dtype) * r.abs() + tiny(c.dtype), "r")
    if not c.next_norm:
        assert n_got is None
        return
    n = ob.norm_before(r, d(c.nw), d(c.ns), d(c.nb), EPS, c.offset)
    f = ob.norm_factor(d(c.nw), d(c.ns), c.offset, r).abs()
    inv = ob.rstd(r, EPS)
    hat = (r * inv).abs()
    # r's own error moves the element and, through the root of the mean square, the whole row
    moved = inv * tol + hat * (hat * inv * tol).mean(-1, keepdim=True)
    mag = hat * f + (0 if c.nb is None else d(c.nb).abs()[:, None, :])
    assert_within(n_got, n, f * moved + K_ROW * U * mag + half_step(c.dtype) * n.abs() + tiny(c.dtype), "n")


def through_norm_bound(v, v_tol, hat, inv):
    """Bound of inv * (v - hat * mean(v hat)) for v off by v_tol; hat and inv off by K_ROW u relative."""
    mean = (v * hat).abs().mean(-1, keepdim=True)
    mean_tol = (v_tol * hat.abs()).mean(-1, keepdim=True) + 2 * K_ROW * U * mean
    return inv * (v_tol + hat.abs() * mean_tol + 3 * K_ROW * U * (v.abs() + hat.abs() * mean))


def sum_tol(terms_abs, terms_tol, rows, axes):
    return terms_tol.sum(axes) + (rows + 64 + K_ROW) * U * terms_abs.sum(axes)


def check_backward(c, x, g, after):
    """g: the gradients by name; x: the row tensor under the next norm (r, or the input before)."""
    xs, dn, dr = d(x), d(c.dn), d(c.dr)
    hs = half_step(c.dtype)
    ph = half_step(c.pdtype)
    dR, dR_tol = dr, torch.zeros_like(dr)
    if c.next_norm:
        dR, dnw, dns, dnb = ob.norm_before_backward(dn, xs, d(c.nw), d(c.ns), dr, EPS, c.offset)
        inv = ob.rstd(xs, EPS)
        hat = xs * inv
        f = ob.norm_factor(d(c.nw), d(c.ns), c.offset, xs)
        v = dn * f
        dR_tol = through_norm_bound(v, 4 * U * v.abs(), hat, inv) + 4 * U * (dr.abs() + dR.abs())
        t = (dn * hat).abs()
        w = torch.ones_like(xs[:, 0]) if c.nw is None else (d(c.nw) + c.offset).expand_as(xs[:, 0]).abs()
        s = torch.ones_like(xs[:, 0]) if c.ns is None else (1 + d(c.ns)).abs()
        p_tol = sum_tol(t, K_ROW * U * t, c.rows, 1)
        if c.nw is not None:
            tol = (s * p_tol).sum(0) + (c.batch + 4) * U * (s * t.sum(1)).sum(0)
            assert_within(g["nw"], dnw, tol + ph * dnw.abs() + tiny(c.pdtype), "dnext_weight")
        if c.ns is not None:
            assert_within(g["ns"], dns, w * p_tol + 4 * U * w * t.sum(1) + ph * dns.abs() + tiny(c.pdtype), "dscale")
        if c.nb is not None:
            assert_within(g["nb"], dnb, sum_tol(dn.abs(), 0 * dn, c.rows, 1) + ph * dnb.abs() + tiny(c.pdtype),
                          "dshift")
    want = c.res_scale * dR
    assert_within(g["res"], want, abs(c.res_scale) * dR_tol + 2 * U * want.abs() + hs * want.abs() + tiny(c.dtype),
                  "dresidual")
    if not after:
        return
    y = d(c.y)
    dy, _, dw, dgate = ob.norm_after_backward(dR, y, d(c.weight), d(c.gate), c.post, c.res_scale, EPS, c.offset)
    inv = ob.rstd(y, EPS) if c.post else torch.ones_like(y[..., :1])
    hat = y * inv
    f = ob.branch_factor(d(c.weight), d(c.gate), c.offset, y)
    q, q_tol = dR * f, dR_tol * f.abs() + 4 * U * (dR * f).abs()
    tol = through_norm_bound(q, q_tol, hat, inv) if c.post else q_tol
    assert_within(g["y"], dy, tol + hs * dy.abs() + tiny(c.dtype), "dy")
    t, t_tol = (dR * hat).abs(), dR_tol * hat.abs() + K_ROW * U * (dR * hat).abs()
    p_tol = sum_tol(t, t_tol, c.rows, 1)
    gt = torch.ones_like(y[:, 0]) if c.gate is None else d(c.gate).abs()
    wt = torch.ones_like(y[:, 0]) if c.weight is None else (d(c.weight) + c.offset).expand_as(y[:, 0]).abs()
    if c.weight is not None:
        assert_within(g["w"], dw, (gt * p_tol).sum(0) + (c.batch + 4) * U * (gt * t.sum(1)).sum(0) + ph * dw.abs() +
                      tiny(c.pdtype), "dweight")
    if c.gate is not None:
        assert_within(g["gate"], dgate, wt * p_tol + 4 * U * wt * t.sum(1) + ph * dgate.abs() + tiny(c.pdtype), "dgate")


def run_all(c):
    """Both forwards and both backwards of a case."""
    if c.next_norm:
        check_before(c, rla.norm_before(c.dev("residual"), c.dev("nw"), c.dev("ns"), c.dev("nb"), **c.kw()))
    r, n = rla.norm_after(c.dev("y"), c.dev("residual"), c.dev("weight"), c.dev("gate"), **c.after_kw())
    check_after(c, r, n)
    g = rla.norm_after_backward(c.dev("dr"), c.dev("dn"), c.dev("y"), r, c.dev("weight"), c.dev("gate"), **c.after_kw())
    check_backward(c, r, dict(res=g.dresidual, y=g.dy, w=g.dweight, gate=g.dgate, nw=g.dnext_weight,
                              ns=g.dnext_scale, nb=g.dnext_shift), True)
    if c.next_norm and c.res_scale == 1.0:
        b = rla.norm_before_backward(c.dev("dn"), c.dev("residual"), c.dev("nw"), c.dev("ns"), c.dev("nb"),
                                     dresidual=c.dev("dr"), **c.kw())
        check_backward(c, c.residual, dict(res=b.dx, nw=b.dweight, ns=b.dscale, nb=b.dshift), False)


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
@pytest.mark.parametrize("post,weight,gate,nxt,mod", [(p, w, g, n, m) for p in (0, 1) for w in (0, 1) for g in (0, 1)
                                                      for n in (0, 1) for m in (0, 1) if n or not m])
def test_parts_left_out(post, weight, gate, nxt, mod, dtype, pdtype):
    """Every combination of post norm, weight, gate, next norm and its modulation; offset and residual scale."""
    run_all(Case(2, 9, 648, dtype, pdtype, 7, bool(post), bool(weight), bool(gate), bool(nxt), bool(mod), offset=1.0))
    run_all(Case(2, 9, 648, dtype, pdtype, 8, bool(post), bool(weight), bool(gate), bool(nxt), bool(mod),
                 res_scale=0.5))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_unaligned_rows(dtype):
    """Row tensors that start one element past a 16-byte boundary give the aligned call's values."""
    c = Case(2, 11, 1024, dtype, torch.float32, 5)

    def shifted(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
        v = buf[1:].view(t.shape)
        v.copy_(t)
        assert v.data_ptr() % 16 != 0 and v.is_contiguous()
        return v

    r, n = rla.norm_after(shifted(c.y), shifted(c.residual), c.dev("weight"), c.dev("gate"), **c.after_kw())
    check_after(c, r, n)
    g = rla.norm_after_backward(shifted(c.dr), shifted(c.dn), shifted(c.y), shifted(r.cpu()), c.dev("weight"),
                                c.dev("gate"), **c.after_kw())
    check_backward(c, r, dict(res=g.dresidual, y=g.dy, w=g.dweight, gate=g.dgate, nw=g.dnext_weight,
                              ns=g.dnext_scale, nb=g.dnext_shift), True)


def test_two_dimensional_rows_and_vector():
    c = Case(1, 6, 256, torch.bfloat16, torch.float32, 3)
    a = rla.norm_before(c.dev("residual"), c.dev("nw"), c.dev("ns"), c.dev("nb"), **c.kw())
    b = rla.norm_before(c.dev("residual")[0], c.dev("nw"), c.dev("ns")[0], c.dev("nb")[0], **c.kw())
    assert torch.equal(a[0], b)


def test_special_rows():
    """Zero rows, infinities and NaN stay in their own row; the rows beside them are as without them."""
    c = Case(1, 8, 512, torch.float32, torch.float32, 4)
    kw = c.after_kw()
    args = (c.dev("weight"), c.dev("gate"))
    y, res = c.dev("y"), c.dev("residual")
    r0, n0 = rla.norm_after(y, res, *args, **kw)
    y2, res2 = y.clone(), res.clone()
    y2[0, 1] = 0.0
    res2[0, 1] = 0.0
    y2[0, 3, 17] = float("nan")
    y2[0, 5, 100] = float("inf")
    r, n = rla.norm_after(y2, res2, *args, **kw)
    for row in (0, 2, 4, 6, 7):
        assert torch.equal(r[0, row], r0[0, row]) and torch.equal(n[0, row], n0[0, row])
    assert torch.equal(r[0, 1], torch.zeros_like(r[0, 1]))
    assert torch.equal(n[0, 1], c.dev("nb")[0])
    assert torch.isnan(r[0, 3]).all() and torch.isnan(n[0, 3]).all()
    assert torch.isnan(r[0, 5, 100]) and torch.isnan(n[0, 5]).all()


def test_outputs_over_inputs():
    for dtype in (torch.float32, torch.bfloat16):
        c = Case(2, 13, 2048, dtype, torch.float32, 9)
        r0, n0 = rla.norm_after(c.dev("y"), c.dev("residual"), c.dev("weight"), c.dev("gate"), **c.after_kw())
        y, res = c.dev("y"), c.dev("residual")
        r, n = rla.norm_after(y, res, c.dev("weight"), c.dev("gate"), r_out=res, n_out=y, **c.after_kw())
        assert r.data_ptr() == res.data_ptr() and torch.equal(r, r0) and torch.equal(n, n0)
        x = c.dev("residual")
        want = rla.norm_before(x, c.dev("nw"), c.dev("ns"), c.dev("nb"), **c.kw())
        rla.norm_before(x, c.dev("nw"), c.dev("ns"), c.dev("nb"), out=x, **c.kw())
        assert torch.equal(x, want)


def test_rows_behind_the_outputs_are_left_alone():
    c = Case(1, 3, 520, torch.bfloat16, torch.bfloat16, 2)
    big = torch.full((1, 5, 520), 7.0, dtype=torch.bfloat16, device=DEV)
    rla.norm_before(c.dev("residual"), c.dev("nw"), out=big[:, 1:4], **c.kw())
    assert bool((big[:, 0] == 7).all()) and bool((big[:, 4] == 7).all()) and not bool((big[:, 1:4] == 7).all())


def test_empty_calls():
    x = torch.empty(2, 0, 64, device=DEV)
    w, v = torch.ones(64, device=DEV), torch.ones(2, 64, device=DEV)
    assert rla.norm_before(x, w, v, v).shape == x.shape
    g = rla.norm_after_backward(x, x, x, x, w, v, next_weight=w, next_scale=v, next_shift=v)
    for t in (g.dweight, g.dgate, g.dnext_weight, g.dnext_scale, g.dnext_shift):
        assert bool((t == 0).all())
    x0 = torch.empty(0, 3, 64, device=DEV)
    v0 = torch.empty(0, 64, device=DEV)
    g = rla.norm_before_backward(x0, x0, w, v0, v0)
    assert bool((g.dweight == 0).all()) and g.dscale.shape == (0, 64)


def test_equal_calls_give_equal_bits():
    c = Case(2, 700, 1024, torch.bfloat16, torch.float32, 6)
    r, _ = rla.norm_after(c.dev("y"), c.dev("residual"), c.dev("weight"), c.dev("gate"), **c.after_kw())
    outs = [rla.norm_after_backward(c.dev("dr"), c.dev("dn"), c.dev("y"), r, c.dev("weight"), c.dev("gate"),
                                    **c.after_kw()) for _ in range(4)]
    for o in outs[1:]:
        for a, b in zip(outs[0], o):
            assert torch.equal(a, b)


def test_gradients_against_differences():
    """Central differences of the fp32 kernel along one direction against its own gradients."""
    c = Case(2, 6, 96, torch.float32, torch.float32, 11, offset=1.0, res_scale=0.75)
    names = ["y", "residual", "weight", "gate", "nw", "ns", "nb"]
    base = {n: c.dev(n) for n in names}
    gen = torch.Generator().manual_seed(1)
    dirs = {n: torch.randn(base[n].shape, generator=gen).to(DEV) for n in names}
    dr, dn = c.dev("dr"), c.dev("dn")

    def loss(step, only):
        v = {n: base[n] + (step * dirs[n] if n == only else 0) for n in names}
        r, n = rla.norm_after(v["y"], v["residual"], v["weight"], v["gate"], post_norm=True, residual_scale=0.75,
                              next_weight=v["nw"], next_scale=v["ns"], next_shift=v["nb"], **c.kw())
        return float((d(r) * d(dr)).sum() + (d(n) * d(dn)).sum())

    r, _ = rla.norm_after(base["y"], base["residual"], base["weight"], base["gate"], **c.after_kw())
    g = rla.norm_after_backward(dr, dn, base["y"], r, base["weight"], base["gate"], **c.after_kw())
    grads = dict(y=g.dy, residual=g.dresidual, weight=g.dweight, gate=g.dgate, nw=g.dnext_weight, ns=g.dnext_scale,
                 nb=g.dnext_shift)
    h = 2.0 ** -9
    # each of the 2304 products r*dr, n*dn carries about 8 roundings of 2^-24 of size ~4, random in sign
    noise = 8 * 2.0 ** -24 * 4 * 2304 ** 0.5 / h
    for n in names:
        slope = float((d(grads[n]) * d(dirs[n])).sum())
        diff = (loss(h, n) - loss(-h, n)) / (2 * h)
        # the truncation error is h^2/6 of the third derivative, which these norms keep below about 60
        # times the first derivatives' size, taken as the root of the sum of squares of the gradient
        size = float(d(grads[n]).norm())
        assert abs(diff - slope) <= 4 * noise + 10 * h * h * size * 6, (n, diff, slope)


def test_other_stream_and_graph():
    """The calls on a side stream, then captured and replayed with new inputs against eager calls."""
    c = Case(2, 40, 1024, torch.bfloat16, torch.float32, 12)
    args = {n: c.dev(n) for n in ("y", "residual", "weight", "gate", "dr", "dn")}
    kw = c.after_kw()

    def step():
        r, n = rla.norm_after(args["y"], args["residual"], args["weight"], args["gate"], **kw)
        return (r, n) + tuple(rla.norm_after_backward(args["dr"], args["dn"], args["y"], r, args["weight"],
                                                      args["gate"], **kw))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r, n = rla.norm_after(args["y"], args["residual"], args["weight"], args["gate"], stream=side, **kw)
    g = rla.norm_after_backward(args["dr"], args["dn"], args["y"], r, args["weight"], args["gate"], stream=side, **kw)
    side.synchronize()
    for a, b in zip(want, (r, n) + tuple(g)):
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

    def refused(reason, f):
        with pytest.raises(rla.Ltx3dRopeUnsupported) as e:
            f()
        assert e.value.reason == reason

    refused("OVERLAP", overlap)
    refused("NOT_DEVICE_PTR", lambda: rla.norm_before(x, w.cpu()))
    refused("NOT_CONTIGUOUS", lambda: rla.norm_before(torch.zeros(2, 3, 128, device=DEV)[..., :64], w))
    refused("SHAPE_MISMATCH", lambda: rla.norm_before(x, torch.ones(65, device=DEV)))
    refused("SHAPE_MISMATCH", lambda: rla.norm_before(x, w, torch.ones(3, 64, device=DEV)))
    refused("DTYPE", lambda: rla.norm_before(x, w.bfloat16()))
    refused("DTYPE", lambda: rla.norm_before(x.half(), w.half()))
    refused("TOO_LARGE", lambda: rla.norm_before(torch.zeros(1, 1, 16385, device=DEV)))
    with pytest.raises(rla.Ltx3dRopeError) as e:
        rla.norm_before(x, w, eps=0.0)
    assert e.value.status == _lib.E_INVALID
    assert rla.stats()["fast_launches"] == 0


def overlap():
    buf = torch.zeros(7 * 64, device=DEV)
    rla.norm_before(buf[:384].view(2, 3, 64), out=buf[64:448].view(2, 3, 64))


def test_ranges_past_an_allocation_are_refused():
    import ctypes

    L, reason = _lib.lib(), ctypes.c_int(-1)
    x = torch.zeros(1024, device=DEV)
    # rows of half a terabyte, in place
    call = _lib.Norm(dtype=_lib.DTYPE_F32, param_dtype=_lib.DTYPE_F32, after=0, post_norm=0, next_norm=1, batch=1,
                     rows=1 << 27, dim=1024, eps=1e-6, weight_offset=0.0, residual_scale=1.0, residual=x.data_ptr(),
                     n=x.data_ptr())
    assert L.ltx3drope_norm(call, None, reason) == _lib.E_UNSUPPORTED
    assert _lib.REASONS[reason.value] == "EXTENT"
    # output and input inside an allocation, weights that begin in it and pass its end
    hidden, dim = 1 << 19, 1 << 13
    buf = torch.zeros(hidden + 2 * dim, device=DEV)
    at = buf.data_ptr()
    call = _lib.GatedFfn(dtype=_lib.DTYPE_F32, activation=0, tokens=1, dim=dim, hidden=hidden, x=at + 4 * hidden,
                         w_gate=at + 4 * (hidden + dim), w_up=at + 4 * (hidden + dim), h=at)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    assert L.ltx3drope_gated_ffn(call, None, reason) == _lib.E_UNSUPPORTED
    assert _lib.REASONS[reason.value] == "EXTENT"
    assert rla.stats()["fast_launches"] == 0


@pytest.mark.parametrize("dtype,pdtype", TYPES)
@pytest.mark.parametrize("dim", [64, 2053, 4096, 16384])
@pytest.mark.parametrize("scale", [2.0 ** 55, 2.0 ** 61])
def test_rows_whose_squares_add_up_past_fp32(scale, dim, dtype, pdtype):
    """mean(v^2) is finite in fp32 (around 2e37 for the larger scale) where the sum of the squares, or one of
    them alone, is not; and the same rows as far below 1.  The scaling is exact, so the bounds are those of any row."""
    for post in (True, False):
        for s in (scale, 1.0 / scale):
            c = Case(2, 5, dim, dtype, pdtype, dim + 1, post=post)
            c.y, c.residual = c.y * s, c.residual * s
            run_all(c)


@pytest.mark.parametrize("eps", [1e-30, 2e-33, 1e-36])
def test_smallest_eps(eps):
    """Rows around sqrt(eps): the squares lie close to fp32's smallest normal number."""
    g = torch.Generator().manual_seed(6)
    x = randn(g, 3, 4096) * float(torch.tensor(eps).sqrt())
    got = rla.norm_before(x.to(DEV), eps=eps)
    eps32 = float(torch.tensor(eps))  # as the call takes it
    # squares under the smallest normal number are off by 2^-150 each, with an eps of 2^-110 or more after
    # they were scaled by 2^-14
    want = ob.norm_before(d(x)[None], None, None, None, eps32, 0.0)[0]
    under = 2.0 ** (-136 if eps >= 2.0 ** -110 else -150) / (d(x) ** 2).mean(-1, keepdim=True).clamp_min(eps32)
    assert_within(got, want, (K_ROW * U + under) * want.abs() + tiny(torch.float32), "n")
