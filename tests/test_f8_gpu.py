"""The linear layer in 8-bit floating point on the GPU against oracle.f8: the quantisers bit for bit, the product
exactly on integers with powers of two as scales, and otherwise within the rounding of its sums.

Bounds.  A block's 128 products are added by the matrix cores in fp32, each addition within a step of 2^-23
(whether it rounds or cuts off); a block's sum takes a product with the scales (three roundings) and an
addition, and what is split over k is added 16 times at the most.  With y in bf16 and more than 16 tokens the
products of each 8 neighbours of k are added by units that keep 2^-13 of the largest, by its exponents
(2^e for a product in [2^e, 2^(e+2))): seven of them may lose 2^-13 of it each.
"""
from __future__ import annotations

import pytest
import torch

import oracle.f8 as of
from tests.block_tools import U, assert_within, d, half_step, randn, tiny

pytestmark = pytest.mark.gpu

rla = pytest.importorskip("rope_ltx3drope_amd")
from rope_ltx3drope_amd import _lib  # noqa: E402

DEV = "cuda:0"
TYPES = [torch.float32, torch.bfloat16]
F8 = torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def fresh():
    assert torch.cuda.is_available()
    _lib.lib()
    rla.stats_reset()
    yield
    torch.cuda.synchronize()


def same_bits(got, want, what):
    got, want = got.cpu().contiguous(), want.contiguous()
    assert got.shape == want.shape and got.dtype == want.dtype, what
    if got.dtype is F8:
        assert torch.equal(got.view(torch.uint8), want.view(torch.uint8)), what
    else:
        same = (got.view(torch.int32) == want.view(torch.int32)) | (torch.isnan(got) & torch.isnan(want))
        assert bool(same.all()), what


def check_quantize(x):
    q, s = rla.f8_quantize(x.to(DEV))
    want_q, want_s = of.quantize_rows(x)
    same_bits(q, want_q, "q")
    same_bits(s, want_s, "scale")
    q, s, t, st = rla.f8_quantize(x.to(DEV), turned=True)
    same_bits(q, want_q, "q of both")
    same_bits(s, want_s, "scale of both")
    want_t, want_st = of.quantize_rows(x.t().contiguous())
    same_bits(t, want_t, "turned q")
    same_bits(st, want_st, "turned scale")
    return q, s, t, st


def check_weight(w):
    want_q, want_s = of.quantize(w, 128)
    q, s = rla.f8_quantize_weight(w.to(DEV))
    same_bits(q, want_q, "q")
    same_bits(s, want_s, "scale")
    q, s, t, st = rla.f8_quantize_weight(w.to(DEV), turned=True)
    for got, want, what in ((q, want_q, "q of both"), (s, want_s, "scale of both"), (t, want_q.t(), "turned q"),
                            (st, want_s.t(), "turned scale")):
        same_bits(got, want, what)


SHAPES = [(1, 1), (3, 7), (1, 4096), (5, 127), (2, 128), (4, 129), (127, 8), (128, 128), (129, 136), (7, 1000),
          (300, 264), (33, 2053), (2, 10240), (257, 520), (1000, 24), (16, 255), (640, 16)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,dim", SHAPES)
def test_quantize(rows, dim, dtype):
    g = torch.Generator().manual_seed(dim)
    x = randn(g, rows, dim, std=3.0)
    check_quantize((x * torch.exp(randn(g, dim, std=2.0))).to(dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,dim", SHAPES)
def test_quantize_weight(rows, dim, dtype):
    check_weight(randn(torch.Generator().manual_seed(rows), rows, dim, std=0.02, dtype=dtype))


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_special_blocks(dtype):
    g = torch.Generator().manual_seed(2)
    for dim in (384, 390):
        x = randn(g, 140, dim, dtype=dtype)
        x[1] = 0
        x[2, 17] = float("nan")
        x[3, 130] = float("inf")
        x[4, 299] = float("-inf")
        x[5] *= 1e-38  # subnormal scales
        x[6] *= 1e30
        x[7] *= 1e-44
        x[8] = -0.0
        x[9, :128] = torch.where(torch.arange(128) % 2 == 0, 448.0, 1.0).to(dtype) * torch.linspace(0.001, 1, 128).to(dtype)
        x[9, 0] = 448.0  # a scale of 1: ties of e4m3 itself
        x[9, 1:128] = ((torch.arange(1, 128) + 0.5) * 2.0 ** -4).to(dtype)
        x[10, :] = 3e38
        check_quantize(x)
        w = randn(g, 300, dim, dtype=dtype)
        w[140, 200] = float("nan")
        w[10, 5] = float("inf")
        w[:128, 256:] = 0
        w[256:, :128] *= 1e-40
        check_weight(w)


def test_quantize_every_tie():
    """Blocks with a scale of 1 that hold every e4m3 value, every middle between two and its neighbours in fp32."""
    v = torch.arange(0, 0x7f, dtype=torch.uint8).view(F8).float()
    mid = (v[1:] + v[:-1]) / 2
    x = torch.cat([v, mid, torch.nextafter(mid, torch.tensor(0.0)), torch.nextafter(mid, torch.tensor(1e9))])
    x = torch.cat([x, -x])
    x = torch.nn.functional.pad(x, (0, -x.numel() % 127)).view(-1, 127)
    x = torch.cat([torch.full((x.shape[0], 1), 448.0), x], 1)
    check_quantize(x)
    check_quantize(x * 2.0 ** -90)  # beside the usual range of scales
    check_quantize(x * 2.0 ** 110)


def test_scales_and_quotients_round_like_divisions():
    """Largest magnitudes over all exponents and significands, those whose scale is all ones or a power of two
    among them, and other numbers at random ratios to them: as columns and as rows."""
    g = torch.Generator().manual_seed(9)
    n = 1 << 13
    top = torch.randint(0x00800000, 0x7f000000, (n,), generator=g, dtype=torch.int32)
    top[: n // 2] = torch.randint(0x30000000, 0x50000000, (n // 2,), generator=g, dtype=torch.int32)
    top = top.view(torch.float32)
    # scales of all ones, and one step beside
    ones = (torch.arange(40, 240, dtype=torch.int32) * 0x800000 + 0x7fffff).view(torch.float32) * 448.0
    near = torch.cat([torch.nextafter(ones, torch.zeros(())), ones, torch.nextafter(ones, torch.full((), 3e38))])
    top[100:100 + near.numel()] = near.clamp(max=3e38)
    x = top[:, None] * torch.rand(n, 128, generator=g) ** 2
    x[torch.arange(n), torch.randint(0, 128, (n,), generator=g)] = top
    check_quantize(x)
    check_quantize(x.t().contiguous())


def test_unaligned_and_offset_inputs():
    for dtype in TYPES:
        x = randn(torch.Generator().manual_seed(1), 150, 256, dtype=dtype)
        buf = torch.empty(x.numel() + 1, dtype=dtype, device=DEV)[1:].view(x.shape)
        buf.copy_(x)
        q, s, t, st = rla.f8_quantize(buf, turned=True)
        want = of.quantize_rows(x)
        same_bits(q, want[0], "q")
        same_bits(t, of.quantize_rows(x.t().contiguous())[0], "t")


def check_matmul(a, sa, b, sb, bias, dtype, exact=False):
    dev = [None if v is None else v.to(DEV) for v in (a, sa, b, sb, bias)]
    y = rla.f8_matmul(*dev[:4], bias=dev[4], dtype=dtype)
    assert y.dtype == dtype
    want, mag = of.matmul(a, sa, b, sb, bias)
    if exact:
        assert torch.equal(y.cpu(), want.to(dtype))
        if dtype is torch.float32:
            assert torch.equal(rla.f8_matmul(*dev[:4], bias=dev[4]).cpu(), want.bfloat16())
        return y
    M, K = a.shape
    tol = (2 * 128 + 4 + -(-K // 128) + 17) * U * mag
    if M > 16 and dtype is torch.bfloat16:
        rows = 1 if b.shape[0] == 1 or sb.shape[0] == b.shape[0] else 128
        largest = lambda t, s, r: torch.nn.functional.pad(  # noqa: E731
            t.double().abs() * of.spread(s, *t.shape, r), (0, -K % 8)).view(t.shape[0], -1, 8).amax(2)
        tol = tol + 7 * 2.0 ** -13 * (largest(a, sa, 1) @ largest(b, sb, rows).t())
    assert_within(y, want, tol + half_step(dtype) * (want.abs() + tol) + tiny(dtype), "y")
    return y


def integers(M, K, N, seed, b_rows, bias):
    """Integers up to 8 and scales of 1/2, 1 and 2: every sum is a multiple of 1/4 below 2^22."""
    g = torch.Generator().manual_seed(seed)
    blocks = -(-K // 128)
    a = torch.randint(-8, 9, (M, K), generator=g).float().to(F8)
    b = torch.randint(-8, 9, (N, K), generator=g).float().to(F8)
    power = lambda *s: 2.0 ** torch.randint(-1, 2, s, generator=g).float()  # noqa: E731
    sa, sb = power(M, blocks), power(N if b_rows else -(-N // 128), blocks)
    return a, sa, b, sb, torch.randint(-9, 10, (N,), generator=g).float() if bias else None


@pytest.mark.parametrize("b_rows", [False, True])
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9, 16, 17, 40, 64, 65, 127, 128, 130, 300])
def test_token_counts(M, b_rows):
    check_matmul(*integers(M, 272, 140, M, b_rows, M % 2 == 0), torch.float32, True)
    check_matmul(*integers(M, 2000, 300, M, b_rows, M % 2 == 1), torch.float32, True)


@pytest.mark.parametrize("M", [1, 4, 9, 30, 100, 300])
@pytest.mark.parametrize("K", [1, 2, 3, 4, 15, 16, 17, 64, 100, 127, 128, 129, 200, 255, 256, 257, 512, 1000, 4100, 8192, 8195])
def test_depths(K, M):
    for b_rows in (False, True):
        check_matmul(*integers(M, K, 70, K, b_rows, False), torch.float32, True)


@pytest.mark.parametrize("M", [1, 4, 9, 30, 100, 300])
@pytest.mark.parametrize("N", [1, 2, 3, 5, 15, 16, 17, 63, 64, 127, 128, 129, 260, 513])
def test_output_widths(N, M):
    for b_rows in (False, True):
        check_matmul(*integers(M, 160, N, N, b_rows, True), torch.float32, True)


@pytest.mark.parametrize("b_rows", [False, True])
@pytest.mark.parametrize("M,K,N", [(4096, 144, 3328), (4095, 400, 3329), (2048, 1040, 2050), (1024, 2064, 1090),
                                   (512, 3008, 640), (700, 4112, 900), (257, 6160, 300), (140, 8208, 520), (8192, 272, 1000),
                                   (5000, 1290, 515), (300, 5001, 700)])
def test_tiles(M, K, N, b_rows):
    """Every tile, whole and split, aligned and not."""
    check_matmul(*integers(M, K, N, M + K, b_rows, True), torch.float32, True)


@pytest.mark.parametrize("b_rows", [False, True])
@pytest.mark.parametrize("M,K,N", [(4095, 401, 3329), (2048, 1041, 2050), (4095, 4672, 576), (4095, 4673, 576),
                                   (1000, 8195, 100)])
def test_tiles_of_rows_further_apart(M, K, N, b_rows):
    """Wide tiles, whole and split, whose rows start on 16 bytes and end anywhere; NaN between the rows."""
    a, sa, b, sb, bias = integers(M, K, N, K, b_rows, True)
    want = of.matmul(a, sa, b, sb, bias)[0]

    def wide(t):
        v = torch.full((t.shape[0], -(-K // 16) * 16 + 16), 0x7f, dtype=torch.uint8, device=DEV).view(F8)
        v.view(torch.uint8)[:, :K] = t.to(DEV).view(torch.uint8)
        return v[:, :K]

    for dtype in TYPES:
        y = rla.f8_matmul(wide(a), sa.to(DEV), wide(b), sb.to(DEV), bias=bias.to(DEV), dtype=dtype)
        assert torch.equal(y.cpu(), want.to(dtype))


@pytest.mark.parametrize("b_rows", [False, True])
def test_the_widest_tiles_split(b_rows):
    """So few outputs of so deep a product that tiles of 256 x 256 are split; sums stay below 2^22 steps of 1/4."""
    M, K, N = 256, 131072, 4096
    a, sa, b, sb, bias = (v.to(DEV) for v in integers(M, K, N, 1, b_rows, True))
    x = a.double() * sa.double().repeat_interleave(128, 1)
    want = torch.cat([x @ (b[n:n + 1024].double() * (sb[n:n + 1024] if b_rows else sb[n // 128:n // 128 + 8].repeat_interleave(
        128, 0)).double().repeat_interleave(128, 1)).t().contiguous() for n in range(0, N, 1024)], 1) + bias.double()
    assert float(want.abs().max()) < 2.0 ** 20
    for dtype in TYPES:
        y = rla.f8_matmul(a, sa, b, sb, bias=bias, dtype=dtype)
        assert torch.equal(y, want.to(dtype))


def random_operands(M, K, N, seed, b_rows=False, bias=True):
    g = torch.Generator().manual_seed(seed)
    a, sa = of.quantize_rows(randn(g, M, K) * torch.exp(randn(g, K)))
    b, sb = (of.quantize_rows if b_rows else lambda t: of.quantize(t, 128))(randn(g, N, K, std=K ** -0.5))
    return a, sa, b, sb, randn(g, N) if bias else None


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("b_rows", [False, True])
@pytest.mark.parametrize("M,K,N", [(1, 4096, 512), (7, 1111, 130), (33, 2064, 257), (200, 4100, 300), (1000, 1024, 640),
                                   (2050, 528, 2300)])
def test_quantised_data(M, K, N, b_rows, dtype):
    check_matmul(*random_operands(M, K, N, M, b_rows), dtype)


def test_largest_values():
    """Every operand at 448 over long rows, and the smallest subnormal against it."""
    for M in (3, 40, 300):
        a, b = torch.full((M, 3000), 448.0).to(F8), torch.full((5, 3000), 448.0).to(F8)
        b[1] = torch.tensor(2.0 ** -9).to(F8)
        b[2] = (-b[2].float()).to(F8)
        b[3, ::2] = torch.tensor(-448.0).to(F8)
        sa, sb = torch.full((M, 24), 2.0 ** -10), torch.full((1, 24), 0.5)
        check_matmul(a, sa, b, sb, None, torch.float32)


def test_rows_further_apart():
    """Operands with a row pitch; what lies between rows is never used, whatever it holds."""
    for M, K, N in ((3, 130, 20), (100, 200, 70), (100, 1001, 300), (300, 4100, 520), (600, 135, 900)):
        a, sa, b, sb, bias = integers(M, K, N, K, False, True)
        want = check_matmul(a, sa, b, sb, bias, torch.float32, True)
        for pitch in (K + 1, -(-K // 16) * 16, -(-K // 128) * 128 + 128):
            def wide(t):
                v = torch.full((t.shape[0], pitch), 0x7f, dtype=torch.uint8, device=DEV).view(F8)  # NaN
                v.view(torch.uint8)[:, :K] = t.to(DEV).view(torch.uint8)
                return v[:, :K]
            y = rla.f8_matmul(wide(a), sa.to(DEV), wide(b), sb.to(DEV), bias=bias.to(DEV), dtype=torch.float32)
            assert torch.equal(y, want), (M, K, N, pitch)
        shifted = torch.empty(M * K + 1, dtype=torch.uint8, device=DEV)[1:].view(M, K)
        shifted.copy_(a.to(DEV).view(torch.uint8))
        y = rla.f8_matmul(shifted.view(F8), sa.to(DEV), b.to(DEV), sb.to(DEV), bias=bias.to(DEV), dtype=torch.float32)
        assert torch.equal(y, want)


def test_a_block_that_is_not_finite():
    for M in (4, 80, 300):
        g = torch.Generator().manual_seed(3)
        x, w = randn(g, M, 300), randn(g, 200, 300)
        b, sb = rla.f8_quantize_weight(w.to(DEV))
        x[1, 3], x[2, 299] = float("nan"), float("inf")
        q, s = rla.f8_quantize(x.to(DEV))
        y = rla.f8_matmul(q, s, b, sb, dtype=torch.float32)
        assert torch.isnan(y[1]).all() and torch.isnan(y[2]).all()
        assert torch.isfinite(y[0]).all() and torch.isfinite(y[3:]).all()
        w[130, 5] = float("inf")
        b, sb = rla.f8_quantize_weight(w.to(DEV))
        y = rla.f8_matmul(q[3:], s[3:], b, sb, dtype=torch.float32)
        assert torch.isfinite(y[:, :128]).all() and torch.isnan(y[:, 128:]).all()


@pytest.mark.parametrize("M,K,N", [(256, 384, 512), (300, 200, 130), (77, 1000, 333), (17, 64, 2000), (1000, 520, 264)])
def test_a_training_step(M, K, N):
    """y and both gradients from the turned operands: each is the product of what the quantisers made."""
    g = torch.Generator().manual_seed(M)
    x, w, dy = randn(g, M, K, dtype=torch.bfloat16), randn(g, N, K, std=0.05, dtype=torch.bfloat16), \
        randn(g, M, N, dtype=torch.bfloat16)
    xq, xs, xt, xts = rla.f8_quantize(x.to(DEV), turned=True)
    wq, ws, wt, wts = rla.f8_quantize_weight(w.to(DEV), turned=True)
    dq, ds, dt, dts = rla.f8_quantize(dy.to(DEV), turned=True)
    cpu = lambda *t: [v.cpu().contiguous() for v in t]  # noqa: E731
    for a, b, what in (((xq, xs), (wq, ws), "y"), ((dq, ds), (wt, wts), "dx"), ((dt, dts), (xt, xts), "dw")):
        got = rla.f8_matmul(*a, *b, dtype=torch.float32)
        want, mag = of.matmul(*cpu(*a), *cpu(*b), None)
        blocks = a[1].shape[1]
        assert_within(got, want, (2 * 128 + 4 + blocks + 17) * U * mag + tiny(torch.float32), what)
    # and near the product of what they were made from: each operand is off by half a step of e4m3, 2^-4 of
    # a value (2^-10 of its block's largest for values that are subnormal), and each scale by 2^-24
    full = lambda t: d(t)  # noqa: E731
    got = rla.f8_matmul(dq, ds, wt, wts, dtype=torch.float32)
    want = full(dy) @ full(w)
    slack = (full(dy).abs() + 6.0 / 448) @ (full(w).abs() + 0.3 / 448) * (2 * 2.0 ** -4 + 2.0 ** -8 + 1e-4)
    assert_within(got, want, slack, "dx against the unrounded product")


def test_leading_dimensions_out_and_empty():
    a, sa, b, sb, _ = (None if v is None else v.to(DEV) for v in integers(6, 200, 20, 4, False, False))
    y = rla.f8_matmul(a, sa, b, sb)
    assert y.dtype is torch.bfloat16
    big = torch.full((8, 20), 7.0, dtype=torch.bfloat16, device=DEV)
    rla.f8_matmul(a, sa, b, sb, out=big[1:7])
    assert torch.equal(big[1:7], y) and bool((big[0] == 7).all()) and bool((big[7] == 7).all())
    assert torch.equal(rla.f8_matmul(a.view(2, 3, 200), sa.view(2, 3, 2), b, sb).view(6, 20), y)
    assert rla.f8_matmul(a[:0], sa[:0], b, sb).shape == (0, 20)
    assert rla.f8_matmul(a, sa, b[:0], sb[:0]).shape == (6, 0)
    q, s = rla.f8_quantize(torch.empty(0, 200, device=DEV))
    assert q.shape == (0, 200) and s.shape == (0, 2)
    x = randn(torch.Generator().manual_seed(1), 2, 3, 300).to(DEV)
    q, s = rla.f8_quantize(x)
    q2, s2 = rla.f8_quantize(x.view(6, 300))
    assert q.shape == x.shape and s.shape == (2, 3, 3) and torch.equal(s.view(6, 3), s2)
    assert torch.equal(q.view(torch.uint8).view(6, 300), q2.view(torch.uint8))


def test_scales_of_any_strides():
    """Scales row by row, block by block, inside wider tensors and spread out: the same bits."""
    for M, K, N in ((3, 300, 40), (100, 1000, 70), (600, 520, 300)):
        for b_rows in (False, True):
            a, sa, b, sb, _ = (None if v is None else v.to(DEV) for v in integers(M, K, N, K, b_rows, False))
            want = rla.f8_matmul(a, sa, b, sb, dtype=torch.float32)
            turned = lambda t: t.t().contiguous().t()  # noqa: E731
            wide = lambda t: torch.full((t.shape[0] + 2, t.shape[1] * 2 + 5), float("nan"), device=DEV)[  # noqa: E731
                1:-1, 3:3 + 2 * t.shape[1]:2].copy_(t)
            for f in (turned, wide, lambda t: turned(wide(t))):
                for d16 in (torch.float32, torch.bfloat16):
                    got = rla.f8_matmul(a, f(sa), b, f(sb), dtype=d16)
                    assert torch.equal(got, want.to(d16)), (M, b_rows)
            assert torch.equal(rla.f8_matmul(a, sa[:, :1].expand(-1, sa.shape[1]), b, sb, dtype=torch.float32),
                               rla.f8_matmul(a, sa[:, :1].repeat(1, sa.shape[1]), b, sb, dtype=torch.float32))
    x = randn(torch.Generator().manual_seed(1), 70, 300).to(DEV)
    q, s = rla.f8_quantize(x)
    out = torch.full((70, 5), 7.0, device=DEV)
    q2, s2 = rla.f8_quantize(x, scale_out=out[:, 1:4])
    assert torch.equal(s, s2) and bool((out[:, 0] == 7).all()) and bool((out[:, 4] == 7).all())


def test_the_stride_of_one_row():
    """One token, one row of weights' scales: their row strides are any numbers."""
    a, sa, b, sb, _ = (None if v is None else v.to(DEV) for v in integers(1, 400, 70, 6, False, False))
    want = rla.f8_matmul(a, sa, b, sb)
    far = lambda v: v.as_strided(v.shape, (1 << 40, 1))  # noqa: E731
    assert torch.equal(rla.f8_matmul(a, far(sa), b, far(sb)), want)
    x = torch.randn(1, 400, device=DEV)
    q, s = rla.f8_quantize(x)
    given = torch.empty_like(s)
    rla.f8_quantize(x, scale_out=far(given))
    assert torch.equal(given, s)


def test_outputs_that_are_given():
    x = randn(torch.Generator().manual_seed(1), 5, 200, dtype=torch.bfloat16).to(DEV)
    want = rla.f8_quantize(x)
    q, s = torch.zeros(7, 200, dtype=torch.uint8, device=DEV).view(F8), torch.full((7, 2), 7.0, device=DEV)
    rla.f8_quantize(x, q_out=q[1:6], scale_out=s[1:6])
    assert torch.equal(q[1:6].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(s[1:6], want[1])
    assert bool((s[0] == 7).all()) and bool((s[6] == 7).all()) and not bool(q.view(torch.uint8)[0].any())


def test_equal_calls_give_equal_bits():
    a, sa, b, sb, _ = (None if v is None else v.to(DEV) for v in random_operands(100, 8192, 64, 3, bias=False))
    ys = [rla.f8_matmul(a, sa, b, sb, dtype=torch.float32) for _ in range(4)]
    assert all(torch.equal(ys[0], y) for y in ys[1:])


def test_other_stream_and_graph():
    x = randn(torch.Generator().manual_seed(1), 70, 4101).to(DEV)
    w = randn(torch.Generator().manual_seed(2), 50, 4101).to(DEV)

    def step(stream=None):
        q = rla.f8_quantize(x, turned=True, stream=stream)
        b = rla.f8_quantize_weight(w, turned=True, stream=stream)
        y = rla.f8_matmul(*q[:2], *b[:2], stream=stream)  # sums split: a workspace
        return [t.view(torch.uint8) if t.dtype is F8 else t for t in q + b] + [y]

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    for u, v in zip(want, got):
        assert torch.equal(u, v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(4):
        x.copy_(randn(torch.Generator().manual_seed(10 + i), 70, 4101))
        w.copy_(randn(torch.Generator().manual_seed(20 + i), 50, 4101))
        eager = step()
        graph.replay()
        torch.cuda.synchronize()
        for u, v in zip(eager, outs):
            assert torch.equal(u, v), i


def test_refusals_on_the_device():
    a, sa, b, sb, _ = (None if v is None else v.to(DEV) for v in integers(3, 200, 150, 6, False, False))

    def refused(reason, f):
        with pytest.raises(rla.Ltx3dRopeUnsupported) as e:
            f()
        assert e.value.reason == reason, e.value.reason

    refused("DTYPE", lambda: rla.f8_matmul(a.float(), sa, b, sb))
    refused("DTYPE", lambda: rla.f8_matmul(a, sa, b.view(torch.int8), sb))
    refused("DTYPE", lambda: rla.f8_matmul(a, sa, b, sb, dtype=torch.float16))
    refused("DTYPE", lambda: rla.f8_quantize(sa.half()))
    refused("SHAPE_MISMATCH", lambda: rla.f8_matmul(a, sa, b[:, :100].contiguous(), sb))
    refused("SHAPE_MISMATCH", lambda: rla.f8_matmul(a, sa[:2], b, sb))
    refused("SHAPE_MISMATCH", lambda: rla.f8_matmul(a, sa[:, :1], b, sb))
    refused("SHAPE_MISMATCH", lambda: rla.f8_matmul(a, sa, b, sb[:1]))
    refused("SHAPE_MISMATCH", lambda: rla.f8_quantize(torch.zeros(2, 3, 4, device=DEV), turned=True))
    refused("SHAPE_MISMATCH", lambda: rla.f8_quantize_weight(torch.zeros(4, device=DEV)))
    refused("NOT_CONTIGUOUS", lambda: rla.f8_matmul(a, sa, b.view(torch.uint8).t().contiguous().t().view(F8), sb))
    refused("NOT_CONTIGUOUS", lambda: rla.f8_quantize(torch.zeros(4, 4, device=DEV).t()))
    refused("NOT_DEVICE_PTR", lambda: rla.f8_matmul(a, sa, b.cpu(), sb))
    refused("NOT_DEVICE_PTR", lambda: rla.f8_quantize(torch.zeros(4, 4)))
    assert rla.stats()["fast_launches"] == 0


def test_more_than_two_to_the_32_elements():
    """Outputs and inputs beyond 2^32 elements: the last rows against the same rows alone."""
    M, K, N = 70001, 144, 65536
    a, sa, b, sb, _ = (None if v is None else v.to(DEV) for v in integers(M, K, N, 5, False, False))
    y = rla.f8_matmul(a, sa, b, sb)
    for lo in (0, 40000, M - 300):
        assert torch.equal(y[lo:lo + 300], rla.f8_matmul(a[lo:lo + 300], sa[lo:lo + 300], b, sb))
    q, s, t, st = rla.f8_quantize(y, turned=True)
    lo = M // 128 * 128 - 128
    part = rla.f8_quantize(y[lo:], turned=True)
    assert torch.equal(q[lo:].view(torch.uint8), part[0].view(torch.uint8)) and torch.equal(s[lo:], part[1])
    assert torch.equal(t[:, lo:].contiguous().view(torch.uint8), part[2].contiguous().view(torch.uint8))
    assert torch.equal(st[:, lo // 128:], part[3])
    q2, s2 = rla.f8_quantize(y)
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)
