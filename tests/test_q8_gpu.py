"""The 8-bit linear layer on the GPU against oracle.block: the quantiser bit for bit, the product's
integer sums exactly, and its fp32 scaling within three roundings and the output's own."""
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
TYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(autouse=True)
def fresh():
    assert torch.cuda.is_available()
    _lib.lib()
    rla.stats_reset()
    yield
    torch.cuda.synchronize()


def check_quantize(x):
    q, s = rla.q8_quantize(x.to(DEV))
    want_q, want_s = ob.q8_quantize(x)
    same = (s.cpu().view(torch.int32) == want_s.view(torch.int32)) | (torch.isnan(s.cpu()) & torch.isnan(want_s))
    assert bool(same.all())
    assert torch.equal(q.cpu(), want_q)
    return q, s


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,dim", [(1, 1), (3, 7), (1, 4096), (5, 63), (2, 255), (4, 256), (7, 1000), (33, 2053),
                                      (2, 10240), (1, 40001), (70000, 8)])
def test_quantize(rows, dim, dtype):
    check_quantize(randn(torch.Generator().manual_seed(dim), rows, dim, std=3.0, dtype=dtype))


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_special_rows(dtype):
    g = torch.Generator().manual_seed(2)
    x = randn(g, 10, 300, dtype=dtype)
    x[1] = 0
    x[2, 17] = float("nan")
    x[3, 0] = float("inf")
    x[4, 299] = float("-inf")
    x[5] *= 1e-38  # a subnormal scale
    x[6] *= 1e30
    x[7] = 127.0 * torch.sign(x[7].float()).to(dtype)  # ties between steps: halves of a step of 1
    x[7, :100] = torch.arange(100).to(dtype) + 0.5
    x[8] = -0.0
    check_quantize(x)


def check_matmul(a, sa, b, sb, bias, dtype):
    dev = [None if v is None else v.to(DEV) for v in (a, sa, b, sb, bias)]
    y = rla.q8_matmul(*dev[:4], bias=dev[4], dtype=dtype)
    assert y.dtype == dtype
    want = ob.q8_matmul(a, sa, b, sb, bias)
    scaled = (want if bias is None else want - bias.double()).abs()
    tol = 4 * U * (scaled + (0 if bias is None else bias.double().abs()))
    assert_within(y, want, tol + half_step(dtype) * (want.abs() + tol) + tiny(dtype), "y")
    return y


def operands(M, K, N, seed, bias=True):
    g = torch.Generator().manual_seed(seed)
    a = torch.randint(-127, 128, (M, K), generator=g, dtype=torch.int8)
    b = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int8)
    sa, sb = torch.rand(M, generator=g) * 0.02 + 1e-3, torch.rand(N, generator=g) * 0.01 + 1e-4
    return a, sa, b, sb, randn(g, N) if bias else None


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 16, 17, 40, 64, 65, 127, 128, 130, 300])
def test_token_counts(M, dtype):
    check_matmul(*operands(M, 272, 140, M, M % 2 == 0), dtype)


@pytest.mark.parametrize("M", [1, 4, 9, 30, 100])
@pytest.mark.parametrize("K", [1, 2, 15, 16, 17, 64, 100, 127, 128, 129, 512, 1000, 4100])
def test_depths(K, M):
    check_matmul(*operands(M, K, 70, K), torch.float32)


@pytest.mark.parametrize("M", [1, 4, 9, 30, 100])
@pytest.mark.parametrize("N", [1, 2, 3, 5, 15, 16, 17, 63, 64, 127, 128, 129, 260])
def test_output_widths(N, M):
    check_matmul(*operands(M, 160, N, N), torch.bfloat16)


def test_large_tiles():
    check_matmul(*operands(4096, 144, 3328, 1), torch.bfloat16)
    check_matmul(*operands(4095, 100, 3329, 2), torch.float32)


@pytest.mark.parametrize("M", [1, 3, 7, 65])
def test_longest_sums(M):
    """Every product at its largest over the longest row that is taken: the sums stay within 32 bits."""
    K = 131071
    a = torch.full((M, K), -128, dtype=torch.int8)
    b = torch.full((3, K), -128, dtype=torch.int8)
    b[1] = 127
    b[2, ::2] = 127
    check_matmul(a, torch.full((M,), 0.5), b, torch.full((3,), 0.25), None, torch.float32)


def test_unaligned_operands():
    for M in (1, 3, 7, 100):
        a, sa, b, sb, bias = operands(M, 256, 64, 8)
        want = check_matmul(a, sa, b, sb, bias, torch.float32)

        def shifted(v):
            t = torch.empty(v.numel() + 1, dtype=v.dtype, device=DEV)[1:].view(v.shape)
            t.copy_(v)
            return t

        y = rla.q8_matmul(shifted(a), sa.to(DEV), shifted(b), sb.to(DEV), bias=bias.to(DEV), dtype=torch.float32)
        assert torch.equal(y, want)


def test_a_row_that_is_not_finite():
    for M in (4, 80):
        g = torch.Generator().manual_seed(3)
        x = randn(g, M, 64)
        _, _, b, sb, _ = operands(1, 64, 32, 1)
        x[1, 3] = float("nan")
        x[2, 5] = float("inf")
        q, s = rla.q8_quantize(x.to(DEV))
        y = rla.q8_matmul(q, s, b.to(DEV), sb.to(DEV), dtype=torch.float32)
        assert torch.isnan(y[1]).all() and torch.isnan(y[2]).all()
        assert torch.isfinite(y[0]).all() and torch.isfinite(y[3:]).all()


def test_leading_dimensions_out_and_empty():
    a, sa, b, sb, _ = (None if v is None else v.to(DEV) for v in operands(6, 64, 20, 4, False))
    y = rla.q8_matmul(a, sa, b, sb)
    big = torch.full((8, 20), 7.0, dtype=torch.bfloat16, device=DEV)
    rla.q8_matmul(a, sa, b, sb, out=big[1:7])
    assert torch.equal(big[1:7], y) and bool((big[0] == 7).all()) and bool((big[7] == 7).all())
    assert torch.equal(rla.q8_matmul(a.view(2, 3, 64), sa.view(2, 3), b, sb).view(6, 20), y)
    assert rla.q8_matmul(a[:0], sa[:0], b, sb).shape == (0, 20)
    assert rla.q8_matmul(a, sa, b[:0], sb[:0]).shape == (6, 0)
    q, s = rla.q8_quantize(torch.empty(0, 64, device=DEV))
    assert q.shape == (0, 64) and s.shape == (0,)


def test_other_stream_and_graph():
    a, sa, b, sb, bias = (v.to(DEV) for v in operands(70, 4101, 50, 5))  # sums split: a workspace
    x = randn(torch.Generator().manual_seed(1), 70, 4101).to(DEV)

    def step(stream=None):
        q, s = rla.q8_quantize(x, stream=stream)
        return q, s, rla.q8_matmul(q, s, b, sb, bias=bias, stream=stream)

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
        eager = step()
        graph.replay()
        torch.cuda.synchronize()
        for u, v in zip(eager, outs):
            assert torch.equal(u, v), i


def test_refusals_on_the_device():
    a, sa, b, sb, _ = (None if v is None else v.to(DEV) for v in operands(3, 64, 8, 6, False))

    def refused(reason, f):
        with pytest.raises(rla.Ltx3dRopeUnsupported) as e:
            f()
        assert e.value.reason == reason

    refused("DTYPE", lambda: rla.q8_matmul(a.float(), sa, b, sb))
    refused("DTYPE", lambda: rla.q8_matmul(a, sa, b, sb, dtype=torch.float16))
    refused("DTYPE", lambda: rla.q8_quantize(sa.view(1, 3).half()))
    refused("SHAPE_MISMATCH", lambda: rla.q8_matmul(a, sa, b[:, :32].contiguous(), sb))
    refused("SHAPE_MISMATCH", lambda: rla.q8_matmul(a, sa[:2], b, sb))
    refused("NOT_CONTIGUOUS", lambda: rla.q8_matmul(a, sa, b[:, :].t().contiguous().t(), sb))
    refused("NOT_DEVICE_PTR", lambda: rla.q8_matmul(a, sa, b.cpu(), sb))
    wide = torch.zeros(2, 131072, dtype=torch.int8, device=DEV)
    refused("TOO_LARGE", lambda: rla.q8_matmul(wide, sa[:2], wide, sb[:2]))
    assert rla.stats()["fast_launches"] == 0


def test_block_in_a_row():
    """norm_before -> gated_ffn -> 8-bit down projection -> norm_after, each stage against 64 bits on
    the stage before's own output, eagerly and from a graph."""
    B, S, D, F, eps = 2, 37, 256, 520, 1e-6
    for rows in (1, S):  # single tokens and a prompt
        g = torch.Generator().manual_seed(7)
        bf = torch.bfloat16
        x = randn(g, B, rows, D, std=2.0, dtype=bf).to(DEV)
        w1, w2 = (randn(g, D, std=0.1).to(DEV) for _ in range(2))
        scale, shift, gate = (randn(g, B, D, std=0.3).to(DEV) for _ in range(3))
        wg, wu = (randn(g, F, D, std=1 / math.sqrt(D), dtype=bf).to(DEV) for _ in range(2))
        wd, sd = rla.q8_quantize(randn(g, D, F, std=1 / math.sqrt(F)).to(DEV))

        def block(x):
            n = rla.norm_before(x, w1, scale, shift, eps=eps, weight_offset=1.0)
            h = rla.gated_ffn(n, wg, wu, "gelu_tanh")
            q, s = rla.q8_quantize(h)
            y = rla.q8_matmul(q, s, wd, sd)
            r, n2 = rla.norm_after(y, x, w2, gate, next_weight=w1, next_scale=scale, next_shift=shift, eps=eps,
                                   weight_offset=1.0)
            return n, h, q, s, y, r, n2

        def check(x, outs):
            n, h, q, s, y, r, n2 = outs
            hs = half_step(bf)
            want = ob.norm_before(d(x), d(w1), d(scale), d(shift), eps, 1.0)
            mag = want.abs() + d(shift).abs()[:, None, :] * 2
            assert_within(n, want, 40 * U * mag + hs * want.abs() + tiny(bf), "n")
            nn, hh = d(n).view(-1, D), d(h).view(-1, F)
            want, gg, uu = ob.gated_ffn(nn, d(wg), d(wu), "gelu_tanh")
            e = 2 * (D + 2) * U
            tol = e * (1.2 * (nn.abs() @ d(wg).abs().T) * (uu.abs() + 1) + gg.abs() * (nn.abs() @ d(wu).abs().T))
            tol = tol + (1.6 * gg.abs() + 0.08 * gg.abs() ** 3 + 16) * U * (gg * uu).abs()
            assert_within(hh, want, tol + hs * (want.abs() + tol) + tiny(bf), "h")
            wq, ws = ob.q8_quantize(h.cpu())
            assert torch.equal(q.cpu(), wq) and torch.equal(s.cpu(), ws)
            want = ob.q8_matmul(q.cpu().view(-1, F), s.cpu().view(-1), wd.cpu(), sd.cpu(), None)
            assert_within(y.view(-1, D), want, (4 * U + hs) * 1.001 * want.abs() + tiny(bf), "y")
            want = ob.norm_after(d(y), d(x), d(w2), d(gate), True, 1.0, eps, 1.0)
            tol = 40 * U * (want - d(x)).abs() + 40 * U * d(x).abs()
            assert_within(r, want, tol + hs * want.abs() + tiny(bf), "r")
            inv = ob.rstd(want, eps)
            f = ob.norm_factor(d(w1), d(scale), 1.0, want).abs()
            hat = (want * inv).abs()
            moved = f * (inv * tol + hat * (hat * inv * tol).mean(-1, keepdim=True))
            want2 = ob.norm_before(want, d(w1), d(scale), d(shift), eps, 1.0)
            mag = hat * f + d(shift).abs()[:, None, :]
            assert_within(n2, want2, moved + 40 * U * mag + hs * want2.abs() + tiny(bf), "n2")

        check(x, block(x))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = block(x)
        for i in range(3):
            x.copy_(randn(torch.Generator().manual_seed(20 + i), B, rows, D, std=2.0, dtype=bf))
            eager = block(x)
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(eager, outs):
                assert torch.equal(a, b)
            check(x, outs)


@pytest.mark.parametrize("dtype,dim", [(torch.bfloat16, 16384), (torch.bfloat16, 16392), (torch.bfloat16, 20480),
                                       (torch.bfloat16, 32768), (torch.bfloat16, 32776), (torch.float32, 8192),
                                       (torch.float32, 8196), (torch.float32, 16384), (torch.float32, 16388)])
def test_quantize_wide_rows(dtype, dim):
    """Two vectors a thread, four, and rows that are read twice; the largest magnitude in the last column too."""
    x = randn(torch.Generator().manual_seed(dim), 5, dim, dtype=dtype)
    x[1, -1] = 40.0
    x[2] = 0
    x[3, dim // 2] = float("inf")
    check_quantize(x)
