"""From the residual stream to rotated queries and keys as a block uses them, and the gradients' way back: the layer
norm after the block before, rows in 8-bit floating point against the weights of one projection of q, k and v, and
the rotation of views of its output.  Each step against float64 on what the step before handed on, within the step's
own bound; the whole on several threads' streams and as a captured graph; many draws of sizes."""
from __future__ import annotations

import random
import threading

import pytest
import torch

import oracle.f8 as of
from tests.block_tools import U, assert_within, half_step, randn, tiny
from tests.test_axes_gpu import check as check_axes
from tests.test_f8_gpu import same_bits
from tests.test_layer_norm_gpu import Case, check_after, check_backward

pytestmark = pytest.mark.gpu

rla = pytest.importorskip("rope_ltx3drope_amd")

DEV = "cuda:0"


class Block:
    def __init__(self, batch, tokens, dim, heads, k_heads, head_dim, dtype, seed, pairing="adjacent", joint=False):
        g = torch.Generator().manual_seed(seed)
        self.case = Case(batch, tokens, dim, dtype, torch.float32, seed)
        self.heads, self.k_heads, self.head_dim, self.pairing = heads, k_heads, head_dim, pairing
        self.cols = (heads + 2 * k_heads) * head_dim
        self.w = randn(g, self.cols, dim, std=dim ** -0.5, dtype=dtype).to(DEV)
        third = head_dim // 8 * 2
        self.freq, self.axis = rla.axes_frequencies([head_dim - 2 * third, third, third], joint=joint, device=DEV)
        grid = torch.arange(tokens)
        self.pos = torch.stack([grid // 60, grid // 10 % 6, grid % 10])[:, None].expand(3, batch, tokens).to(DEV)
        self.dqkv = randn(g, batch, tokens, self.cols, dtype=dtype).to(DEV)
        self.dev = {n: self.case.dev(n) for n in ("y", "residual", "gate", "dr")}
        self.kw = self.case.kw()

    def views(self, t):
        t = t.view(*t.shape[:2], -1, self.head_dim)
        return t[:, :, :self.heads], t[:, :, self.heads:self.heads + self.k_heads]

    def forward(self):
        r, n = rla.layer_norm_after(self.dev["y"], self.dev["residual"], self.dev["gate"], **self.kw)
        rows = n.view(-1, n.shape[-1])
        nq, ns, nt, nts = rla.f8_quantize(rows, turned=True)
        wq, ws, wt, wts = rla.f8_quantize_weight(self.w, turned=True)
        qkv = rla.f8_matmul(nq, ns, wq, ws, dtype=n.dtype).view(*n.shape[:2], -1)
        q, k = self.views(qkv)
        qo, ko = rla.axes_apply_qk(q, k, self.pos, self.freq, self.axis, pairing=self.pairing)
        return r, n, nq, ns, nt, nts, wq, ws, wt, wts, qkv, qo, ko

    def backward(self, f):
        """The gradients of q and k turned back in place, beside v's."""
        r, n, nt, nts, wt, wts = f[0], f[1], f[4], f[5], f[8], f[9]
        d = self.dqkv.clone()
        dq, dk = self.views(d)
        rla.axes_apply_qk_backward(dq, dk, self.pos, self.freq, self.axis, pairing=self.pairing, inplace=True)
        rows = d.view(-1, self.cols)
        gq, gs, gt, gts = rla.f8_quantize(rows, turned=True)
        dn = rla.f8_matmul(gq, gs, wt, wts, dtype=n.dtype).view(n.shape)
        dw = rla.f8_matmul(gt, gts, nt, nts, dtype=torch.float32)
        grads = rla.layer_norm_after_backward(self.dev["dr"], dn, self.dev["y"], r, self.dev["gate"], **self.kw)
        return d, gq, gs, gt, gts, dn, dw, grads


def cpu(*t):
    return [v.cpu().contiguous() for v in t]


def check_product(got, a, sa, b, sb, b_rows):
    """Within the bound of tests/test_f8_gpu.py: the additions of a block, its scales, the blocks' sum and its parts, and
    for bf16 and more than 16 rows seven of each 8 products off by 2^-13 of their largest."""
    a, sa, b, sb = cpu(a, sa, b, sb)
    got = got.reshape(a.shape[0], -1)
    want, mag = of.matmul(a, sa, b, sb, None)
    M, K = a.shape
    tol = (2 * 128 + 4 + -(-K // 128) + 17) * U * mag
    if M > 16 and got.dtype is torch.bfloat16:
        largest = lambda t, s, r: torch.nn.functional.pad(  # noqa: E731
            t.double().abs() * of.spread(s, *t.shape, r), (0, -K % 8)).view(t.shape[0], -1, 8).amax(2)
        tol = tol + 7 * 2.0 ** -13 * (largest(a, sa, 1) @ largest(b, sb, 1 if b_rows else 128).t())
    assert_within(got, want, tol + half_step(got.dtype) * (want.abs() + tol) + tiny(got.dtype), "product")


def check(b):
    f = b.forward()
    r, n, nq, ns, nt, nts, wq, ws, wt, wts, qkv, qo, ko = f
    check_after(b.case, r, n)
    rows = n.cpu().view(-1, n.shape[-1])
    for got, want in zip((nq, ns, nt, nts), (*of.quantize_rows(rows), *of.quantize_rows(rows.t().contiguous()))):
        same_bits(got, want, "rows")
    for got, want in zip((wq, ws), of.quantize(b.w.cpu(), 128)):
        same_bits(got, want, "weights")
    check_product(qkv, nq, ns, wq, ws, False)
    pos, freq, axis = b.pos.cpu(), b.freq.cpu(), b.axis.cpu()
    for x, got in zip(b.views(qkv), (qo, ko)):
        check_axes(x.cpu(), got, pos, freq, axis, b.pairing, False, "rotated")

    d, gq, gs, gt, gts, dn, dw, grads = b.backward(f)
    for x, got in zip(b.views(b.dqkv), b.views(d)):
        check_axes(x.cpu(), got, pos, freq, axis, b.pairing, True, "turned back")
    v = (b.heads + b.k_heads) * b.head_dim
    assert torch.equal(d[..., v:], b.dqkv[..., v:])
    rows = d.cpu().view(-1, b.cols)
    for got, want in zip((gq, gs, gt, gts), (*of.quantize_rows(rows), *of.quantize_rows(rows.t().contiguous()))):
        same_bits(got, want, "gradient rows")
    check_product(dn, gq, gs, wt, wts, False)
    check_product(dw, gt, gts, nt, nts, True)
    b.case.dn = dn.cpu()
    check_backward(b.case, r, dict(res=grads.dresidual, y=grads.dy, gate=grads.dgate, weight=grads.dweight,
                                   bias=grads.dbias, scale=grads.dscale, shift=grads.dshift), True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("batch,tokens,dim,heads,k_heads,head_dim,pairing",
                         [(2, 150, 256, 4, 4, 64, "adjacent"), (1, 1, 512, 8, 2, 64, "halves"),
                          (3, 33, 200, 3, 1, 40, "halves"), (1, 700, 512, 4, 1, 128, "adjacent"),
                          (2, 65, 101, 1, 1, 26, "adjacent")])
def test_block(batch, tokens, dim, heads, k_heads, head_dim, pairing, dtype):
    check(Block(batch, tokens, dim, heads, k_heads, head_dim, dtype, tokens, pairing, joint=k_heads == 1))


@pytest.mark.parametrize("seed", range(12))
def test_drawn_blocks(seed):
    rng = random.Random(seed)
    head_dim = 2 * rng.randrange(4, 70)
    check(Block(rng.randrange(1, 4), rng.randrange(1, 260), rng.randrange(1, 700), rng.randrange(1, 5), rng.randrange(1, 4),
                head_dim, rng.choice([torch.float32, torch.bfloat16]), seed, rng.choice(["adjacent", "halves"])))


def tensors(out):
    for t in out:
        if isinstance(t, torch.Tensor):
            yield t
        elif t is not None:
            yield from tensors(t)


def bits(t):
    return t.contiguous().view(torch.uint8)


def test_threads_on_their_own_streams():
    """No call shares memory with another: results on busy streams are those of each call alone."""
    blocks = [Block(2, 130 + 40 * i, 384, 4, 2, 32, torch.bfloat16, i) for i in range(4)]

    def both(b):
        f = b.forward()
        return list(tensors((*f, *b.backward(f))))

    want = [[t.clone() for t in both(b)] for b in blocks]
    torch.cuda.synchronize()
    errors = []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(15):
                    got = both(blocks[i])
                    stream.synchronize()
                    for a, c in zip(want[i], got):
                        assert torch.equal(bits(a), bits(c))
        except BaseException as e:  # noqa: BLE001 - reported by the main thread
            errors.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_captured_and_replayed():
    """Forward and backward as one graph, twice captured, each replayed on new inputs beside eager calls."""
    b = Block(2, 200, 256, 4, 2, 64, torch.bfloat16, 3)
    side = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(side):
        for _ in range(2):
            f = b.forward()
            b.backward(f)
        side.synchronize()
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                f = b.forward()
                out = list(tensors((*f, *b.backward(f))))
            graphs.append((g, out))
    torch.cuda.synchronize()
    for i in range(3):
        gen = torch.Generator().manual_seed(i)
        for t in (b.dev["y"], b.dev["residual"], b.dqkv):
            t.copy_(randn(gen, *t.shape, dtype=t.dtype))
        f = b.forward()
        want = [t.clone() for t in tensors((*f, *b.backward(f)))]
        torch.cuda.synchronize()
        for g, out in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            for a, c in zip(want, out):
                assert torch.equal(bits(a), bits(c))
