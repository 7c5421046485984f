"""The transformer-block operators called from several host threads, each on its own stream: no call
shares memory with another, so every result is that of the call alone."""
from __future__ import annotations

import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

rla = pytest.importorskip("rope_ltx3drope_amd")

DEV = "cuda:0"


def test_threads_on_their_own_streams():
    def work(seed):
        gen = torch.Generator().manual_seed(seed)
        x = torch.randn(200, 1024, generator=gen).bfloat16().to(DEV)
        w = torch.randn(1024, generator=gen).to(DEV)
        wg, wu = ((torch.randn(300, 1024, generator=gen) / 32).bfloat16().to(DEV) for _ in range(2))
        wd, sd = rla.q8_quantize(torch.randn(1024, 300, generator=gen).to(DEV))
        torch.cuda.synchronize()

        def calls():
            n = rla.norm_before(x, w)
            h, g, u = rla.gated_ffn(n, wg, wu, save=True)
            q, s = rla.q8_quantize(h)
            y = rla.q8_matmul(q, s, wd, sd)
            r, n2 = rla.norm_after(y, x, w, next_weight=w)
            grads = rla.norm_after_backward(n2, n2, y, r, w, next_weight=w)
            dx, dwg, dwu = rla.gated_ffn_backward(h, n, wg, wu, g, u)
            return [n, h, y, r, n2, grads.dy, grads.dresidual, grads.dweight, grads.dnext_weight, dx, dwg, dwu]

        return calls

    jobs = [work(s) for s in range(4)]
    want = [[t.clone() for t in j()] for j in jobs]
    torch.cuda.synchronize()
    errors = []

    def run(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    got = jobs[i]()
                    stream.synchronize()
                    for a, b in zip(want[i], got):
                        assert torch.equal(a, b)
        except BaseException as e:  # noqa: BLE001 - reported by the main thread
            errors.append((i, e))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
