"""The turned outputs of the 8-bit quantisers through the C ABI: any distance between their rows and any start, and
what lies between the rows."""
from __future__ import annotations

import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu

rla = pytest.importorskip("rope_ltx3drope_amd")
from rope_ltx3drope_amd import _lib  # noqa: E402

DEV = "cuda:0"
REST = 0x5a  # what the buffer holds before


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("blocks", [0, 1])
@pytest.mark.parametrize("rows,dim", [(1, 7), (16, 128), (129, 136), (200, 300), (255, 24), (300, 1000)])
def test_rows_any_distance_apart(rows, dim, blocks, dtype):
    L = _lib.lib()
    gen = torch.Generator(device=DEV).manual_seed(rows)
    x = torch.randn(rows, dim, generator=gen, device=DEV).to(dtype)
    want = (rla.f8_quantize_weight if blocks else rla.f8_quantize)(x, turned=True)
    as_bytes = lambda t: t.contiguous().view(torch.uint8)  # noqa: E731
    down, across = -(-rows // 128), -(-dim // 128)
    for pitch in (rows, rows + 1, rows + 5, -(-rows // 16) * 16, -(-rows // 16) * 16 + 32):
        for start in (0, 1, 16):
            buf = torch.full((start + dim * pitch + 64,), REST, dtype=torch.uint8, device=DEV)
            q = torch.empty(rows, dim, dtype=torch.uint8, device=DEV)
            scale = torch.empty(down if blocks else rows, across, device=DEV)
            scale_t = torch.empty(across if blocks else dim, down, device=DEV)
            call = _lib.F8Quantize(dtype=0 if dtype is torch.float32 else 1, blocks=blocks, rows=rows, dim=dim,
                                   turned_pitch=pitch, scale_strides=(_lib.i64 * 2)(across, 1),
                                   scale_turned_strides=(_lib.i64 * 2)(down, 1), x=x.data_ptr(), q=q.data_ptr(),
                                   scale=scale.data_ptr(), q_turned=buf.data_ptr() + start, scale_turned=scale_t.data_ptr())
            reason = ctypes.c_int(-1)
            assert L.ltx3drope_f8_quantize(call, torch.cuda.current_stream().cuda_stream, reason) == _lib.OK, reason.value
            assert torch.equal(q, as_bytes(want[0])) and torch.equal(scale, want[1])
            got = buf[start:start + dim * pitch].view(dim, pitch)
            assert torch.equal(got[:, :rows], as_bytes(want[2])) and torch.equal(scale_t, want[3]), (pitch, start)
            # up to the next multiple of 16 there may be zeros; all else is as it was
            spare = got[:, rows:min(pitch, -(-rows // 16) * 16)]
            assert bool(((spare == 0) | (spare == REST)).all())
            assert bool((got[:, -(-rows // 16) * 16:] == REST).all())
            assert bool((buf[:start] == REST).all()) and bool((buf[start + dim * pitch:] == REST).all())
