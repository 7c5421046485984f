"""Sizes that between them run every tile kernel of the 8-bit floating point product (csrc/f8.hip): each tile, by direct
copies and through registers, whole steps of k and a ragged last one, in one piece and split over k, with odd and
even numbers of steps, four of them at least, and for the walking kernels one tile a compute unit and more.

tests/test_f8_plan_host.py holds the list to that, whatever the costs in csrc/f8_plan.h are tuned to;
tests/test_f8_tiles_gpu.py runs it, each size with either result type, a scale for each row of b and for
each 128, and its rows packed and 128 bytes or a multiple apart.  A size is (tokens, dim, out).
"""
from __future__ import annotations

SIZES = [
    (19, 444, 9), (19, 1545, 8), (19, 2789, 8), (21, 565, 8), (65, 608, 9817), (196, 6525, 9989), (204, 8768, 2923),
    (259, 393, 7701), (343, 7515, 4086), (449, 548, 6300), (652, 419, 8406), (1355, 388, 8228), (1381, 6992, 3180),
    (1413, 528, 5520), (1898, 1520, 13), (2940, 8364, 1469), (3411, 592, 1161), (3545, 7948, 1280),
    (4684, 528, 7132), (5035, 2112, 13), (5206, 6997, 788), (5411, 400, 1596), (5488, 5568, 196), (5587, 7170, 8),
    (5729, 520, 1148), (5784, 5632, 174), (5905, 464, 5404), (7189, 400, 586), (7977, 571, 1324), (8244, 5719, 83),
    (8345, 8176, 9), (8431, 4821, 70), (8588, 5562, 215), (8799, 5680, 466)]
STEP = 128  # numbers of k in a step


def products(tokens, dim, out):
    """The products (layout, M, N, k, direct, bytes from row to row) of operands whose rows are packed and apart."""
    apart = -(-dim // 128) * 128
    return [("packed", tokens, out, dim, int(dim % 16 == 0), dim), ("apart", tokens, out, dim, 1, apart)]


def question(product):
    """The line that f8_plan_check.cpp takes."""
    _, M, N, k, direct, row = product
    return f"{M} {N} {k} {direct} {row}"


def kernels(product, plan):
    """What a plan (bm, bn, tiles, splits) launches, for either result type, and the steps of one workgroup's part."""
    _, _, _, k, direct, _ = product
    bm, bn, tiles, splits = plan
    steps = -(-k // STEP) // splits
    ragged = "ragged" if direct and k % 16 else "whole steps"
    part = "split" if splits > 1 else "one piece"
    parity = "odd" if steps % 2 else "even"
    way = "direct" if direct else "registers"
    found = [("fp32", f"{bm}x{bn}", way, ragged, part, parity)]
    if bn >= 128 and k % 16 == 0:
        found.append(("bf16", f"{bm}x{bn}", "walk on" if tiles * splits > 256 else "walk", ragged, part, parity))
    else:
        found.append(("bf16", f"{bm}x{bn}", way, ragged, part, parity))
    return found, steps
