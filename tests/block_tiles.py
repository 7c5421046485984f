"""Sizes that between them run every tile kernel of the block's matrix products (csrc/product.h): each type,
each storage of the operands (forward: k innermost; dx: the weights with k outermost; dw: both), each tile,
by direct copies and through registers, in one piece and split over k, with odd and even numbers of steps,
at least seven of them a workgroup (four where the sums are split), and ragged edges.

tests/test_product_plan_host.py holds the list to that, whatever the costs in product.h are tuned to;
tests/test_block_tiles_gpu.py runs it.  A size is (tokens, dim, hidden) or, in 8 bits, (tokens, dim, out).
"""
from __future__ import annotations

FFN_BF16 = [
    (17, 752, 10), (17, 936, 11), (18, 392, 9), (22, 456, 10), (133, 920, 9), (214, 1295, 2089), (390, 713, 243),
    (401, 396, 3927), (403, 2448, 1583), (410, 608, 5051), (415, 4112, 4680), (442, 400, 228), (460, 2344, 2156),
    (463, 464, 591), (466, 3560, 695), (598, 495, 326), (612, 407, 666), (717, 656, 4503), (753, 756, 4025),
    (758, 8, 323), (760, 4024, 1355), (778, 583, 11), (812, 1160, 4857), (897, 744, 9), (1176, 3928, 1754),
    (1357, 2512, 197), (1521, 2888, 2741), (3275, 2128, 210), (3603, 3419, 201), (3949, 2760, 323),
    (4558, 203, 2422), (4586, 456, 2231), (4654, 608, 881), (4807, 400, 2537), (423, 2784, 9915),
    (5445, 1632, 1274), (5281, 208, 8639)]
FFN_F32 = [
    (200, 264, 102), (202, 259, 129), (217, 1552, 2517), (232, 240, 276), (233, 320, 139), (291, 230, 2118),
    (334, 201, 113), (531, 3047, 1810), (628, 592, 3254), (661, 722, 3801), (685, 506, 5250), (932, 280, 107),
    (949, 312, 1906), (1251, 1054, 99), (2626, 3626, 435), (2783, 1584, 12), (3419, 79, 4042), (4745, 11, 4538),
    (4830, 1576, 103)]
Q8 = [
    (17, 1280, 10), (19, 968, 11), (20, 1424, 12), (22, 804, 15), (22, 864, 8), (22, 1906, 8), (25, 1856, 8),
    (107, 4448, 2884), (354, 6012, 1381), (502, 800, 2413), (723, 4816, 2871), (995, 4416, 2061),
    (2105, 834, 1709), (2110, 944, 3925), (2159, 925, 81), (2743, 966, 1235), (3423, 1120, 3030),
    (4130, 1008, 1084), (4382, 7312, 44), (4389, 912, 213), (4686, 816, 996), (4957, 3035, 221),
    (2532, 8256, 1625), (1628, 7920, 2497)]
# Up to 16 tokens: kernels without tiles, or one round of tiles of 64 (bf16 from five tokens on, 8161 and more
# hidden columns), on 16 bytes and off them, rows shorter and longer than a wavefront's kilobytes.
FEW = [(tokens, dim, hidden) for tokens in (1, 2, 4, 5, 8, 9, 16)
       for dim, hidden in ((8, 3), (520, 8161), (1001, 77), (4104, 8200), (6152, 33))]

FFN = {"bf16": FFN_BF16, "f32": FFN_F32}
STEP = {"bf16": 64, "f32": 32, "int8": 128}  # k of a step of 128 bytes
STREAMED_ROWS = 128  # rows of A up to which bf16 tiles of 64 take whole steps


def products(kind, tokens, dim, width):
    """The products (form, M, N, k, direct, bytes from row to row) that a call makes."""
    if kind == "int8":
        return [("forward", tokens, width, dim, int(dim % 16 == 0), dim)]
    row = dim * (4 if kind == "f32" else 2)
    padded = -(-width // STEP[kind]) * STEP[kind]
    direct = int(row % 16 == 0)
    return [("forward", tokens, width, dim, direct, row), ("dx", tokens, dim, 2 * padded, direct, row),
            ("dw", 2 * padded, dim, tokens, direct, row)]


def question(kind, product):
    """The line that plan_check.cpp takes."""
    form, M, N, k, direct, row = product
    return f"{kind} {int(form == 'forward' and kind != 'int8')} {int(form != 'forward')} {M} {N} {k} {direct} {row}"


def kernel(kind, product, plan):
    """The instantiation that a plan (bm, bn, tiles, splits) launches, and the steps of one workgroup."""
    form, M, _, k, direct, _ = product
    bm, bn, _, splits = plan
    whole_steps = bm == 64 and direct and form == "forward" and (kind != "bf16" or M <= STREAMED_ROWS)
    steps = -(-k // STEP[kind]) // splits
    return (kind, form, f"{bm}x{bn}" + (" whole steps" if whole_steps else ""), "direct" if direct else "registers",
            "split" if splits > 1 else "whole"), steps
