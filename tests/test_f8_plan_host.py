"""CPU test of the tiles and splits that the 8-bit floating point product chooses: the rules of csrc/f8_plan.h and
csrc/product.h, built for the host alone, asked about sizes over their whole range and about the sizes that the
GPU tests run."""
from __future__ import annotations

import math
import os
import random
import shutil
import subprocess

import pytest

from tests import f8_tiles as ft

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "tests", "host_sanitize", "f8_plan_check.cpp")
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not found")


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    exe = tmp_path_factory.mktemp("plan") / "f8_plan_check"
    cmd = [HIPCC, "-x", "hip", "--cuda-host-only", "--offload-arch=gfx950", "-O1", "-std=c++17",
           "-I" + os.path.join(ROOT, "rope_ltx3drope_amd", "csrc"), SRC, "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]

    def run(products):
        lines = "\n".join(ft.question(p) for p in products) + "\n"
        r = subprocess.run([str(exe)], input=lines, capture_output=True, text=True, timeout=120, check=True)
        plans = [tuple(int(v) for v in line.split()) for line in r.stdout.splitlines()]
        assert len(plans) == len(products)
        return plans

    return run


def spread(rng, low, high):
    return int(math.exp(rng.uniform(math.log(low), math.log(high))))


def drawn(rng, count):
    """Products of sizes spread over their range, half of them on 16 bytes."""
    found = []
    for _ in range(count):
        dim = spread(rng, 8, 9000)
        if rng.random() < 0.5:
            dim = max(16, dim // 16 * 16)
        found += ft.products(spread(rng, 17, 9000), dim, spread(rng, 8, 10300))
    return found


def listed():
    return [p for s in ft.SIZES for p in ft.products(*s)]


def runs(products, plans):
    found = {}
    for p, (bm, bn, tiles, splits, _) in zip(products, plans):
        names, steps = ft.kernels(p, (bm, bn, tiles, splits))
        if steps >= 4:
            for name in names:
                found.setdefault(name, p)
    return found


def test_gpu_sizes_run_every_kernel_that_sizes_of_the_range_reach(ask):
    products = drawn(random.Random(7), 20000)
    reached = runs(products, ask(products))
    ours = listed()
    tested = runs(ours, ask(ours))
    missing = {k: v for k, v in reached.items() if k not in tested}
    assert not missing, f"add to tests/f8_tiles.py sizes that run {missing}"
    tiles = {k[:3] for k in tested}
    assert {("bf16", t, w) for t in ("256x256", "256x128") for w in ("walk", "walk on")} <= tiles
    assert {(u, t, w) for u in ("fp32", "bf16") for t in ("128x64", "64x64") for w in ("direct", "registers")} <= tiles


def test_plans_are_within_what_the_kernels_take(ask):
    """Tiles cover the output, splits leave every part at least four steps, sums of the parts fit their bytes."""
    products = drawn(random.Random(8), 5000) + listed()
    for p, (bm, bn, tiles, splits, parts) in zip(products, ask(products)):
        _, M, N, k, direct, _ = p
        assert tiles == -(-M // bm) * -(-N // bn), p
        assert 1 <= splits <= 16 and (splits == 1 or -(-k // ft.STEP) // splits >= 4), p
        assert parts == (splits * tiles * bm * bn * 4 if splits > 1 else 0), p
        assert direct or bm < 256, p
        assert (bm, bn) in ((256, 256), (256, 128), (128, 64), (64, 64)), p
