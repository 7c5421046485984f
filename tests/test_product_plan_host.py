"""CPU test of the tiles and splits that the block's matrix products choose: the rules of csrc/product.h, built
for the host alone, asked about sizes over their whole range and about the sizes that the GPU tests run."""
from __future__ import annotations

import math
import os
import random
import shutil
import subprocess

import pytest

from tests import block_tiles as bt

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "tests", "host_sanitize", "plan_check.cpp")
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not found")


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    exe = tmp_path_factory.mktemp("plan") / "plan_check"
    cmd = [HIPCC, "-x", "hip", "--cuda-host-only", "--offload-arch=gfx950", "-O1", "-std=c++17",
           "-I" + os.path.join(ROOT, "rope_ltx3drope_amd", "csrc"), SRC, "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]

    def run(pairs):
        lines = "\n".join(bt.question(kind, p) for kind, p in pairs) + "\n"
        r = subprocess.run([str(exe)], input=lines, capture_output=True, text=True, timeout=120, check=True)
        plans = [tuple(int(v) for v in line.split()) for line in r.stdout.splitlines()]
        assert len(plans) == len(pairs)
        return plans

    return run


def spread(rng, low, high):
    return int(math.exp(rng.uniform(math.log(low), math.log(high))))


def drawn(rng, count):
    """(kind, product) pairs of sizes spread over their range, most of them on 16 bytes."""
    pairs = []
    for _ in range(count):
        kind = rng.choice(["bf16", "f32", "int8"])
        dim = spread(rng, 8, 9000 if kind == "int8" else 4200)
        if rng.random() < 0.7:
            dim = max(16, dim // 16 * 16)
        pairs += [(kind, p) for p in bt.products(kind, spread(rng, 17, 9000), dim, spread(rng, 8, 10300))]
    return pairs


def listed():
    pairs = [(kind, p) for kind, sizes in bt.FFN.items() for s in sizes for p in bt.products(kind, *s)]
    return pairs + [("int8", p) for s in bt.Q8 for p in bt.products("int8", *s)]


def runs(pairs, plans):
    """The instantiations that run long enough to go round their rings, with the parity of their steps."""
    found = {}
    for (kind, p), (bm, bn, tiles, splits, _) in zip(pairs, plans):
        name, steps = bt.kernel(kind, p, (bm, bn, tiles, splits))
        if steps >= (4 if splits > 1 else 7):
            found.setdefault(name + ("odd" if steps % 2 else "even",), p)
    return found


def test_gpu_sizes_run_every_kernel_that_sizes_of_the_range_reach(ask):
    pairs = drawn(random.Random(7), 20000)
    reached = runs(pairs, ask(pairs))
    ours = listed()
    tested = runs(ours, ask(ours))
    missing = {k: v for k, v in reached.items() if k not in tested}
    assert not missing, f"add to tests/block_tiles.py sizes that run {missing}"
    tiles = {k[:4] for k in tested}
    assert {("bf16", f, t, "direct") for f in ("forward", "dx", "dw") for t in ("256x256", "256x128", "128x64")} <= tiles


def test_plans_are_within_what_the_kernels_take(ask):
    """Tiles cover the output, splits leave every part at least four steps, sums of the parts fit their bytes."""
    pairs = drawn(random.Random(8), 5000) + listed()
    for (kind, p), (bm, bn, tiles, splits, parts) in zip(pairs, ask(pairs)):
        form, M, N, k, direct, _ = p
        columns = bn // 2 if form == "forward" and kind != "int8" else bn
        assert tiles == -(-M // bm) * -(-N // columns), (kind, p)
        assert 1 <= splits <= 16 and (splits == 1 or -(-k // bt.STEP[kind]) // splits >= 4), (kind, p)
        assert parts == (splits * tiles * bm * bn * 4 if splits > 1 else 0), (kind, p)
        assert direct or bm < 256, (kind, p)
