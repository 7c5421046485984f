"""CPU test of the launches that the rotation with several axes makes: csrc/axes.h, built for the host alone, asked
about the corners of the documented sizes and about sizes drawn over their whole range."""
from __future__ import annotations

import itertools
import math
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "tests", "host_sanitize", "axes_shape_check.cpp")
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
HEADS = WIDTH = 65536  # the most heads of q and of k, and the widest head
TOKENS = (1 << 31) - 1

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not found")


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    exe = tmp_path_factory.mktemp("axes") / "axes_shape_check"
    cmd = [HIPCC, "-x", "hip", "--cuda-host-only", "--offload-arch=gfx950", "-O1", "-std=c++17",
           "-I" + os.path.join(ROOT, "rope_ltx3drope_amd", "csrc"), SRC, "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]

    def run(problems):
        lines = "\n".join(" ".join(str(int(v)) for v in p) for p in problems) + "\n"
        r = subprocess.run([str(exe)], input=lines, capture_output=True, text=True, timeout=120, check=True)
        out = [tuple(int(v) for v in line.split()) for line in r.stdout.splitlines()]
        assert len(out) == len(problems)
        return out

    return run


def accesses(f32, halves, head_dim, pairs):
    """The accesses (elements) that the widths allow: 16 bytes, two elements, one."""
    return [v for v in (4 if f32 else 8, 2, 1)
            if (pairs if halves else 2 * pairs) % v == 0 and (head_dim - 2 * pairs) % v == 0]


def corners():
    sizes = [(1, 1), (2, 1), (8, 3), (128, 64), (WIDTH, 1), (WIDTH, 8), (WIDTH - 1, 1), (WIDTH - 2, 32767), (WIDTH, 32768),
             (WIDTH, 16384), (16384, 8192), (32768, 4)]
    heads = [(1, 0), (0, 1), (1, 1), (32, 8), (8200, 0), (16384, 0), (32768, 0), (HEADS, 0), (0, HEADS), (HEADS, HEADS)]
    for f32, halves, (head_dim, pairs), (hq, hk), tokens, batch in itertools.product(
            (0, 1), (0, 1), sizes, heads, (1, 63, 5003, TOKENS), (1, 65535)):
        if 2 * pairs > head_dim:
            continue
        for v in accesses(f32, halves, head_dim, pairs):
            yield (f32, halves, v, batch, tokens, hq, hk, head_dim, pairs, 3)


def spread(rng, low, high):
    return int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))


def drawn(rng, count):
    for _ in range(count):
        f32, halves = rng.randint(0, 1), rng.randint(0, 1)
        head_dim = max(2, spread(rng, 1, WIDTH))
        if rng.random() < 0.6:
            head_dim = max(16, head_dim // 16 * 16)
        pairs = head_dim // 2 if rng.random() < 0.5 else max(1, min(head_dim // 2, spread(rng, 1, head_dim // 2)))
        if rng.random() < 0.5:
            pairs = max(1, pairs // 8 * 8)
        hq, hk = spread(rng, 1, HEADS), rng.choice([0, spread(rng, 1, HEADS)])
        yield (f32, halves, rng.choice(accesses(f32, halves, head_dim, pairs)), spread(rng, 1, 65535),
               spread(rng, 1, TOKENS), hq, hk, head_dim, pairs, rng.randint(1, 255))


def test_every_call_ends_in_launches_that_the_chip_takes(ask):
    problems = list(corners()) + list(drawn(random.Random(3), 20000))
    largest = 0
    for p, (planes, together, jobs, tokens, groups) in zip(problems, ask(problems)):
        assert tokens >= 1, p  # or the launches would never reach the last token
        assert 1 <= groups < 1 << 26, p  # 64 threads each, fewer than 2^32 in all
        assert 1 <= jobs <= 1 << 25 and planes <= 1026, p
        largest = max(largest, jobs)
    assert largest > 1 << 23  # the range is reached


def test_sizes_whose_tokens_make_a_million_workgroups(ask):
    """One token of 2 to 8 GB."""
    problems = [(0, 0, 8, 1, 1, 32768, 0, WIDTH, 32768, 1), (0, 1, 1, 1, 3, 16384, 0, WIDTH - 2, 32767, 1),
                (0, 0, 1, 1, 2, 8200, 0, WIDTH - 1, 1, 3), (0, 0, 8, 1, 1, HEADS, 0, WIDTH, 8, 1)]
    for p, (_, _, jobs, tokens, groups) in zip(problems, ask(problems)):
        assert jobs >= 1 << 20 and tokens >= 1 and groups == min(tokens, p[4]) * jobs, p
