"""CPU test of the rotation's sine and cosine (csrc/axes_math.h), built for the host with g++ (the same IEEE operations
as on the device, contraction off), against the exact ones.

Bound.  With r quarters left, |r| <= 1/2: the polynomials with their rounded coefficients leave 6.7e-9 (sine 3.1e-9),
r's rounding 2^-26 of a quarter, 2.34e-8.  Cosine: z = r r is off by 2^-24 of itself, 1.24 z 2^-24 <= 1.84e-8, the
last but one step rounds at 1.23 (2^-24), which z scales to 1.5e-8, the steps before it to less than 1e-9, and the
last rounds at 1 (2^-25): 2.99e-8; in all 9.4e-8.  Sine: p is off by 2^-24 of 0.65 z and 2^-24 for its steps, at
r <= 1/2 in all 1.4e-8, the product r p rounds at 0.08 (3.8e-9) and the sum at 0.71 (2.99e-8): 7.5e-8.
The device has the same operations, so what it adds is the angle's own error.
"""
from __future__ import annotations

import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "rope_ltx3drope_amd", "csrc")
SRC = os.path.join(ROOT, "tests", "host_sanitize", "axes_math_check.cpp")


@pytest.fixture(scope="module")
def evaluate(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not found")
    exe = tmp_path_factory.mktemp("axes") / "axes_math_check"
    cmd = [gxx, "-O2", "-std=c++20", "-ffp-contract=off", "-fno-fast-math", "-D__host__=", "-D__device__=", "-I" + CSRC,
           SRC, "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]

    def run(part):
        part = np.ascontiguousarray(part, np.float64)
        lines = "\n".join("%x" % b for b in part.view(np.uint64).tolist())
        out = subprocess.run([str(exe)], input=lines, capture_output=True, text=True, timeout=300, check=True)
        bits = np.array([int(v, 16) for v in out.stdout.split()], np.uint32).reshape(-1, 2)
        assert len(bits) == len(part)
        return bits.view(np.float32)

    return run


def exact(part):
    """Cosine and sine of the fraction of a turn, to 64 bits: exact in eighths of a turn, the library's beyond."""
    part = np.asarray(part, np.longdouble)
    quarter = np.rint(part * 4)
    rest = (part * 4 - quarter) * (np.longdouble("1.57079632679489661923132169163975144"))
    c, s = np.cos(rest), np.sin(rest)
    k = quarter.astype(np.int64) % 4
    return (np.choose(k, [c, -s, -c, s]), np.choose(k, [s, c, -s, -c]))


def test_within_the_bound(evaluate):
    rng = np.random.default_rng(1)
    part = np.concatenate([np.arange(0, 1, 2.0 ** -20), rng.random(1 << 20), 1.0 - rng.random(1000) * 1e-9,
                           rng.random(1000) * 1e-9, (np.arange(8) / 8), np.nextafter(np.arange(1, 9) / 8, 0.0),
                           np.nextafter(np.arange(8) / 8, 1.0)])
    got = evaluate(part)
    c, s = exact(part)
    worst = max(float(np.abs(got[:, 0] - c).max()), float(np.abs(got[:, 1] - s).max()))
    assert worst <= 9.4e-8, worst


def test_quarters_are_exact(evaluate):
    got = evaluate([0.0, 0.25, 0.5, 0.75, 1.0 - 2.0 ** -53])
    want = [(1, 0), (0, 1), (-1, 0), (0, -1), (1, 0)]
    for (c, s), (wc, ws) in zip(got.tolist(), want):
        assert abs(c - wc) < 1e-15 and abs(s - ws) < 1e-15
