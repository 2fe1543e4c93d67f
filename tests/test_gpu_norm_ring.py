"""The norms' rings of bulk copies after a wait that was given up: nothing more is copied, and what is on its way
is waited for (tests/c/norm_ring_check.cu; the wait is given up by the test, not by a copy)."""
from __future__ import annotations

import subprocess

import pytest

from unpermute_routing_indices_gb300 import _build

pytestmark = pytest.mark.gpu


def test_a_wait_given_up(tmp_path):
    exe = str(tmp_path / "ring")
    r = subprocess.run([_build.NVCC, *_build.ARCH, "-O2", "-std=c++17", "--expt-relaxed-constexpr", "-I", _build.INCLUDE,
                        "-I", _build.CSRC, f"{_build.ROOT}/tests/c/norm_ring_check.cu", "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
