"""How the norms' rows are laid out over threads and shared memory, on the host: every width, norm,
gate and sum beside them gets whole warps, each column once, and room (tests/c/norm_plan_check.cu)."""
from __future__ import annotations

import subprocess

import pytest

from unpermute_routing_indices_gb300 import _build

SRC = "norm_plan_check.cu"


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("norm_plan") / "check")
    r = subprocess.run([_build.NVCC, *_build.ARCH, "-O2", "-std=c++17", "--expt-relaxed-constexpr", "-I", _build.INCLUDE,
                        "-I", _build.CSRC, f"{_build.ROOT}/tests/c/{SRC}", "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return exe


def test_every_plan(program):
    r = subprocess.run([program], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout == "0 wrong\n", r.stdout
