"""The list of tiles and pieces of the linear-layer kernels, on the host."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


def test_every_tile_is_covered_once(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.fail("g++ is needed to build the check")
    exe = str(tmp_path / "pieces")
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I",
                    os.path.join(os.path.dirname(HERE), "dense_gemm_03_amd", "csrc"),
                    os.path.join(HERE, "linear_pieces.cpp"), "-o", exe], check=True)
    res = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0, res.stdout
