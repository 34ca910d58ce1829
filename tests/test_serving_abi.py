"""The C ABI of gemm_serving.h without a GPU: exported symbols, a header that is plain C
with the structures that the binding has, and Python names."""
from __future__ import annotations

import ctypes
import os
import re
import shutil
import subprocess

import pytest

import dense_gemm_03_amd as dg
from dense_gemm_03_amd import serving

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gemm_serving.h")
STRUCTS = {"gemm_moe_params": dg.MoeParams, "gemm_adapter_params": dg.AdapterParams,
           "gemm_log_probs_params": dg.LogProbsParams}


def test_exports_the_headers_symbols():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:int|int64_t)\s+(gemm_\w+)\s*\(", text, re.M))
    assert names == set(serving.SIGNATURES)
    lib = ctypes.CDLL(dg.LIB_PATH)
    for name in names:
        assert hasattr(lib, name) and callable(getattr(dg, name)), name


def test_structures_are_the_headers(tmp_path):
    """Offsets of every field, as a C compiler sees them."""
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.fail("gcc is needed to read the header")
    lines = ["#include <stddef.h>", "#include <stdio.h>", "#include \"gemm_serving.h\"", "int main(void) {"]
    for name, kind in STRUCTS.items():
        lines.append('printf("%%zu\\n", sizeof(%s));' % name)
        lines += ['printf("%%zu\\n", offsetof(%s, %s));' % (name, f) for f, _ in kind._fields_]
    (tmp_path / "t.c").write_text("\n".join(lines + ["return 0; }"]))
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    subprocess.run([gcc, "-std=gnu11", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(rocm, "include"),
                    "-I", os.path.join(ROOT, "include"), str(tmp_path / "t.c"), "-o", str(tmp_path / "t")], check=True)
    got = [int(v) for v in subprocess.run([str(tmp_path / "t")], check=True, capture_output=True, text=True).stdout.split()]
    want = []
    for kind in STRUCTS.values():
        want.append(ctypes.sizeof(kind))
        want += [getattr(kind, f).offset for f, _ in kind._fields_]
    assert got == want
