"""The optimizer and routing calls from plain C: tests/c/abi_operators.c, compiled as C99 against the header and linked
to the in-tree library and the CUDA runtime."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "reduction_reducer_gb300")


def build(out):
    from reduction_reducer_gb300 import _lib, build as b
    if not os.path.exists(_lib.LIB_PATH):
        b.build()
    cc = shutil.which("gcc") or shutil.which("cc")
    nvcc = b.nvcc()
    cuda = os.environ.get("CUDA_HOME") or os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    if cc is None:
        pytest.skip("no C compiler")
    lib64 = os.path.join(cuda, "lib64")
    subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(cuda, "include"), os.path.join(ROOT, "tests", "c", "abi_operators.c"), "-L", PKG,
                    "-lddpreducer", "-L", lib64, "-lcudart", "-lm", f"-Wl,-rpath,{PKG}", f"-Wl,-rpath,{lib64}", "-o",
                    str(out)], check=True, capture_output=True, text=True)


def test_it_builds(tmp_path):
    build(tmp_path / "abi_operators")


@pytest.mark.gpu
def test_it_runs(tmp_path):
    exe = tmp_path / "abi_operators"
    build(exe)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip() == "c operators ok"
