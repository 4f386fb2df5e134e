"""The host table of rotations (csrc/rope_table.cpp) where memory runs out at
any of its allocations, those that start its threads among them."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ is not installed")
def test_rope_table_without_memory(tmp_path):
    exe = str(tmp_path / "rope_table_memory")
    src = os.path.join(ROOT, "gemm_block_bit_amd", "csrc")
    cmd = ["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "include"), "-I", src,
           os.path.join(ROOT, "tests", "rope_table_memory.cpp"), os.path.join(src, "rope_table.cpp"),
           os.path.join(src, "pack.cpp"), "-pthread", "-o", exe]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0, r.stdout
    r = subprocess.run([exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stdout[-2000:])
    assert "ok" in r.stdout
