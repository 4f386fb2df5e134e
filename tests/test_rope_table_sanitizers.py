"""The host table of rotations (csrc/rope_table.cpp) under AddressSanitizer,
UndefinedBehaviorSanitizer and ThreadSanitizer."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ is not installed")
@pytest.mark.parametrize("which", ["address,undefined", "thread"])
def test_rope_table_under_sanitizers(tmp_path, which):
    exe = str(tmp_path / "rope_table_sanitize")
    src = os.path.join(ROOT, "gemm_block_bit_amd", "csrc")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=" + which,
           "-fno-sanitize-recover=undefined", "-I", os.path.join(ROOT, "include"), "-I", src,
           os.path.join(ROOT, "tests", "rope_table_sanitize.cpp"), os.path.join(src, "rope_table.cpp"),
           os.path.join(src, "pack.cpp"), "-pthread", "-o", exe]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0, r.stdout
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:verify_asan_link_order=0")
    r = subprocess.run([exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, env=env, timeout=600)
    assert r.returncode == 0, r.stdout[-4000:]
    assert "ok" in r.stdout
