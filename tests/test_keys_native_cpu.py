"""Host-only checks of the key-set operators (tests/native/keys_check.cu, built
from the host side's source and the library's other objects; no GPU needed)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("nvcc") is None, reason="nvcc not on PATH")
def test_host_checks(tmp_path):
    from token_locking_b200 import build as b
    b.build()
    objs = [os.path.join(b.BUILD, os.path.splitext(s)[0] + ".o") for s in b.SOURCES
            if s != "api_keys.cu"]
    exe = str(tmp_path / "keys_check")
    cmd = ["nvcc", "-gencode", "arch=compute_100a,code=sm_100a", "-O1", "-std=c++17",
           "-I" + os.path.join(ROOT, "include"), "-I" + b.CSRC,
           os.path.join(ROOT, "tests", "native", "keys_check.cu"), *objs, "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    print(r.stdout)
    assert r.returncode == 0, r.stdout[-4000:]
    assert " 0 failures" in r.stdout
