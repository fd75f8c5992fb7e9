"""The routed block's launch rules under AddressSanitizer and UndefinedBehaviorSanitizer (no GPU); see
block_rules_sanitized.cpp."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ is not installed")
def test_block_rules_under_asan_and_ubsan(tmp_path):
    exe = tmp_path / "block_rules_sanitized"
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
           "-I", os.path.join(ROOT, "swiglu_mlp_fwd_amd", "csrc"), os.path.join(HERE, "block_rules_sanitized.cpp"),
           "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, f"build failed:\n{r.stderr}"
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "block rules: ok" in r.stdout, f"{r.stdout}\n{r.stderr}"
