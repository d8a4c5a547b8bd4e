"""How attention work is cut up and shared out, checked on the CPU: the plan's
header compiled by the host compiler into tests/attend_plan_check.cpp."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a host C++ compiler")
def test_plan_arithmetic(tmp_path):
    exe = str(tmp_path / "plan")
    csrc = os.path.join(ROOT, "speculative_decoding_verification_89_b200", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O2", "-fsanitize=undefined", "-I", csrc,
                    os.path.join(ROOT, "tests", "attend_plan_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and r.stderr == "", r.stdout + r.stderr
