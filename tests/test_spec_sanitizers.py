"""tg_fork and tg_tree_masks under AddressSanitizer and UndefinedBehaviorSanitizer, with injected
allocation failures (tests/native/fork_faults.cpp)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_fork_under_sanitizers(tmp_path):
    exe = str(tmp_path / "fork_faults")
    csrc = os.path.join(ROOT, "non_uniform_paged_flash_b200", "csrc")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                           "-I" + os.path.join(ROOT, "include"), "-I" + csrc,
                           os.path.join(ROOT, "tests", "native", "fork_faults.cpp"),
                           os.path.join(csrc, "tg_host.cpp"), "-o", exe])
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "injected failures" in r.stdout
