"""The backward pass's shares of a row (csrc/logprobs_index.h), on the host: up to the longest row, every
element of a stretch is taken once and nothing outside it."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MAX = (1 << 31) - 1


@pytest.mark.skipif(shutil.which("g++") is None, reason="no C++ compiler")
def test_every_element_once(tmp_path):
    exe = tmp_path / "logprob_elements"
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-fsanitize=undefined",
                    "-fno-sanitize-recover=all", "-I", os.path.join(ROOT, "nvfp4_w4a4_moe_02_b200", "csrc"),
                    os.path.join(ROOT, "tests", "host_math", "logprob_elements.cpp"), "-o", str(exe)],
                   check=True, capture_output=True, text=True)
    cases = [(1, 1, 8, -1), (3, 1025, 4, -1), (2, 50257, 8, -1), (1, 300001, 4, -1), (100000, 131072, 8, -1)]
    cases += [(1, MAX - d, N, -2) for d in (0, 1, 127, 255, 256, 5000) for N in (4, 8)] + [(MAX, 9000, 8, -1)]
    text = "".join("%d %d %d %d\n" % c for c in cases)
    r = subprocess.run([str(exe)], input=text, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout + r.stderr
