"""The kernels' own arithmetic of the K split (csrc/moe_few_split.h), on the host: every lane's value is
defined, and the choice is the restated one."""
import os
import random
import shutil
import subprocess

import pytest

import few_split

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def build(tmp_path, name):
    exe = tmp_path / name
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-fsanitize=undefined",
                    "-fno-sanitize-recover=all", "-I", os.path.join(ROOT, "nvfp4_w4a4_moe_02_b200", "csrc"),
                    os.path.join(ROOT, "tests", "host_math", name + ".cpp"), "-o", str(exe)],
                   check=True, capture_output=True, text=True)
    return str(exe)


@pytest.mark.skipif(shutil.which("g++") is None, reason="no C++ compiler")
def test_every_lane_is_defined_and_the_least_wins(tmp_path):
    rng = random.Random(1)
    cases = [(0, 148, 1), (1, 148, 1), (1, 1, 256), (2048 * 1024, 148, 256), (2048 * 1024, 1, 256), (1440, 148, 16)]
    cases += [(rng.randrange(0, 1 << rng.randrange(1, 21)), rng.choice([1, 4, 74, 132, 148, 160]), rng.randint(1, 256))
              for _ in range(3000)]
    text = "".join(f"{u} {sms * few_split.WARPS} {nch}\n" for u, sms, nch in cases)
    r = subprocess.run([build(tmp_path, "few_split")], input=text, capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    got = [int(v) for v in r.stdout.split()]
    assert got == [few_split.choose(*c) for c in cases]
    assert set(got) == {1, 2, 4, 8, 16}


def test_the_sizes_meant_for_each_split_take_it():
    # counts per expert, H, I -> S of gate_up and down on 148 SMs
    for counts, H, I, want in [((1, 1), 2048, 64, (16, 1)), ((1, 1), 1152, 1152, (8, 8)), ((3, 3), 1280, 1344, (8, 8)),
                               ((64, 64), 512, 1600, (2, 8)), ((64, 64), 128, 32768, (1, 16))]:
        assert few_split.of_call(counts, H, I, 148) == want
