"""The rotary kernels' angles (csrc/rotary_angle.h, compiled for the host): position times frequency modulo a turn, in arithmetic that
C++ defines for every position and frequency."""
import os
import random
import shutil
import subprocess

import pytest

import local_linear_attention_flashlla_gb300 as lla

CSRC = os.path.join(os.path.dirname(lla.__file__), "csrc")

PROGRAM = r"""
#include "rotary_angle.h"
#include <cstdio>

int main() {
    long long position, turns;
    while (std::scanf("%lld %lld", &position, &turns) == 2) std::printf("%d\n", lla::rotary::turn_of(position, turns));
}
"""


def test_angles_wrap_by_defined_arithmetic(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "angle.cpp", tmp_path / "angle"
    src.write_text(PROGRAM)
    # a signed product that overflows ends the program
    subprocess.run([cxx, "-O1", "-std=c++17", "-fsanitize=signed-integer-overflow", "-fsanitize-undefined-trap-on-error", "-I" + CSRC,
                    str(src), "-o", str(exe)], check=True)
    rng = random.Random(1)
    turns = lla.rotary_table(128, device="cpu").turns.tolist() + [0, 1, -1, 2 ** 63 - 1, -2 ** 63]
    positions = [0, 1, 3, 4, 5, -1, -4, 2 ** 31 - 1, -2 ** 31, 2 ** 32 - 2, -2 ** 32] + [rng.randrange(-2 ** 31, 2 ** 31) for _ in range(40)]
    pairs = [(p, t) for p in positions for t in turns]
    r = subprocess.run([str(exe)], input="\n".join(f"{p} {t}" for p, t in pairs), capture_output=True, text=True, check=True)
    got = [int(x) for x in r.stdout.split()]
    assert len(got) == len(pairs)
    for (p, t), x in zip(pairs, got):
        assert (x - (p * t % 2 ** 64 >> 32)) % 2 ** 32 == 0 and -2 ** 31 <= x < 2 ** 31
