"""The fixed-point angle of the rotation, compiled for the host with a check for signed
overflow and compared with whole numbers of any size (no device needed)."""
import os
import random
import subprocess

import pytest

import attention_decode_megakernel_b200 as mk
from attention_decode_megakernel_b200 import build

SOURCE = """
#include <cstdio>
#include "mk_rope.cuh"
int main() {
  int position;
  unsigned long long turns;
  while (std::scanf("%d %llu", &position, &turns) == 2)
    std::printf("%u\\n", mk::rp::turn_at(position, turns));
}
"""


def test_angle_at_any_position(tmp_path):
    """Positions and frequencies of the whole range: the product modulo 2^64, and no step
    that C++ leaves undefined."""
    if not os.path.exists(build.NVCC):
        pytest.skip("no nvcc")
    source, program = tmp_path / "angle.cu", tmp_path / "angle"
    source.write_text(SOURCE)
    subprocess.run([build.NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17",
                    "--expt-relaxed-constexpr", "-I", os.path.join(build.PKG, "csrc"),
                    "-Xcompiler", "-fsanitize=signed-integer-overflow", "-Xcompiler",
                    "-fno-sanitize-recover=all", "-Xcompiler", "-static-libubsan",
                    str(source), "-o", str(program)], check=True, capture_output=True)
    rng = random.Random(3)
    turns = list(mk.Rope(256, 1e7).c.turns) + [0, 1, 2 ** 62, 2 ** 64 - 1]
    places = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 131071, -70000]
    places += [rng.randint(-2 ** 31, 2 ** 31 - 1) for _ in range(50)]
    cases = [(p, t) for p in places for t in turns]
    run = subprocess.run([str(program)], input="".join("%d %d\n" % c for c in cases), text=True,
                         capture_output=True)
    assert run.returncode == 0, run.stderr[-500:]
    assert [int(x) for x in run.stdout.split()] == [(p * t % 2 ** 64) >> 32 for p, t in cases]
