"""The step of a rotary frequency (csrc/rope_step.h, compiled for the host) against whole-number arithmetic."""
import ctypes
import os
import random
import shutil
import subprocess
from fractions import Fraction

import pytest

from tests.pi_bits import two_pi
from tests.test_cache_cpu import lib, rope_args  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_steps(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("no C++ compiler")
    src, so = tmp_path / "step.cpp", tmp_path / "step.so"
    src.write_text('#include "rope_step.h"\nextern "C" uint64_t step(double f) { return fvattn::rope_step(f); }\n')
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=undefined", "-fno-sanitize-recover", "-static-libubsan",
                        "-shared", "-fPIC", "-I", os.path.join(ROOT, "top_routed_block_b200", "csrc"), str(src), "-o", str(so)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    step = ctypes.CDLL(str(so)).step
    step.restype, step.argtypes = ctypes.c_uint64, [ctypes.c_double]
    rng = random.Random(3)
    freqs = [0.0, -0.0, 1.0, -1.0, 6.283185307179586, 2.0 ** 63, 2.0 ** 64 - 2048, 2.0 ** -61, -1e-30, 5e-324, 1e-300, 10000.0 ** -0.7]
    freqs += [rng.choice([-1, 1]) * rng.random() * 2.0 ** rng.randint(-70, 64) for _ in range(4000)]
    for f in freqs:
        turns = Fraction(f) / two_pi(320)
        off = turns * 2 ** 64 - step(f)
        off -= round(off / 2 ** 64) * 2 ** 64
        assert abs(off) <= Fraction(1, 2) + Fraction(1, 2 ** 60), f


@pytest.mark.parametrize("freq,rc", [(2.0 ** 64, -2), (-1e300, -2), (float("inf"), -1), (float("nan"), -1)])
def test_frequencies_refused(lib, freq, rc):  # noqa: F811
    args = rope_args(Qr=ctypes.c_void_p(4096))
    for i in (0, 31):
        args[15] = (ctypes.c_double * 32)(*[freq if j == i else 1.0 for j in range(32)])
        assert lib.fvattn_rope(*args) == rc
