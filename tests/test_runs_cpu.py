"""The shared-prefix attention's plan on the CPU (runs_check.cu): every block that the join reads is one that this call
left, also where a warp or a CTA gave up in the middle of its work."""
import ctypes
import random
import subprocess

import pytest

from decode_attention_split_gb300 import build as td_build


@pytest.fixture(scope="module")
def checks(tmp_path_factory):
    import os
    so = str(tmp_path_factory.mktemp("runs") / "runs_check.so")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "runs_check.cu")
    subprocess.run([td_build.nvcc(), *td_build.ARCH, "-O1", "-std=c++17", "-shared", "-Xcompiler", "-fPIC",
                    f"-I{td_build.INCLUDE}", f"-I{td_build.CSRC}", src, "-o", so], check=True)
    return ctypes.CDLL(so)


def test_runs_leave_every_block_that_the_join_reads(checks):
    rng = random.Random(1)
    behind = 0
    for n in range(400):
        B, Hkv, RB = rng.choice([1, 2, 5, 40, 130]), rng.choice([1, 2, 3, 8]), rng.choice([1, 1, 2, 5])
        most = rng.choice([1, 16, 17, 100, 600, 5000])
        lens = [rng.choice([0, 1, 16, 17, most, rng.randint(0, most)]) for _ in range(B)]
        grid = rng.choice([1, 2, 7, 30, 152])
        met = ctypes.c_int()
        quits = rng.randrange(grid * 4) if n % 3 else rng.randrange(min(grid * 4, 4))
        r = checks.check_runs(B, Hkv, RB, rng.randint(1, 24), grid, (ctypes.c_int * B)(*lens), quits, rng.choice([0, 0, 1, 3]),
                              ctypes.byref(met))
        assert r == 0, f"runs_check.cu:{r}, case {n}"
        behind += met.value
    assert behind > 1000  # there were groups behind the ones given up in


def test_ctas_leave_every_prefix_block_that_the_join_reads(checks):
    rng = random.Random(2)
    for n in range(300):
        tiles, Hkv, chunks = rng.choice([1, 2, 3, 9]), rng.choice([1, 2, 8]), rng.choice([1, 2, 5, 19])
        P = rng.choice([0, 1, 127, 128, 129, rng.randint(0, 5000)])
        grid = rng.choice([1, 3, 40, 152])
        r = checks.check_items(tiles, Hkv, chunks, grid, P, rng.randrange(grid))
        assert r == 0, f"runs_check.cu:{r}, case {n}"
