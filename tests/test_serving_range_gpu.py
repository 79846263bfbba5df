"""A serving step's calls around the 4-bit window cache on the GPU at sizes, scores and values where
they reach their limits, against their reference (oracle/serving.py).  Bounds are those that
test_serving_gpu.py derives."""
import os
import subprocess
import sys

import numpy as np
import pytest

from test_kv4_gpu import hq  # noqa: F401  (the fixture)
from test_serving_gpu import Pool

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


# ------------------------------------------------------------------ resize
def resize_there_and_back(hq, B):
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(0, 30, B)]
    have = sum(-(-n // 16) for n in lens)
    pool = Pool(hq, rng, B, 16, 5, have + B // 2, lens)
    granted = pool.step(hq, lens, [int(x) for x in rng.integers(0, 80, B)], 50 * B)
    pool.step(hq, granted, lens, 50 * B)


@pytest.mark.parametrize("B", [4010, 4011, 4096, 4097, 16384])
def test_resize_of_many_sequences_first(hq, B):
    """In a process of its own, whose first large resize it is: no call may need another before it."""
    code = ("import test_serving_range_gpu as t\nfrom weights_hq_encode_gb300 import hq\n"
            f"t.resize_there_and_back(hq, {B})\nt.resize_there_and_back(hq, 600)\n"
            f"t.resize_there_and_back(hq, {B})\n")
    path = os.pathsep.join([os.path.dirname(HERE), HERE, os.environ.get("PYTHONPATH", "")])
    got = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, PYTHONPATH=path), cwd=HERE,
                         capture_output=True, text=True, timeout=300)
    assert got.returncode == 0, got.stderr[-2000:]
