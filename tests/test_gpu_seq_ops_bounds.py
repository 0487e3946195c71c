"""The operators on several tokens and whole sequences under the bounds-check build of the library
(see test_gpu_bounds_checked.py): no check fails, and the comparisons still hold."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_sequence_operators_pass_every_bounds_check():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    env = dict(os.environ, KVQ_LIBRARY="debug")
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.join(ROOT, "tests", "test_gpu_seq_ops.py"), "-m", "gpu",
                        "-x", "-q", "-p", "no:cacheprovider"], cwd=ROOT, env=env, capture_output=True, text=True,
                       timeout=1200)
    tail = "\n".join((r.stdout + r.stderr).splitlines()[-30:])
    assert r.returncode == 0, tail
    assert " passed" in r.stdout, tail
