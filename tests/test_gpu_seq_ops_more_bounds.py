"""Many tiles a CTA, padded chunks and side-code prompts under the bounds-check build of the library
(see test_gpu_bounds_checked.py): no check fails, and the comparisons still hold."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_long_and_padded_chunks_pass_every_bounds_check():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    env = dict(os.environ, KVQ_LIBRARY="debug")
    files = [os.path.join(ROOT, "tests", f) for f in ("test_gpu_seq_ops_ranges.py", "test_gpu_seq_ops_tiles.py")]
    r = subprocess.run([sys.executable, "-m", "pytest", *files, "-m", "gpu", "-x", "-q", "-p", "no:cacheprovider", "-k",
                        "side_code or padding or groups_and_pages or query_groups or one_split"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    tail = "\n".join((r.stdout + r.stderr).splitlines()[-30:])
    assert r.returncode == 0, tail
    assert " passed" in r.stdout, tail
