"""sps_page_tables over the batch sizes whose sums pass the shared memory that a launch has without asking:
each size before any larger one, in a process of its own (what a launch may ask for stays granted)."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

SCRIPT = """
import numpy as np
from paged_top_sparse_gb300 import build
build.build()
from tests.test_gpu_page_tables import Call
for batch in list(range(first, last + 1)) + [16384]:
    rng = np.random.default_rng(batch)
    q, c = rng.integers(0, 3, batch).tolist(), rng.integers(0, 300, batch).tolist()
    call = Call(q, c, 4, 40000, seed=batch)
    assert call.run() == 0, batch
    call.check()
"""


@pytest.mark.parametrize("first,last", [(4090, 4100), (6118, 6150)])
def test_batches_around_the_default_shared_memory(first, last):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", f"first, last = {first}, {last}\n{SCRIPT}"], cwd=root,
                          capture_output=True, text=True, timeout=600)
    assert done.returncode == 0, done.stderr[-2000:]
