"""The page map at the batch sizes where its launch changes.  The cases and their check are those of test_page_map_gpu."""

import os
import subprocess
import sys

import pytest

from test_page_map_gpu import _case, _check

pytestmark = pytest.mark.gpu


def _batch(n):
    ctx, new, table, free, page, t = _case(n, n, 50, 1, 16)
    assert _check(ctx, new, table, free, page, t + 3)[-1][1] == 0


# 6128 requests are the first whose prefix sums and the kernel's other shared memory pass 48 KB together, 6144 the first
# whose prefix sums do so alone.  A kernel keeps a limit that was raised: each size in a process of its own.
@pytest.mark.parametrize("n", [6127, 6128, 6143, 6144])
def test_large_batches_as_a_process_first_call(n):
    code = f"from top_sparse_mla_gb300 import build; build(); import test_page_map_edges_gpu as t; t._batch({n})"
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([here, os.path.dirname(here), os.environ.get("PYTHONPATH", "")]))
    run = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]
