"""Operators on packed requests at the edges of what their documentation allows: sizes at a limit, inputs that are not
finite, offsets that spoil one request and must spoil no other, mixed batches, loops that run long enough to reuse
every buffer.  Oracles and tolerances are those of test_gpu_packed.py."""
import os
import subprocess
import sys

import numpy as np
import pytest

from checkpoint_input_replay_rssm_b200 import rssm
from oracle import packed
from tests.test_gpu_packed import _i, _tables_case, _tables_run

pytestmark = pytest.mark.gpu

ROOT = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..")


# ---------------------------------------------------------------- block tables
def _tables_equal(B):
    case = _tables_case(B, B, 16, 40, 2, 0)
    tab, out, err = _tables_run(case)
    want = packed.tables(*case)
    assert err == [0, 0, 0, 0] and tab == want[0] and out[4] == [want[5]]
    for got, w in zip(out, want[1:5]):
        assert got == w


@pytest.mark.parametrize("B", [6015, 6016, 6110, 6111, 6143, 6144])
def test_tables_of_batches_around_the_shared_memory_that_needs_no_permission(B):
    """In a process of its own: a larger batch before it would leave the kernel with the permission."""
    code = f"from tests.test_gpu_packed_edges import _tables_equal; _tables_equal({B})"
    done = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]
