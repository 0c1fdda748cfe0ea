"""First verify launches of different lengths from several host threads at once are all accepted: each raises the shared
memory limit of the same kernel (tests/verify_threads_case.py; a process shows a lost limit about one time in four)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_first_launches_of_different_lengths_at_once():
    import __graft_entry__
    __graft_entry__.build()
    for _ in range(8):
        r = subprocess.run([sys.executable, "-m", "tests.verify_threads_case"], cwd=ROOT, capture_output=True, text=True,
                           timeout=300)
        assert r.returncode == 0, r.stdout[-1000:] + r.stderr[-3000:]
