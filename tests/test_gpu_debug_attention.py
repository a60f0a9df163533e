"""The attention kernels in the bounds-checking build: no index out of range, and
a planted out-of-range column is recorded instead of read.  The cases run in a
process that loads libsla_debug_bounds.so."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_attention_in_the_bounds_checking_build():
    script = os.path.join(ROOT, "tests", "debug_bounds_attention.py")
    r = subprocess.run([sys.executable, script], capture_output=True, text=True, timeout=1500)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-4000:]
    assert "debug bounds: ok" in r.stdout
