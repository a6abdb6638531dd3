"""A bounded wait of the tcgen05 attention kernel that runs out ends in NaN rows, not in a hang.

The kernel has a test hook, off unless SPEC_VERIFY_TEST_STALL_ATTENTION names a batch row: the
row's CTAs never report one tile's notes (one plain barrier arrival is left out), so the
softmax's wait for it runs out after a quarter of a second, then those of the products, the
copies and the other roles, and every CTA returns.  The library reads the variable once, so
each case runs in a child process."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.parametrize("row", [0, 2])
def test_a_wait_that_runs_out_writes_nan(row):
    env = dict(os.environ, SPEC_VERIFY_TEST_STALL_ATTENTION=str(row))
    res = subprocess.run([sys.executable, os.path.join(HERE, "_attention_stall_check.py")], env=env,
                         capture_output=True, text=True, timeout=600)
    assert res.returncode == 0, res.stdout[-2000:] + res.stderr[-4000:]
    assert res.stdout.strip().endswith("ok")
