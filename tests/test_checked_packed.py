"""The kernels over packed sequences in the range-checked build
(-DATTN_CHECK): every copy that they issue is checked against the tensor it
reads, in a process of its own (tests/checked_packed_cases.py); none may fail."""
import os
import subprocess
import sys

import pytest

from causal_head_self_gb300 import build as _build

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_packed_cases_pass_every_range_check():
    _build.build(check=True)
    env = dict(os.environ, CHS_ATTN_CHECK="1")
    r = subprocess.run([sys.executable, os.path.join(HERE, "checked_packed_cases.py")], env=env,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "packed_cases ok" in r.stdout
