"""The paged cache's kernels in the range-checked build, in the forms that
test_checked_paged.py does not reach (tests/checked_paged_forms.py)."""
import os
import subprocess
import sys

import pytest

from causal_head_self_gb300 import build as _build

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_the_other_forms_pass_every_range_check():
    _build.build(check=True)
    env = dict(os.environ, CHS_ATTN_CHECK="1")
    r = subprocess.run([sys.executable, os.path.join(HERE, "checked_paged_forms.py")], env=env,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "long_cases ok" in r.stdout
