"""Rotations, the plan, the listing of tiles and the kernels that make D, in the
range-checked build (-DATTN_CHECK): their own tests once more in a process that
loads it, where every address that they compute is checked before it is used."""
import glob
import os
import subprocess
import sys

import pytest

from causal_head_self_gb300 import build as _build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_every_file_of_kernels_has_range_checks():
    files = [f for f in glob.glob(os.path.join(_build.CSRC, "*.cuh"))
             if "__global__" in open(f, encoding="utf-8").read()]
    assert len(files) >= 10
    for f in files:
        assert "attn_check(" in open(f, encoding="utf-8").read(), f


@pytest.mark.gpu
@pytest.mark.parametrize("file,which", [("test_tokens.py", "rope or plan or slots or length or page"),
                                        ("test_packed.py", "short_sequences or few_keys or many")])
def test_cases_pass_every_range_check(file, which):
    _build.build(check=True)
    env = dict(os.environ, CHS_ATTN_CHECK="1")
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.join(HERE, file), "-x", "-q", "-m", "gpu",
                        "-k", which, "-p", "no:cacheprovider"], env=env, capture_output=True, text=True,
                       timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert " passed" in r.stdout
