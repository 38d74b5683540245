"""The range-checked build (-DGQA_DEBUG) on the paged cache's tests: in a child
process with GQA_ATTN_DEBUG=1 each must match the oracle as before, and the
autouse fixture in conftest.py fails any test after which a check had failed."""

import os
import re
import subprocess
import sys

import pytest

from gqa_decode_attention_place_gb300 import _build

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
FILES = ["test_paged_decode_gpu.py", "test_pages_gpu.py", "test_paged_chain_gpu.py",
         "test_paged_limits_gpu.py"]
DESELECT = "not past_32_bits"  # the 9 GB of pools are left out for memory and time


def test_range_checked_build_parity():
    _build.build(debug=True)
    env = dict(os.environ, GQA_ATTN_DEBUG="1")
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
           "-k", DESELECT] + [os.path.join(HERE, f) for f in FILES]
    r = subprocess.run(cmd, cwd=os.path.dirname(HERE), env=env, capture_output=True, text=True,
                       timeout=900)
    tail = "\n".join((r.stdout + r.stderr).splitlines()[-30:])
    assert r.returncode == 0, f"range-checked build:\n{tail}"
    m = re.search(r"(\d+) passed", r.stdout)
    assert m and int(m.group(1)) >= 100 and " failed" not in r.stdout, tail
