"""The SSM block's operators in the bounds-checked build (libattamba_checked.so): token ranges, tiles, windows and state
rows are tested against the arrays they address while the parity cases run, and malformed sequence tables raise no
ATTAMBA_DEV_BOUNDS either: their clamps keep every access inside."""

import os
import subprocess
import sys

import pytest

from test_gpu_checked import ROOT, RUNNER

pytestmark = pytest.mark.gpu


def test_ssm_block_cases_pass_with_every_index_checked():
    env = dict(os.environ, ATTAMBA_LIBRARY="checked", PYTHONPATH=os.pathsep.join((ROOT, os.path.join(ROOT, "tests"))))
    r = subprocess.run([sys.executable, "-c", RUNNER, "tests/test_gpu_ssm_block.py", "tests/test_gpu_ssm_layer.py"], cwd=ROOT,
                       env=env, capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout and "failed" not in r.stdout, r.stdout[-2000:]
