"""The bounds-checked build (libattamba_checked.so) on the cases of many rows and tiles, of padded rows and of NaN."""

import os
import subprocess
import sys

import pytest

from test_gpu_checked import ROOT, RUNNER

pytestmark = pytest.mark.gpu


def test_rows_padding_and_nan_cases_pass_with_every_index_checked():
    env = dict(os.environ, ATTAMBA_LIBRARY="checked", PYTHONPATH=os.pathsep.join((ROOT, os.path.join(ROOT, "tests"))))
    r = subprocess.run([sys.executable, "-c", RUNNER, "tests/test_gpu_ssm_rows.py", "tests/test_gpu_ssm_padding.py",
                        "tests/test_gpu_ssm_nan.py", "tests/test_gpu_ssm_blocks.py"], cwd=ROOT, env=env, capture_output=True,
                       text=True, timeout=1200)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout and "failed" not in r.stdout, r.stdout[-2000:]
