"""The training operators' cases in the checked build (see test_gpu_device_checks): every gathered key row, listed
place, slot of a key block and row position that their kernels compute lies inside its buffer."""
import subprocess
import sys

import pytest

from test_gpu_device_checks import ROOT, checked_env

pytestmark = pytest.mark.gpu


def test_training_cases_record_no_index_error():
    r = subprocess.run([sys.executable, "-m", "pytest", "tests/test_gpu_train.py", "-q", "-x", "-m", "gpu", "-k",
                        "list_scores or places or bad_lists or training_step and not captured", "-p",
                        "no:cacheprovider"], cwd=ROOT, env=checked_env(), capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout and "failed" not in r.stdout
