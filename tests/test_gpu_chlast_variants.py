"""The bounds-checked build (TB_DEBUG_BOUNDS=1) through the channels-last and
dropout tests: their kernels check every address before they use it, results stay
within the tolerances, and the device status word reads 0 at the end."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_bounds_checked_build_passes_the_channels_last_tests():
    from patch_groupnorm_gb300 import build
    path = build.build(variant="debug_bounds", defines=["TB_DEBUG_BOUNDS=1"])
    env = dict(os.environ, TILEBLEND_LIB=path)
    r = subprocess.run([sys.executable, "-m", "pytest", "tests/test_gpu_chlast.py", "tests/test_gpu_dropout.py",
                        "tests/test_zz_training_status.py", "-m", "gpu", "-q", "-x", "-p", "no:cacheprovider"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=1800)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout and "failed" not in r.stdout
