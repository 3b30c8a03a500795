"""The head cross entropy in pieces under the debug build, whose kernels check
every direct store against the bounds of its output (see
test_gpu_debug_bounds.py): ragged sizes, pieces and guard bands."""
import os
import subprocess
import sys

import pytest

from backward_tcgen05_tma_gemms_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.gpu
def test_linear_ce_under_the_bounds_checked_build():
    env = dict(os.environ, TPS_LIBRARY=build.build(debug=True))
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.join(HERE, "test_gpu_linear_ce.py"), "-q", "-m", "gpu",
                        "-p", "no:cacheprovider", "-k", "sizes or odd or pieces or fp32 or padding or stray"],
                       env=env, cwd=os.path.dirname(HERE), capture_output=True, text=True, timeout=900)
    assert r.returncode == 0 and " passed" in r.stdout, r.stdout[-3000:] + r.stderr[-2000:]
