"""The combine and its gradient at every number of tokens a step on the
bounds-checked build: an offset outside its tensor would surface as
SQ_ERR_BOUNDS from sq_sync_status or as a skipped store.  No test makes an
out-of-range access."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEBUG_LIB = os.path.join(ROOT, "w8a8_int8_gemm_calib_b200", "libsq_b200_debug.so")


def test_steps_on_the_bounds_checked_build():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    if not os.path.exists(DEBUG_LIB):
        subprocess.check_call([sys.executable, os.path.join(ROOT, "w8a8_int8_gemm_calib_b200",
                                                            "build.py"), "--debug-bounds"])
    r = subprocess.run([sys.executable, "-m", "pytest", "tests/test_experts_steps.py", "-m", "gpu",
                        "-x", "-q", "-p", "no:cacheprovider"],
                       env=dict(os.environ, SQ_B200_LIB=DEBUG_LIB), cwd=ROOT, capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
