"""The vocabulary losses in the debug build, whose kernels check the indices of their accesses."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

HERE = os.path.dirname(os.path.abspath(__file__))


def test_debug_build_index_checks_stay_silent():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_fp32_gemm_04_gb300 import _build

    _build.build(debug=True)
    env = dict(os.environ, SGEMM_GB300_DEBUG_CHECKS="1")
    r = subprocess.run([sys.executable, os.path.join(HERE, "vocab_debug_run.py")], env=env, capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "status word 0 after each" in r.stdout
