"""The host side of the vocabulary losses on machines unlike the one it was measured on, with a pretended CUDA runtime
(fake_runtime.cpp)."""

import os
import shutil
import subprocess

import pytest

import dense_fp32_gemm_04_gb300 as sg
from conftest import ROOT

CSRC = os.path.join(ROOT, "dense_fp32_gemm_04_gb300", "csrc")


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    from dense_fp32_gemm_04_gb300 import _build

    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_build.nvcc())))
    exe = str(tmp_path_factory.mktemp("host") / "host")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(cuda, "include"), "-o", exe,
                    os.path.join(ROOT, "tests", "fake_runtime.cpp")] +
                   [os.path.join(CSRC, f) for f in ("sgemm_api.cpp", "vocab_api.cpp", "vocab_plan.cpp", "planner.cpp")], check=True)

    def call(*args):
        out = subprocess.run([exe] + [str(a) for a in args], capture_output=True, text=True, timeout=60, check=True).stdout
        return [int(x) for x in out.split()]

    return call


@pytest.mark.parametrize("pairs", [0, 1, 40, 75, 76])
@pytest.mark.parametrize("dtype", [0, 1])
def test_workspace_is_the_plans_whatever_is_resident(run, pairs, dtype):
    """Fewer CTA pairs than half the SMs, or none, need no more workspace than sgemm_vocab_plan gives: a captured call fits."""
    for T, V, D in ((400, 32768, 1024), (700, 50021, 513), (2000, 32768, 2048), (4096, 131072, 256), (8, 5000, 64), (1, 300, 40),
                    (300, 9000, 4096), (600, 32768, 1024), (1100, 32768, 2048)):
        for grads in (0, 1, 2, 3):
            made, planned, reserved, rc, more, launches, count = run("workspace", pairs, T, V, D, dtype, grads)
            assert made == planned == reserved == rc == 0
            assert more == 0, (T, V, D, grads, more)
            if grads in (0, 3):
                assert count == launches


def test_a_handle_does_without_the_vocabulary_kernels(run):
    """Where they cannot run, the GEMM does; the losses are refused and launch nothing."""
    made, gemm, loss, grad, launched = run("attributes")
    assert made == sg.SGEMM_OK and gemm == sg.SGEMM_OK
    assert loss == grad == sg.SGEMM_ERR_NOT_SUPPORTED and launched == 0
