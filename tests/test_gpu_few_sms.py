"""The expert operators' suites on the bounds-checked build for few SMs
(-DMR_SM_COUNT): fewer blocks than moe_layer may have tokens, and several tiles
for each block of the persistent kernels, at sizes that otherwise have one."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SUITES = ["test_gpu_layer.py", "test_gpu_expert_products.py", "test_gpu_expert_edges.py"]


def run_suites(suites, **env):
    r = subprocess.run([sys.executable, "-m", "pytest", "-m", "gpu", "-x", "-q", "-p", "no:cacheprovider"]
                       + [os.path.join("tests", f) for f in suites], cwd=ROOT,
                       env=dict(os.environ, **env), capture_output=True, text=True, timeout=1500)
    tail = r.stdout[-4000:] + r.stderr[-2000:]
    assert r.returncode == 0 and " passed" in r.stdout and " failed" not in r.stdout, tail


def test_expert_suites_on_few_sms():
    from unpermute_stable_counting_gb300 import _build, _native
    if _native.checked_requested():
        pytest.skip("this process runs against another build")
    assert _build.FEW_SMS < 64                   # the most tokens of a layer
    _build.build_library(few_sms=True)
    run_suites(SUITES, USC_CHECKED="1", USC_FEW_SMS="1")


def test_several_tiles_on_the_checked_build():
    """(Their sizes go by the device's own SMs.)"""
    from unpermute_stable_counting_gb300 import _build, _native
    if _native.checked_requested():
        pytest.skip("this process runs against another build")
    _build.build_library(checked=True)
    run_suites(["test_gpu_expert_tiles.py"], USC_CHECKED="1")
