"""The suites of the INT8 products' long sums and shared tiles on the bounds-checked builds (all SMs, and few)."""
import pytest

from test_gpu_few_sms import run_suites

pytestmark = pytest.mark.gpu

SUITES = ["test_gpu_int8_sums.py", "test_gpu_int8_shares.py", "test_gpu_int8_long_rows.py", "test_gpu_int8_norm_eps.py"]


@pytest.mark.parametrize("few_sms", [False, True])
def test_suites_on_the_checked_builds(few_sms):
    from unpermute_stable_counting_gb300 import _build, _native
    if _native.checked_requested():
        pytest.skip("this process runs against another build")
    _build.build_library(**({"few_sms": True} if few_sms else {"checked": True}))
    run_suites(SUITES, USC_CHECKED="1", **({"USC_FEW_SMS": "1"} if few_sms else {}))
