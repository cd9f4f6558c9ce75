"""The bounds-checked build reaches every file that has kernels of its own: each
has checks, their reader, and is read by mr_checked_errors."""
import glob
import os

from unpermute_stable_counting_gb300 import _build


def test_every_file_with_kernels_is_checked():
    read = open(os.path.join(_build.CSRC, "runtime.cu")).read()
    seen = []
    for path in sorted(glob.glob(os.path.join(_build.CSRC, "*.cu"))):
        text = open(path).read()
        if "__global__" not in text:
            continue
        name = os.path.splitext(os.path.basename(path))[0]
        assert f"MR_CHECK_ACCESSOR({name})" in text, f"{name}.cu has kernels and no reader of its checks"
        assert f"mr::mr_check_words_{name}," in read.replace("}", ","), f"{name}.cu's checks are not read"
        seen.append(name)
    assert {"grouped_matmul", "layer", "quantize"} <= set(seen)
