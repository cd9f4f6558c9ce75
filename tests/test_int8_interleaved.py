"""interleaved with out: what lies otherwise is refused, and rows are there as without out (no GPU needed)."""
import pytest
import torch

from test_expert_binding import calls, streams, zeros  # noqa: F401
from unpermute_stable_counting_gb300 import api

BF16, I8, F32 = torch.bfloat16, torch.int8, torch.float32


def quantize(rows, cols, out):
    return api.moe_quantize_int8(zeros(rows, cols, dtype=BF16), interleaved=True, out=out)


def norm(rows, cols, out):
    return api.moe_add_rms_norm(zeros(rows, cols, dtype=BF16), zeros(cols, dtype=BF16), quantize="int8", with_y=False,
                                interleaved=True, out=out)


def both(rows, cols, room=4):
    t = zeros(rows, cols + room, dtype=I8)
    return t, dict(values=t[:, :cols], scales=t.view(F32)[:, cols // 4])


@pytest.mark.parametrize("f", [quantize, norm])
def test_rows_are_given(calls, f):
    for rows in (4, 1):
        t, out = both(rows, 8)
        got = f(rows, 8, dict(out, rows=t))
        assert got["rows"] is t
        got = f(rows, 8, out)
        assert got["rows"].shape == (rows, 12) and got["rows"].data_ptr() == t.data_ptr() and got["rows"].stride() == (12, 1)
    assert len(calls.made) == 4


@pytest.mark.parametrize("f", [quantize, norm])
@pytest.mark.parametrize("out", [
    lambda: dict(values=zeros(4, 8, dtype=I8), scales=zeros(4)),              # scales of their own
    lambda: both(4, 8, 8)[1],                                                 # room behind the scales
    lambda: dict(both(4, 8)[1], rows=zeros(4, 12, dtype=I8)),                 # rows of their own
    lambda: dict(both(4, 8)[1], scales=both(4, 8)[1]["scales"]),              # scales of other rows
    lambda: dict(values=both(1, 8)[0][:, :8], scales=zeros(1)),               # a single row
])
def test_what_lies_otherwise_is_refused(calls, f, out):
    out = out()
    with pytest.raises(ValueError, match="interleaved"):
        f(out["values"].shape[0], 8, out)
    assert not calls.made


@pytest.mark.parametrize("f", [quantize, norm])
def test_rows_that_hold_no_scale_are_refused(calls, f):
    t = zeros(4, 12, dtype=I8)
    with pytest.raises(ValueError):
        f(4, 6, dict(values=t[:, :6], scales=t.view(F32)[:, 2]))
    assert not calls.made
