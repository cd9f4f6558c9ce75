"""Calls of the INT8 products that no grid or count of tiles holds are refused before anything is enqueued (no GPU
needed: nothing touches the CUDA runtime)."""
import pytest

from test_int8_host import BF16, INT8, INVALID, L, ffn, matmul  # noqa: F401

ROWS, COLS = 1 << 30, 1 << 24


@pytest.mark.parametrize("kw", [
    dict(rows=ROWS, N=COLS, yst=COLS), dict(rows=ROWS, N=COLS, yst=COLS, dt=BF16),
    dict(rows=ROWS, N=COLS, yst=COLS, g=None, G=-1), dict(rows=ROWS, N=64, K=COLS, xst=COLS),  # rows widened by a kernel
    dict(rows=ROWS, N=1 << 20, yst=1 << 20, G=ROWS),                                           # a tile for each row
])
def test_matmul(L, kw):
    assert matmul(L, **{"size": 1 << 62, **kw}) == INVALID


@pytest.mark.parametrize("kw", [
    dict(rows=ROWS, I=COLS), dict(rows=ROWS, I=COLS, dt=BF16), dict(rows=ROWS, H=COLS, xst=COLS, yst=COLS),
    dict(rows=ROWS, H=COLS, xst=COLS, yst=COLS, dt=BF16, I=64),  # the second product's tiles
])
def test_ffn(L, kw):
    assert ffn(L, **{"size": 1 << 62, **kw}) == INVALID
