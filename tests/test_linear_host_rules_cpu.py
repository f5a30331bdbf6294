"""What the linear layers decide on the host, before any CUDA call."""

import ctypes

import pytest

from shared_token_transformer_b200 import binding as B
from shared_token_transformer_b200 import build as Bd

P = 1 << 20          # an aligned address that no call here reads


@pytest.fixture(scope="module", autouse=True)
def built():
    Bd.build()


def model(dtype):
    return B.model_desc(64, 4, 256, dtype, (0, 8, 8)) if dtype == "f32" else B.model_desc(256, 4, 256, dtype, (0, 32, 32))


def linear(dtype, rows, K, N, x=P, y=P + (1 << 40), scratch=P):
    return B.lib().ts_op_linear(ctypes.byref(model(dtype)), x, rows, K, P, P, N, P, 0, y, scratch, None)


def linear_q8(dtype, rows, K, N, x=P, y=P + (1 << 40)):
    return B.lib().ts_op_linear_q8(ctypes.byref(model(dtype)), x, P, rows, K, P, P, N, P, 0, y, None)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8", "int8"])
def test_no_rows_are_no_work_at_any_size(dtype):
    for K, N in ((64, 64), (100, 64), (64, 100), (200000, 3)):
        assert linear(dtype, 0, K, N) == 0
        if dtype in ("fp8", "int8"):
            assert linear_q8(dtype, 0, K, N) == 0


@pytest.mark.parametrize("dtype", ["fp8", "int8"])
def test_linear_q8_refuses_an_output_over_its_rows(dtype):
    """Tiles are written while others still read the rows."""
    rows, K, N = 4, 128, 64                        # x 512 bytes, y 512 bytes
    for y in (P, P + 16, P + 496, P - 16, P - 496):
        assert linear_q8(dtype, rows, K, N, y=y) == 1, y - P
        assert b"overlap" in B.lib().ts_last_error()
    assert linear_q8(dtype, 0, K, N, y=P) == 0
