"""Calls of the 8-bit integer linear layer that its documentation allows and the other tests do not make."""

import numpy as np
import pytest
import torch

from _gpu import dev
from shared_token_transformer_b200 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def device_status_is_clean():
    yield
    torch.cuda.synchronize()
    B.device_status()


def int8_model():
    return B.model_desc(256, 4, 256, "int8", (0, 32, 32))


@pytest.mark.parametrize("M,K", [(1, 256), (5, 1536), (8, 2048), (12, 1024), (130, 512)])
@pytest.mark.parametrize("part", ["whole", "last row"])
def test_rows_may_be_replaced_by_the_output(M, K, part):
    """y over x: the rows are quantised into the scratch first, in a launch of their own, at any number of rows."""
    N = K
    rng = np.random.default_rng(M + K)
    wq = torch.from_numpy(rng.integers(-127, 128, (N, K)).astype(np.int8)).cuda()
    sw, b = torch.full((N,), 2.0 ** -12, device="cuda"), dev(rng.standard_normal(N), torch.float32)
    buf = torch.zeros((2 * M, K), dtype=torch.bfloat16, device="cuda")
    buf[:M] = dev(rng.standard_normal((M, K)), torch.bfloat16)
    x, y = buf[:M].clone(), torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    scratch = torch.empty(M * (K + 4), dtype=torch.uint8, device="cuda")
    B.op_linear(int8_model(), x, wq, b, y, w_scale=sw, scratch=scratch)
    n = B.launch_count()
    first = 0 if part == "whole" else M - 1
    B.op_linear(int8_model(), buf[:M], wq, b, buf[first:first + M], w_scale=sw, scratch=scratch)
    assert B.launch_count() - n == 2
    assert torch.equal(buf[first:first + M], y)
