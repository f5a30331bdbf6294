"""Which tensors the 8-bit and seam calls of the binding take: checked on host tensors, with a
library that records calls in place of the built one, so that nothing reaches a device."""

import pytest
import torch

from shared_token_transformer_b200 import binding as B


# ---------------------------------------------------------------------------
# descriptors of norms, gates and scales
# ---------------------------------------------------------------------------
def test_a_gate_given_as_a_vector_is_one_group():
    """The kernel holds each row's group against `groups`; every group it lets through must lie in the gate."""
    assert B.norm_gate_desc(gate=torch.zeros(64), scale=torch.zeros(64)).groups == 1
    assert B.norm_gate_desc(gate=torch.zeros(3, 64)).groups == 3
    sw = B.sandwich_weights(gate1=torch.zeros(1, 64), gate2=torch.zeros(64))
    assert (sw.groups, sw.width) == (1, 64)
    with pytest.raises(ValueError):
        B.sandwich_weights(gate1=torch.zeros(64), gate2=torch.zeros(64, 64))


@pytest.mark.parametrize("name", ["post_g", "post_b", "pre_g", "pre_b", "gate", "scale"])
def test_vectors_are_fp32(name):
    for dtype in (torch.int32, torch.uint32, torch.float64, torch.bfloat16):
        with pytest.raises(ValueError):
            B.norm_gate_desc(**{name: torch.zeros(2, 64).to(dtype)})


def test_row_groups_of_a_sandwich_are_int32():
    for dtype in (torch.float32, torch.uint32, torch.int64):
        with pytest.raises(ValueError):
            B.sandwich_weights(row_group=torch.zeros(8).to(dtype))
    with pytest.raises(ValueError):
        B.sandwich_weights(row_group=torch.zeros(16, dtype=torch.int32)[::2])
    assert B.sandwich_weights(row_group=torch.zeros(8, dtype=torch.int32)).row_group


@pytest.mark.parametrize("name", ["post_g", "post_b", "pre_g", "pre_b", "gate", "scale"])
def test_vectors_are_single_and_not_empty(name):
    for shape in ((0,), (0, 64), (2, 0), ()):      # the address of nothing would read as "none"
        with pytest.raises(ValueError):
            B.norm_gate_desc(**{name: torch.zeros(shape)})
    assert getattr(B.norm_gate_desc(**{name: torch.zeros(1, 64)}), name)
    if name != "gate":                             # rows past the first would be left out
        with pytest.raises(ValueError):
            B.norm_gate_desc(**{name: torch.zeros(2, 64)})
