"""What the torch helpers make of their arguments before a call; runs without a GPU."""
import pytest
import torch

from test_decay_abi_cpu import lr  # noqa: F401


@pytest.mark.parametrize("dtype", [torch.uint8, torch.int8, torch.int16, torch.int32, torch.int64, torch.uint16])
@pytest.mark.parametrize("L", [5, 40000, 2 ** 31 - 100])
def test_row_lengths_of_every_integer_type(lr, dtype, L):  # noqa: F811
    """L need not fit the type of the lengths."""
    got = lr._lens_of(torch.tensor([0, 3, 100], dtype=dtype), L, torch.device("cpu"))
    assert got.dtype is torch.int32
    assert got.clamp(max=L).tolist() == [0, 3, min(100, L)]


def test_row_lengths_past_32_bits(lr):  # noqa: F811
    got = lr._lens_of(torch.tensor([-2 ** 40, 2 ** 32 + 1, 7]), 9, torch.device("cpu"))
    assert got.tolist() == [0, 9, 7]
