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


class Elsewhere:
    """A tensor of another GPU, as far as the helpers look before they copy it."""
    is_cuda, dtype, device = True, torch.float32, torch.device("cuda", 1)
    shape = torch.Size((4, 8))

    def __init__(self, here):
        self.here = here

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0

    def float(self):
        return self

    contiguous = float

    def stride(self, i=None):
        return (8, 1) if i is None else (8, 1)[i]

    def numel(self):
        return 32

    def element_size(self):
        return 4

    def to(self, device, non_blocking=False):
        assert device == torch.device("cuda", 0)
        return self.here


def test_a_tensor_of_another_gpu_is_copied(lr):  # noqa: F811
    here, dev = torch.zeros(4, 8), torch.device("cuda", 0)
    for make in (lr._dev, lr._act, lr._par, lambda t, d: lr._rows(t, d)[0], lambda t, d: lr._rows(t, d, True)[0]):
        got = make(Elsewhere(here), dev)
        assert torch.is_tensor(got) and got.shape == (4, 8) and not isinstance(got, Elsewhere)
