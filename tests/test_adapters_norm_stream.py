"""The adapters' and norms' calls given a stream: one of another device than the tensors' is refused before anything is
allocated or launched; it would otherwise become current, and the kernels run on that device with this one's pointers."""
import pytest
import torch

from group_wise_affine_qlinear_b200 import _lib


class _Stream:
    def __init__(self, index):
        self.device = torch.device("cuda", index)


def _never(handle):
    raise AssertionError("called")


@pytest.mark.parametrize("dev,other", [(0, 1), (1, 0), (3, 2)])
def test_stream_of_another_device_is_refused(dev, other):
    with pytest.raises(ValueError, match=f"stream must be on cuda:{dev}, got one on cuda:{other}"):
        _lib._on_stream(dev, _Stream(other), _never)


@pytest.mark.gpu
def test_stream_of_the_tensors_device_is_taken():
    if not torch.cuda.is_available():
        pytest.fail("CUDA GPU required for -m gpu tests")
    for s in (torch.cuda.Stream(), torch.cuda.default_stream(), torch.cuda.ExternalStream(torch.cuda.Stream().cuda_stream)):
        assert _lib._on_stream(torch.cuda.current_device(), s, lambda handle: handle) == s.cuda_stream
