"""Streams of the microscaled and expert-routing calls, on the host."""
from __future__ import annotations

import pytest
import torch

import weight_only_bit_gemv_b200 as q4


class _Stream:
    """What the binding looks at of a torch.cuda.Stream."""

    def __init__(self, index):
        self.device = torch.device("cuda", index)
        self.cuda_stream = 0


def test_a_stream_of_another_device_is_refused():
    """A call there would run on the tensors' device, on its current stream,
    and not be ordered with the stream that was given."""
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        q4._Foreign(0, _Stream(1))
