"""The stream argument of the tensor calls, without a GPU."""
from types import SimpleNamespace

import pytest
import torch

from decoder_greedy_decode_b200 import tensors


def test_a_stream_of_another_device_is_refused():
    here, there = torch.device("cuda", 0), torch.device("cuda", 1)
    with pytest.raises(ValueError, match="cuda:1"):
        tensors.guard(here, SimpleNamespace(device=there, cuda_stream=0))
    tensors.guard(here, SimpleNamespace(device=here, cuda_stream=0))
    for stream in (None, 0, 0x7F0000):     # the current one, and raw handles
        tensors.guard(here, stream)


def test_a_foreign_stream_is_taken_by_its_handle():
    tensors.guard(torch.device("cuda", 0), SimpleNamespace(device="its own device object", cuda_stream=0))
