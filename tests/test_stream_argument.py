"""The stream argument of the 8-bit and distillation calls, as far as no CUDA call is made."""
import pytest
import torch

import sparse_mask_search_b200 as tsl


class _Stream:
    cuda_stream = 1234

    def __init__(self, device):
        self.device = torch.device(device)


def test_a_stream_of_another_device_is_refused():
    # it could not run the call, which would go to the current stream of the tensors' device instead
    with pytest.raises(ValueError, match="stream must be on cuda:0, is on cuda:1"):
        with tsl._on(torch.device("cuda:0"), _Stream("cuda:1")):
            pass
