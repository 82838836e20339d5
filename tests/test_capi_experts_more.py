"""More refusals of the experts' calls, on the host."""
import ctypes

import pytest
import torch

from weight_only_quantization_act_b200 import awq, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return awq.load_library()


def test_status_refusals(lib):
    for bad in (None, [0], torch.zeros(512, dtype=torch.uint8)):
        with pytest.raises(TypeError):
            awq.w4a16_status(bad)
