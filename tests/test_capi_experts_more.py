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


def test_misaligned_words_are_refused(lib):
    """int32 and float arrays that do not start on 4 bytes, one at a time: a kernel would fault on them."""
    fake, odd = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 2)

    def refused(call, args, at):
        """`call` with the argument at this place off its alignment."""
        bad = list(args)
        bad[at] = odd
        assert call(*bad) == 1 and "4-byte aligned" in lib.awq_last_error().decode(), at

    gather = (fake, 4, 64, 64, 2, fake, 8, fake, None, fake, 64, None)
    for at in (5, 7):  # offsets, order
        refused(lib.awq_expert_gather, gather, at)
        refused(lib.awq_expert_gather_backward, gather, at)  # offsets, pos
    combine = (fake, 4, 64, 64, 2, fake, fake, fake, 64, None)
    for at in (5, 6):  # pos, weights
        refused(lib.awq_expert_combine, combine, at)
    back = (fake, 4, 64, 64, fake, 64, 2, fake, fake, fake, 64, fake, None)
    for at in (7, 8, 11):  # pos, weights, dweights
        refused(lib.awq_expert_combine_backward, back, at)
    refused(lib.awq_w4a16_experts, (fake, 4, 256, 256, fake, 8, fake, fake, fake, 64, 0, fake, 64, fake, 1 << 30, None), 4)
