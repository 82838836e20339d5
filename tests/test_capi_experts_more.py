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


def test_expert_weights_that_do_not_fit_are_refused():
    """Looked at before anything is launched: an expert without tokens would be packed with scales of X's width."""
    def bf16(*shape, device="cpu"):
        return torch.zeros(*shape, dtype=torch.bfloat16, device=device)

    X, ids = bf16(4, 256), torch.zeros(4, 1, dtype=torch.int64)
    for W in ([bf16(8, 256), bf16(8, 384)], [bf16(8, 384)] * 2, [bf16(8, 128)], [(bf16(8, 256), bf16(8, 512))],
              [bf16(8, 256), bf16(16, 256)], [bf16(8, 256), (bf16(8, 256), bf16(8, 256))], [], [bf16(8, 256)[None]],
              [bf16(8, 256, device="meta")]):
        with pytest.raises(ValueError):
            awq.quantize_experts(X, ids, W)
    with pytest.raises(TypeError):  # right shapes, but no GPU tensors
        awq.quantize_experts(X, ids, [bf16(8, 256), (bf16(4, 256), bf16(4, 256))])


def test_no_name_of_the_binding_is_given_twice():
    """A second definition takes the first one's place for all that is defined after it."""
    import ast
    import inspect

    names = [node.name for node in ast.parse(inspect.getsource(awq)).body
             if isinstance(node, (ast.FunctionDef, ast.ClassDef))]
    assert len(names) == len(set(names))
