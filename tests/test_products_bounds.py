"""The bounds reject what they are there for: wrong results made on the CPU."""
import pytest
import torch

from tests import _experts_plain as plain
from tests import _products_bounds as bounds


def made(K, wrong, one_sided):
    M, O = 8, 400
    X = torch.randn(M, K, generator=torch.Generator().manual_seed(K))
    X = (X.abs() if one_sided else X).bfloat16()
    codes, steps, zeros = plain.packed(O, K, K)
    zeros = torch.full_like(zeros, 8.0) if one_sided else zeros  # as for weights around zero
    ref = X.double() @ plain.dequantized(codes, steps, zeros).T
    W = plain.dequantized(codes, steps, zeros)
    if wrong == "bf16 weights":
        W = W.bfloat16().double()
    if wrong == "bf16 steps":
        W = plain.dequantized(codes, steps.bfloat16().float(), zeros)
    if wrong == "in-feature left out":
        W[:, K // 2 + 3] = 0
    if wrong == "one group's zero point":
        zeros = zeros.clone()
        zeros[:, 0] += 1
        W = plain.dequantized(codes, steps, zeros)
    got = X.double() @ W.T
    if wrong == "bf16 sums":
        parts = (X.double().view(M, -1, 128).transpose(0, 1) @ W.T.view(-1, 128, O)).float()
        total = torch.zeros(M, O, dtype=torch.bfloat16)
        for part in parts:
            total = (total.float() + part).bfloat16()
        got = total.double()
    if wrong == "sums of 1024 + q":  # 2^-23 of 1024 times the sum of x, once per MMA: what cutting a sum costs
        got = got + 8 * 2.0 ** -23 * 1024 * (X.double().abs().view(M, -1, 128).sum(2) @ steps.double().T)
    return got.bfloat16(), ref


@pytest.mark.parametrize("K", [512, 4096, 28672])
@pytest.mark.parametrize("one_sided", [False, True])
def test_right_results_pass(K, one_sided):
    got, ref = made(K, None, one_sided)
    bounds.assert_rounds(got, ref)


@pytest.mark.parametrize("K", [512, 4096, 28672])
@pytest.mark.parametrize("wrong", ["bf16 weights", "bf16 steps", "in-feature left out", "one group's zero point", "bf16 sums"])
def test_wrong_results_do_not(K, wrong):
    got, ref = made(K, wrong, False)
    with pytest.raises(AssertionError):
        bounds.assert_rounds(got, ref)


def test_lost_bits_of_one_sided_sums_do_not():
    got, ref = made(28672, "sums of 1024 + q", True)
    with pytest.raises(AssertionError):
        bounds.assert_rounds(got, ref)
