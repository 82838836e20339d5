"""What the products' bounds alone would not show: the experts' products and the products of a few tokens at inputs where a
kernel's own way of summing could be seen."""
import pytest
import torch

from tests import _experts_plain as plain
from tests.test_gpu_experts import expert_weights, normal, offsets_of
from weight_only_quantization_act_b200 import awq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    awq.load_library()


def by_definition(X, codes, steps, zeros, gated):
    """Products in 64 bits term by term, so that an infinity meets each weight by itself."""
    P = torch.stack([(x.double() * plain.dequantized(codes, steps, zeros)).sum(1) for x in X])
    if not gated:
        return P
    a, b = P.chunk(2, dim=1)
    return a / (1 + torch.exp(-a)) * b


# rows of the one expert: the few-token kernel up to 8, the grouped one beyond; several slices at K = 4096
@pytest.mark.parametrize("rows", [1, 3, 8, 9, 40])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("K", [640, 4096])
def test_infinities_are_those_of_the_definition(rows, gated, K):
    """An infinity in X gives each output the sign of its weight, a NaN where the weight is zero or where two infinities
    meet; the other tokens keep their bits. The same for an expert's rows and for one layer."""
    O = 150
    parts, W = expert_weights(1, O, K, 90)
    X = normal((rows, K), 91)
    clean = awq.w4a16_experts(X.cuda(), offsets_of([rows]).cuda(), *W, gated=gated)
    X[0, 77] = float("inf")
    if rows > 1:
        X[1, K - 3] = -float("inf")
    if rows > 2:
        X[2, 5], X[2, K - 130] = float("inf"), float("inf")
    bad = min(rows, 3)
    ref = by_definition(X[:bad], *parts[0], gated)
    calls = [awq.w4a16_experts(X.cuda(), offsets_of([rows]).cuda(), *W, gated=gated)]
    if rows <= awq.GEMV_MAX_TOKENS:
        calls.append(awq.w4a16_gemv(X.cuda(), *(t[0] for t in W), gated=gated))
    for got in calls:
        assert torch.equal(got[bad:], clean[bad:])
        got = got[:bad].double().cpu()
        assert torch.equal(got.isnan(), ref.isnan())
        assert torch.equal(got.isinf(), ref.isinf())
        assert torch.equal(got[ref.isinf()], ref[ref.isinf()])
    assert bool(ref.isinf().any())  # the case shows it: not every output is a NaN
